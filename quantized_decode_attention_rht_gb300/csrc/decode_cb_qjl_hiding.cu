// The windowed decode's instances of keys with a residual sketch (see KVQ_CB_HIDES in decode_cb.cuh).
#define KVQ_CB_HIDES
#include "decode_cb_qjl.cu"
