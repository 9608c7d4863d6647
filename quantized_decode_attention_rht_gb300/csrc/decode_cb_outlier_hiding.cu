// The windowed decode's instances of keys with an outlier stream (see KVQ_CB_HIDES in decode_cb.cuh).
#define KVQ_CB_HIDES
#include "decode_cb_outlier.cu"
