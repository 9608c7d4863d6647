// The windowed decode's instances of its 16-warp instances (see KVQ_CB_HIDES in decode_cb.cuh).
#define KVQ_CB_HIDES
#include "decode_cb_wide.cu"
