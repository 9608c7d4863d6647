// The windowed decode's instances of eight query heads per kv head (see KVQ_CB_HIDES in decode_cb.cuh).
#define KVQ_CB_HIDES
#include "decode_cb_g8.cu"
