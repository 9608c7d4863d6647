// The windowed decode's instances of the codebook kernel's plain codes (see KVQ_CB_HIDES in decode_cb.cuh).
#define KVQ_CB_HIDES
#include "decode_cb.cu"
