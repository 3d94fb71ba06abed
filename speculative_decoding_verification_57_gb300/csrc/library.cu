// library.cu -- the library's one translation unit: the verify step's C ABI
// and the calls on the paged KV cache (they share the handle).
#include "specv.cu"

#include "cache_api.cuh"
