// Attention over the 4-bit KV cache, rows of 128 channels.
#define CS_QATTN_KERNELS
#include "cs_qattn.cuh"

template cudaError_t cs::run_qattn<128>(cs::QAttnK, int, int64_t, cudaStream_t);
