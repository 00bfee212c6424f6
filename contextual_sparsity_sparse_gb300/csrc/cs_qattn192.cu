// Attention over the 4-bit KV cache, rows of 192 channels.
#define CS_QATTN_KERNELS
#include "cs_qattn.cuh"

template cudaError_t cs::run_qattn<192>(cs::QAttnK, int, int64_t, cudaStream_t);
