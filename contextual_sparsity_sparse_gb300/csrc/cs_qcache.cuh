// What the translation units of the 4-bit KV cache share.
#pragma once

#include "cs_internal.cuh"

namespace cs {

constexpr int kQGroup = 64;        // channels that share a scale and an offset
constexpr int kQMaxBatch = 4096;
constexpr int kQMaxRows = 1024;    // query rows of one cache head: n_q * n_heads / kv_heads

// A checked cs_qcache: strides filled in, pointers as the kernels use them.
struct QCacheK {
    uint8_t *k, *v;
    uint32_t *ks, *vs;   // (scale, offset) pairs, one word per group
    float *weight;
    int32_t *pos;
    int batch, heads, cap, d;
    int64_t ldb, ldh;    // slots

    __device__ __forceinline__ int64_t slot0(int b, int h) const { return b * ldb + h * ldh; }
};

struct QRowsK {
    char *p;
    int64_t ldb, ldt, ldh;   // elements
    int dt;
    int vec;                 // every row starts on a 16-byte boundary
};

struct QAttnArgs {
    QCacheK c;
    QRowsK q, out;
    int heads, n_q;
    const int32_t *length, *q_pos;
    const uint32_t *mask;
    float scale, decay;
    float *weight;           // or null
    uint32_t *err;
    char *scratch;           // the workspace behind its control words
    int sms;
};
// weights: whether the call gathers them
size_t qattn_scratch(int batch, int kv_heads, int cap, int d, int heads, int n_q, bool weights, int sms);
cudaError_t launch_qattn(const QAttnArgs &a, cudaStream_t s);

__device__ __forceinline__ float q_load1(const QRowsK &r, int64_t i) {
    if (r.dt == CS_F32) return reinterpret_cast<const float *>(r.p)[i];
    if (r.dt == CS_F16) return __half2float(reinterpret_cast<const __half *>(r.p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(r.p)[i]);
}
__device__ __forceinline__ void q_store1(const QRowsK &r, int64_t i, float v) {
    if (r.dt == CS_F32) reinterpret_cast<float *>(r.p)[i] = v;
    else if (r.dt == CS_F16) reinterpret_cast<__half *>(r.p)[i] = __float2half_rn(v);
    else reinterpret_cast<__nv_bfloat16 *>(r.p)[i] = __float2bfloat16_rn(v);
}

// The number of slots in use, clamped to [0, cap]; a value outside is flagged.
__device__ __forceinline__ int q_length(const int32_t *length, int b, int cap, uint32_t *err) {
    const int n = ld_dep(length + b);
    if (n < 0 || n > cap) {
        if (err) atomicOr(err, CS_DEVERR_COUNT);
        return n < 0 ? 0 : cap;
    }
    return n;
}

}  // namespace cs
