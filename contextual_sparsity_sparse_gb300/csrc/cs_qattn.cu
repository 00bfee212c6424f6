// Attention over the 4-bit KV cache, in three plain passes:
//  1. s[row, i] = scale q . k_i for every query row and slot,
//  2. per row its maximum and sum, and out = sum_i p_i v_i,
//  3. per slot the sum of its p over the rows of its cache head.
#include "cs_qcache.cuh"

namespace cs {

namespace {

struct QAttnK {
    QAttnArgs a;
    float *logit;   // [batch, kv_heads, rows, cap]
    float *stat;    // [batch, kv_heads, rows, 2]: maximum and sum
    int group, rows;
};

__device__ __forceinline__ bool head_on(const QAttnK &k, int b, int h) {
    return !k.a.mask || (ld_dep(k.a.mask + (int64_t)b * ((k.a.heads + 31) / 32) + h / 32) >> (h % 32) & 1u);
}

__global__ void __launch_bounds__(128) qattn_logit_kernel(QAttnK k) {
    pdl_wait();
    pdl_launch_dependents();
    const QCacheK &c = k.a.c;
    const int row = blockIdx.y % k.rows, h = blockIdx.y / k.rows, b = blockIdx.z;
    const int t = row / k.group, head = h * k.group + row % k.group;
    __shared__ float q[256];
    for (int i = threadIdx.x; i < c.d; i += 128)
        q[i] = q_load1(k.a.q, b * k.a.q.ldb + t * k.a.q.ldt + head * k.a.q.ldh + i);
    __syncthreads();
    const int n = q_length(k.a.length, b, c.cap, k.a.err);
    const int i = blockIdx.x * 128 + threadIdx.x;
    if (i >= n) return;
    const int64_t slot = c.slot0(b, h) + i;
    float s = 0.f;
    for (int g = 0; g < c.d / kQGroup; ++g) {
        const uint32_t sz = c.ks[slot * (c.d / kQGroup) + g];
        float sc, of;
        half2x(sz, sc, of);
        for (int w = 0; w < kQGroup / 8; ++w) {
            const uint32_t x = reinterpret_cast<const uint32_t *>(c.k)[slot * (c.d / 8) + g * 8 + w];
#pragma unroll
            for (int e = 0; e < 8; ++e) s += q[g * kQGroup + w * 8 + e] * (of + sc * (float)(x >> (4 * e) & 15u));
        }
    }
    bool seen = head_on(k, b, head);
    if (k.a.q_pos) {
        const int p = c.pos[slot];
        seen = seen && p >= 0 && p <= ld_dep(k.a.q_pos + b) + t;
    }
    k.logit[((int64_t)(b * c.heads + h) * k.rows + row) * c.cap + i] = seen ? s * k.a.scale : -INFINITY;
}

__global__ void __launch_bounds__(256) qattn_row_kernel(QAttnK k) {
    pdl_wait();
    pdl_launch_dependents();
    const QCacheK &c = k.a.c;
    const int row = blockIdx.y % k.rows, h = blockIdx.y / k.rows, b = blockIdx.z;
    const int t = row / k.group, head = h * k.group + row % k.group;
    const int n = q_length(k.a.length, b, c.cap, nullptr);
    const float *s = k.logit + ((int64_t)(b * c.heads + h) * k.rows + row) * c.cap;
    __shared__ float red[8];
    float m = -INFINITY;
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += 256) {
        const float x = ld_dep(s + i);
        bad |= x != x;
        m = fmaxf(m, x);
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    __syncthreads();
    if (bad) m = NAN;
    if (m == -INFINITY) m = 0.f;
    float l = 0.f;
    for (int i = threadIdx.x; i < n; i += 256) l += expf(ld_dep(s + i) - m);
    l = warp_sum(l);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = l;
    __syncthreads();
    l = 0.f;
    for (int w = 0; w < 8; ++w) l += red[w];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (threadIdx.x == 0) {
        float *st = k.stat + ((int64_t)(b * c.heads + h) * k.rows + row) * 2;
        st[0] = m;
        st[1] = inv;
    }
    const int ch = threadIdx.x;
    if (ch >= c.d) return;
    float o = 0.f;
    for (int i = 0; i < n; ++i) {
        const int64_t slot = c.slot0(b, h) + i;
        const float p = expf(ld_dep(s + i) - m);
        if (p == 0.f) continue;
        float sc, of;
        half2x(c.vs[slot * (c.d / kQGroup) + ch / kQGroup], sc, of);
        o += p * (of + sc * (float)(c.v[slot * (c.d / 2) + ch / 2] >> (4 * (ch & 1)) & 15u));
    }
    q_store1(k.a.out, b * k.a.out.ldb + t * k.a.out.ldt + head * k.a.out.ldh + ch, o * inv);
}

__global__ void __launch_bounds__(256) qattn_weight_kernel(QAttnK k) {
    pdl_wait();
    pdl_launch_dependents();
    const QCacheK &c = k.a.c;
    const int h = blockIdx.y, b = blockIdx.z, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= q_length(k.a.length, b, c.cap, nullptr)) return;
    const int64_t slot = c.slot0(b, h) + i;
    float w = 0.f;
    for (int r = 0; r < k.rows; ++r) {
        const int64_t row = (int64_t)(b * c.heads + h) * k.rows + r;
        w += expf(ld_dep(k.logit + row * c.cap + i) - ld_dep(k.stat + row * 2)) * ld_dep(k.stat + row * 2 + 1);
    }
    k.a.weight[slot] = (k.a.decay == 0.f ? 0.f : k.a.decay * ld_dep(c.weight + slot)) + w;
}

}  // namespace

size_t qattn_scratch(int batch, int kv_heads, int cap, int d, int heads, int n_q, int sms) {
    const size_t rows = (size_t)batch * heads * n_q;
    return align256(rows * cap * sizeof(float)) + align256(rows * 2 * sizeof(float));
}

cudaError_t launch_qattn(const QAttnArgs &a, cudaStream_t s) {
    QAttnK k{a, reinterpret_cast<float *>(a.scratch), nullptr, a.heads / a.c.heads, 0};
    k.rows = k.group * a.n_q;
    k.stat = reinterpret_cast<float *>(a.scratch + align256((size_t)a.c.batch * a.heads * a.n_q * a.c.cap * sizeof(float)));
    const dim3 rows(1, a.c.heads * k.rows, a.c.batch);
    cudaError_t e = launch(qattn_logit_kernel, dim3((a.c.cap + 127) / 128, rows.y, rows.z), dim3(128), 0, s, pdl_enabled(), k);
    if (e == cudaSuccess) e = launch(qattn_row_kernel, rows, dim3(256), 0, s, pdl_enabled(), k);
    if (e == cudaSuccess && a.weight)
        e = launch(qattn_weight_kernel, dim3((a.c.cap + 255) / 256, a.c.heads, a.c.batch), dim3(256), 0, s, pdl_enabled(), k);
    return e;
}

}  // namespace cs
