// Attention for a tree of drafted tokens over the 4-bit KV cache.
#include "cs_qcache.cuh"

namespace cs {

namespace {

constexpr int kMaxTree = 128;   // drafted tokens of a sequence

struct TreeK {
    QCacheK c;
    QRowsK q, k, v, out;
    int heads, group, n;
    const int32_t *length, *parent, *n_new;
    float scale;
    uint32_t *err;
};

// Drafted rows as the cache would take them: within fp16's range, NaN as 0.
__device__ __forceinline__ float as_drafted(float x) {
    return x != x ? 0.f : __half2float(__float2half_rn(fminf(fmaxf(x, -65504.f), 65504.f)));
}

__device__ __forceinline__ int tree_count(const TreeK &a, int b) {
    if (!a.n_new) return a.n;
    const int n = ld_dep(a.n_new + b);
    if (n < 0 || n > a.n) atomicOr(a.err, CS_DEVERR_COUNT);
    return min(max(n, 0), a.n);
}

__device__ __forceinline__ int tree_parent(const TreeK &a, int b, int t) {
    if (!a.parent) return t - 1;
    const int p = ld_dep(a.parent + (int64_t)b * a.n + t);
    if (p >= -1 && p < t) return p;
    atomicOr(a.err, CS_DEVERR_INDEX);
    return -1;
}

template <int D>
__global__ void __launch_bounds__(256) tree_kernel(TreeK a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (row >= (int64_t)a.c.batch * a.n * a.heads) return;
    const int lane = threadIdx.x & 31, head = (int)(row % a.heads), t = (int)(row / a.heads % a.n);
    const int b = (int)(row / a.heads / a.n), h = head / a.group;
    const int len = q_length(a.length, b, a.c.cap, a.err), n = tree_count(a, b);
    float x[D / 32], o[D / 32], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        x[i] = a.scale * q_load1(a.q, b * a.q.ldb + t * a.q.ldt + head * a.q.ldh + lane + 32 * i);
        o[i] = 0.f;
    }
    auto add = [&](const float (&k)[D / 32], const float (&v)[D / 32]) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s = fmaf(x[i], k[i], s);
        s = warp_sum(s);
        const float up = fmaxf(m, s), base = up == -INFINITY ? 0.f : up;
        const float keep = expf(m - base), p = expf(s - base);
        m = up;
        l = fmaf(l, keep, p);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], keep, p * v[i]);
    };
    if (t < n) {
        const int64_t slot0 = a.c.slot0(b, h);
        for (int j = 0; j < len; ++j) {
            if (a.c.pos && ld_dep(a.c.pos + slot0 + j) < 0) continue;
            float k[D / 32], v[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int ch = lane + 32 * i;
                float s, z;
                half2x(ld_dep(a.c.ks + (slot0 + j) * (D / kQGroup) + ch / kQGroup), s, z);
                k[i] = fmaf(s, (float)(ld_dep(a.c.k + (slot0 + j) * (D / 2) + ch / 2) >> (ch & 1) * 4 & 15), z);
                half2x(ld_dep(a.c.vs + (slot0 + j) * (D / kQGroup) + ch / kQGroup), s, z);
                v[i] = fmaf(s, (float)(ld_dep(a.c.v + (slot0 + j) * (D / 2) + ch / 2) >> (ch & 1) * 4 & 15), z);
            }
            add(k, v);
        }
        for (int u = t; u >= 0; u = tree_parent(a, b, u)) {
            float k[D / 32], v[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                k[i] = as_drafted(q_load1(a.k, b * a.k.ldb + u * a.k.ldt + h * a.k.ldh + lane + 32 * i));
                v[i] = as_drafted(q_load1(a.v, b * a.v.ldb + u * a.v.ldt + h * a.v.ldh + lane + 32 * i));
            }
            add(k, v);
        }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        q_store1(a.out, b * a.out.ldb + t * a.out.ldt + head * a.out.ldh + lane + 32 * i, l == 0.f ? 0.f : o[i] / l);
}

}  // namespace

}  // namespace cs

using namespace cs;

extern "C" {

size_t cs_qcache_tree_workspace_size(int batch, int kv_heads, int capacity, int d_head, int n_heads, int n) {
    if (batch < 1 || batch > kQMaxBatch || kv_heads < 1 || kv_heads > kMaxHeads || capacity < 1 || capacity > kMaxCapacity ||
        (d_head != 64 && d_head != 128) || n_heads < kv_heads || n_heads % kv_heads || n < 1 || n > kMaxTree ||
        (int64_t)n_heads / kv_heads * n > kQMaxRows)
        return 0;
    return kControlBytes;
}

cs_status cs_qcache_tree_attention(const cs_qcache *cache, const cs_head_rows *q, const cs_head_rows *k,
                                   const cs_head_rows *v, int n_heads, int n, const int32_t *length,
                                   const int32_t *parent, const int32_t *n_new, float scale,
                                   const cs_head_rows *out, void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_qcache_tree_attention";
    TreeK a;
    cs_status st = check_cache(cache, true, who, &a.c);
    if (st == CS_OK) st = check_rows(q, false, "q", who, &a.q);
    if (st == CS_OK) st = check_rows(k, false, "k", who, &a.k);
    if (st == CS_OK) st = check_rows(v, false, "v", who, &a.v);
    if (st == CS_OK) st = check_rows(out, false, "out", who, &a.out);
    if (st != CS_OK) return st;
    CS_CHECK(q->dtype == k->dtype && q->dtype == v->dtype && q->dtype == out->dtype, "%s: q, k, v and out differ in dtype", who);
    CS_CHECK(out->data != q->data && out->data != k->data && out->data != v->data, "%s: out must not be q, k or v", who);
    CS_CHECK(n_heads >= 1 && n_heads % cache->n_heads == 0, "%s: n_heads=%d is not a multiple of the cache's %d", who, n_heads,
             cache->n_heads);
    CS_CHECK(n >= 1, "%s: n=%d is below 1", who, n);
    if (q->dtype == CS_F32 || (cache->d_head != 64 && cache->d_head != 128)) {
        set_error("%s: takes fp16 and bf16, and d_head 64 or 128 (%d)", who, cache->d_head);
        return CS_ERR_UNSUPPORTED;
    }
    if (n > kMaxTree || (int64_t)n_heads / cache->n_heads * n > kQMaxRows) {
        set_error("%s: n=%d above %d, or %lld query rows per cache head above %d", who, n, kMaxTree,
                  (long long)n_heads / cache->n_heads * n, kQMaxRows);
        return CS_ERR_UNSUPPORTED;
    }
    CS_CHECK(length && aligned(length, 4), "%s: length is null or misaligned", who);
    CS_CHECK(aligned(parent, 4) && aligned(n_new, 4), "%s: parent and n_new must be 4-byte aligned", who);
    CS_CHECK(scale == scale && scale - scale == 0.f, "%s: scale must be finite", who);
    st = check_qws(ws, ws_bytes,
                   cs_qcache_tree_workspace_size(cache->batch, cache->n_heads, cache->capacity, cache->d_head, n_heads, n), who);
    if (st != CS_OK) return st;
    a.heads = n_heads;
    a.group = n_heads / cache->n_heads;
    a.n = n;
    a.length = length;
    a.parent = parent;
    a.n_new = n_new;
    a.scale = scale != 0.f ? scale : 1.f / sqrtf((float)cache->d_head);
    a.err = static_cast<uint32_t *>(ws);
    const int64_t rows = (int64_t)a.c.batch * n * n_heads;
    auto go = [&](auto kernel) {
        return launch(kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, (cudaStream_t)stream, pdl_enabled(), a);
    };
    const cudaError_t e = a.c.d == 64 ? go(tree_kernel<64>) : go(tree_kernel<128>);
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
