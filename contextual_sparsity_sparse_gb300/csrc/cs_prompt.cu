// Attention of whole prompts, packed one behind the other: causal or not, with
// grouped heads.
#include "cs_qcache.cuh"

namespace cs {

namespace {

constexpr int kMaxGroup = 128;   // query heads of one key/value head

struct PromptK {
    QRowsK q, k, v, out;
    int heads, kv, group, d, batch, q_total, k_total, causal;
    const int32_t *q_start, *k_start;
    float scale;
    uint32_t *err;
};

// The next sequence's rows, [end, its end), where starts are clamped to [0, total] and do not fall.
__device__ __forceinline__ int2 next_rows(const int32_t *start, int b, int total, int end, uint32_t *err) {
    const int x = b == 0 ? ld_dep(start) : end, y = ld_dep(start + b + 1);
    const int first = min(max(x, 0), total), last = min(max(y, first), total);
    if (x != first || y != last) atomicOr(err, CS_DEVERR_COUNT);
    return make_int2(first, last);
}

// One row's attention by one warp, key by key: lane l has channels l + 32 i.
template <typename T, int D>
__device__ __forceinline__ void prompt_row(const PromptK &a, int token, int head, int k0, int keys, float (&o)[D / 32]) {
    const int lane = threadIdx.x & 31;
    const T *q = reinterpret_cast<const T *>(a.q.p) + token * a.q.ldt + head * a.q.ldh;
    const T *k = reinterpret_cast<const T *>(a.k.p) + k0 * a.k.ldt + head / a.group * a.k.ldh;
    const T *v = reinterpret_cast<const T *>(a.v.p) + k0 * a.v.ldt + head / a.group * a.v.ldh;
    float x[D / 32], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        x[i] = a.scale * (float)q[lane + 32 * i];
        o[i] = 0.f;
    }
    for (int j = 0; j < keys; ++j) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s = fmaf(x[i], (float)k[j * a.k.ldt + lane + 32 * i], s);
        s = warp_sum(s);
        const float up = fmaxf(m, s), base = up == -INFINITY ? 0.f : up;
        const float keep = expf(m - base), p = expf(s - base);
        m = up;
        l = fmaf(l, keep, p);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], keep, p * (float)v[j * a.v.ldt + lane + 32 * i]);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = l == 0.f ? 0.f : o[i] / l;
}

template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_kernel(PromptK a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (row >= (int64_t)a.q_total * a.heads) return;
    const int token = (int)(row / a.heads), head = (int)(row % a.heads);
    int2 q{}, k{};
    for (int b = 0; b < a.batch; ++b) {
        q = next_rows(a.q_start, b, a.q_total, q.y, a.err);
        k = next_rows(a.k_start, b, a.k_total, k.y, a.err);
        if (token < q.x || token >= q.y) continue;
        const int n = k.y - k.x, keys = a.causal ? min(n, max(0, token - q.x + 1 + n - (q.y - q.x))) : n;
        float o[D / 32];
        prompt_row<T, D>(a, token, head, k.x, keys, o);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            q_store1(a.out, token * a.out.ldt + head * a.out.ldh + (threadIdx.x & 31) + 32 * i, o[i]);
        return;
    }
}

bool prompt_sizes(int batch, int n_heads, int kv_heads, int d_head, int q_total, int k_total) {
    return batch >= 1 && batch <= kQMaxBatch && kv_heads >= 1 && n_heads >= kv_heads && n_heads <= kMaxHeads &&
           n_heads % kv_heads == 0 && n_heads / kv_heads <= kMaxGroup && (d_head == 64 || d_head == 128) && q_total >= 0 &&
           q_total <= kMaxTokens && k_total >= 0 && k_total <= kMaxTokens;
}

}  // namespace

}  // namespace cs

using namespace cs;

extern "C" {

size_t cs_prompt_workspace_size(int batch, int n_heads, int kv_heads, int d_head, int q_total, int k_total) {
    if (!prompt_sizes(batch, n_heads, kv_heads, d_head, q_total, k_total)) return 0;
    return kControlBytes;
}

cs_status cs_prompt_attention(const cs_head_rows *q, const cs_head_rows *k, const cs_head_rows *v, int n_heads,
                              int kv_heads, int d_head, int batch, const int32_t *q_start, int q_total,
                              const int32_t *k_start, int k_total, int causal, float scale,
                              const cs_head_rows *out, void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_prompt_attention";
    PromptK a;
    CS_CHECK(q_total >= 0 && k_total >= 0, "%s: q_total and k_total must be >= 0 (%d, %d)", who, q_total, k_total);
    cs_status st = check_rows(q, q_total == 0, "q", who, &a.q);
    if (st == CS_OK) st = check_rows(k, k_total == 0, "k", who, &a.k);
    if (st == CS_OK) st = check_rows(v, k_total == 0, "v", who, &a.v);
    if (st == CS_OK) st = check_rows(out, q_total == 0, "out", who, &a.out);
    if (st != CS_OK) return st;
    CS_CHECK(q->dtype == k->dtype && q->dtype == v->dtype && q->dtype == out->dtype, "%s: q, k, v and out differ in dtype", who);
    CS_CHECK(batch >= 1 && n_heads >= 1 && kv_heads >= 1 && n_heads % kv_heads == 0,
             "%s: batch must be >= 1 and n_heads a multiple of kv_heads (%d, %d, %d)", who, batch, n_heads, kv_heads);
    if (q->dtype == CS_F32) {
        set_error("%s: takes fp16 and bf16", who);
        return CS_ERR_UNSUPPORTED;
    }
    if (!prompt_sizes(batch, n_heads, kv_heads, d_head, q_total, k_total)) {
        set_error("%s: d_head=%d is not 64 or 128, or batch %d, n_heads %d, n_heads / kv_heads %d or tokens %d, %d above %d, %d, %d, %d",
                  who, d_head, batch, n_heads, n_heads / kv_heads, q_total, k_total, kQMaxBatch, kMaxHeads, kMaxGroup, kMaxTokens);
        return CS_ERR_UNSUPPORTED;
    }
    CS_CHECK((q_total == 0 || (a.q.vec && a.out.vec)) && (k_total == 0 || (a.k.vec && a.v.vec)),
             "%s: every row of q, k, v and out must start on a 16-byte boundary", who);
    CS_CHECK(q_start && aligned(q_start, 4) && aligned(k_start, 4), "%s: q_start is null, or q_start or k_start misaligned", who);
    CS_CHECK(k_start || q_total == k_total, "%s: without k_start, q_total and k_total must be equal (%d, %d)", who, q_total, k_total);
    CS_CHECK(q_total == 0 || (out->data != q->data && out->data != k->data && out->data != v->data),
             "%s: out must not be q, k or v", who);
    CS_CHECK(scale == scale && scale - scale == 0.f, "%s: scale must be finite", who);
    st = check_qws(ws, ws_bytes, cs_prompt_workspace_size(batch, n_heads, kv_heads, d_head, q_total, k_total), who);
    if (st != CS_OK) return st;
    if (q_total == 0) return CS_OK;
    a.heads = n_heads;
    a.kv = kv_heads;
    a.group = n_heads / kv_heads;
    a.d = d_head;
    a.batch = batch;
    a.q_total = q_total;
    a.k_total = k_total;
    a.causal = causal != 0;
    a.q_start = q_start;
    a.k_start = k_start ? k_start : q_start;
    a.scale = scale != 0.f ? scale : 1.f / sqrtf((float)d_head);
    a.err = static_cast<uint32_t *>(ws);
    auto go = [&](auto kernel) {
        return launch(kernel, dim3((unsigned)(((int64_t)q_total * n_heads + 7) / 8)), dim3(256), 0, (cudaStream_t)stream,
                      pdl_enabled(), a);
    };
    const bool h = q->dtype == CS_F16;
    const cudaError_t e = d_head == 64 ? (h ? go(prompt_kernel<__half, 64>) : go(prompt_kernel<__nv_bfloat16, 64>))
                                       : (h ? go(prompt_kernel<__half, 128>) : go(prompt_kernel<__nv_bfloat16, 128>));
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
