// Sequences of a 4-bit KV cache taken over by others: samples from one prompt,
// beams that change places.
//
// Bound by memory: every copy is written once, and a source that several take is
// read once from memory and then found in the second-level cache.  A CTA has a
// range of slots of one head in all sequences, so that in place it can read
// what all of them take before it writes any: only such a range has to fit
// shared memory, whatever the lengths.
#include "cs_qcache.cuh"

namespace cs {

namespace {

constexpr int kForkThreads = 256;

// One of a cache's six arrays: bytes of a slot, and how wide it can be copied.
struct ForkArray {
    const char *src;
    char *dst;
    int row, wide;
};
struct ForkK {
    ForkArray part[6];
    const int32_t *source, *length;
    int from, to, heads, cap_src, cap_dst, slots, parts;
    int64_t ldb_src, ldh_src, ldb_dst, ldh_dst;
    int in_place;
    uint32_t *err;
};

// The sequence that i takes, or -1: none, or its own in place; and its slots.
__device__ __forceinline__ int fork_source(const ForkK &a, int i, int &len) {
    const int s = ld_dep(a.source + i);
    len = 0;
    if (s < 0 || s >= a.from) {
        if (s != -1) atomicOr(a.err, CS_DEVERR_INDEX);
        return -1;
    }
    const int n = ld_dep(a.length + s);
    len = min(max(n, 0), min(a.cap_src, a.cap_dst));
    if (n != len) atomicOr(a.err, CS_DEVERR_COUNT);
    return a.in_place && s == i ? -1 : s;
}

template <typename V>
__device__ __forceinline__ void fork_copy(const ForkK &a, const ForkArray &p, int h, int t0) {
    const int units = a.slots * p.row / (int)sizeof(V);   // of the range
    for (int u = threadIdx.x; u < units; u += kForkThreads) {
        const int slot = t0 + u * (int)sizeof(V) / p.row;
        for (int i = 0; i < a.to; ++i) {
            int len;
            const int s = fork_source(a, i, len);
            if (s < 0 || slot >= len) continue;
            const int64_t at = ((int64_t)t0 * p.row) / (int)sizeof(V) + u;
            reinterpret_cast<V *>(p.dst + (i * a.ldb_dst + h * a.ldh_dst) * p.row)[at] =
                ld_dep(reinterpret_cast<const V *>(p.src + (s * a.ldb_src + h * a.ldh_src) * p.row) + at);
        }
    }
}

// One thread's sequences in order, so this is for copies between caches alone.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkK a) {
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.y, t0 = blockIdx.x * a.slots;
    for (int x = 0; x < a.parts; ++x) fork_copy<uint32_t>(a, a.part[x], h, t0);
}

// In place: words of all sequences, then written.
__global__ void __launch_bounds__(kForkThreads) fork_in_place_kernel(ForkK a) {
    extern __shared__ uint32_t held[];   // [to, slots x words of a slot]
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.y, t0 = blockIdx.x * a.slots;
    for (int x = 0; x < a.parts; ++x) {
        const ForkArray &p = a.part[x];
        const int words = a.slots * p.row / 4;
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t e = threadIdx.x; e < (int64_t)words * a.to; e += kForkThreads) {
                const int i = (int)(e / words), u = (int)(e % words);
                int len;
                const int s = fork_source(a, i, len);
                if (s < 0 || t0 + u * 4 / p.row >= len) continue;
                const int64_t at = (int64_t)t0 * p.row / 4 + u;
                if (pass == 0) held[e] = ld_dep(reinterpret_cast<const uint32_t *>(p.src + (s * a.ldb_src + h * a.ldh_src) * p.row) + at);
                else reinterpret_cast<uint32_t *>(p.dst + (i * a.ldb_dst + h * a.ldh_dst) * p.row)[at] = held[e];
            }
            __syncthreads();
        }
    }
}

}  // namespace

}  // namespace cs

using namespace cs;

extern "C" {

cs_status cs_qcache_fork(const cs_qcache *src, const int32_t *source, const int32_t *length, const cs_qcache *dst,
                         void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_qcache_fork";
    QCacheK c, to;
    cs_status st = check_cache(src, true, who, &c);
    if (st == CS_OK) st = check_cache(dst ? dst : src, true, who, &to);
    if (st != CS_OK) return st;
    CS_CHECK(to.heads == c.heads && to.d == c.d, "%s: dst and src differ in n_heads or d_head", who);
    CS_CHECK((to.weight != nullptr) == (c.weight != nullptr) && (to.pos != nullptr) == (c.pos != nullptr),
             "%s: dst needs weights (positions) if and only if src has them", who);
    const int same = (to.k == c.k) + (to.v == c.v) + (to.ks == c.ks) + (to.vs == c.vs) + (c.weight && to.weight == c.weight) +
                     (c.pos && to.pos == c.pos);
    const int all = 4 + (c.weight != nullptr) + (c.pos != nullptr);
    CS_CHECK(same == 0 || (same == all && to.batch == c.batch && to.cap == c.cap && (to.batch == 1 || to.ldb == c.ldb) &&
                           (to.heads == 1 || to.ldh == c.ldh)),
             "%s: dst must be src or have memory of its own", who);
    CS_CHECK(source && aligned(source, 4) && length && aligned(length, 4), "%s: source or length is null or misaligned", who);
    st = check_qws(ws, ws_bytes, kControlBytes, who);
    if (st != CS_OK) return st;
    ForkK a{};
    const int g4 = c.d / kQGroup * 4;
    auto put = [&](const void *s, void *d, int row) {
        if (s) a.part[a.parts++] = ForkArray{static_cast<const char *>(s), static_cast<char *>(d), row, 4};
    };
    put(c.k, to.k, c.d / 2);
    put(c.v, to.v, c.d / 2);
    put(c.ks, to.ks, g4);
    put(c.vs, to.vs, g4);
    put(c.weight, to.weight, 4);
    put(c.pos, to.pos, 4);
    a.source = source;
    a.length = length;
    a.from = c.batch;
    a.to = to.batch;
    a.heads = c.heads;
    a.cap_src = c.cap;
    a.cap_dst = to.cap;
    a.ldb_src = c.ldb;
    a.ldh_src = c.ldh;
    a.ldb_dst = to.ldb;
    a.ldh_dst = to.ldh;
    a.in_place = same == all;
    a.err = static_cast<uint32_t *>(ws);
    a.slots = 64;
    cudaError_t e;
    if (a.in_place) {
        a.slots = 1;
        e = allow_smem(reinterpret_cast<const void *>(&fork_in_place_kernel));
        const size_t smem = (size_t)a.to * a.slots * (c.d / 2);
        if (smem > 200 * 1024) {
            set_error("%s: %d sequences in place are too many", who, a.to);
            return CS_ERR_UNSUPPORTED;
        }
        if (e == cudaSuccess)
            e = launch(fork_in_place_kernel, dim3((c.cap + a.slots - 1) / a.slots, c.heads), dim3(kForkThreads), smem,
                       (cudaStream_t)stream, pdl_enabled(), a);
    } else {
        e = launch(fork_kernel, dim3((c.cap + a.slots - 1) / a.slots, c.heads), dim3(kForkThreads), 0, (cudaStream_t)stream,
                   pdl_enabled(), a);
    }
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
