// Sequences of a 4-bit KV cache taken over by others: samples from one prompt,
// beams that change places.
//
// Bound by memory and the way to it: every copy is written once, and a source read
// once however many take it.  All ranges of kForkSlots slots of the heads of the
// sources that somebody takes are one list, which the CTAs go through; a CTA's
// threads take a range's six arrays as one list of steps, all loads before the
// stores, and store to every sequence that takes the source.  15 copies of 5 MB
// (writing 80 MB alone takes 12 us) take 15.4 us, ranges of 32 or 128 slots 18.9 and 23.1; with a CTA
// for each copy and range, which reads a source again for each, 24; with one for
// each source and range, most of which nobody takes, 35.
//
// In place, a sequence that is read may be written, too.  Then a CTA does a range
// of all sequences, in pieces of which it reads what they take into shared memory
// before it writes any, whatever the lengths.  That is ten times slower: 32 beams
// of up to 2,049 slots of 8 heads of 64 that change places take 178 us so, and 17
// into another cache; two of them alone 86 and 5 (4 bytes a step, behind a
// division and two loads of which sequence and how long).
#include "cs_qcache.cuh"

namespace cs {

namespace {

constexpr int kForkThreads = 256;
constexpr int kForkSlots = 64;           // of a range: a multiple of 16, so that every array's part starts a step
constexpr int kForkSteps = 3;            // of a thread, under way together
constexpr int kForkHeld = 32 * 1024;     // bytes read ahead in place

// One of a cache's six arrays: bytes of a slot, and of a copy's step (16, 8 or 4, by what all rows start on).
struct ForkArray {
    const char *src;
    char *dst;
    int row, wide;
};
struct ForkK {
    ForkArray part[6];
    const int32_t *source, *length;
    int begin[7];                        // the arrays' first steps in a range's list
    int from, to, heads, cap_src, cap_dst, parts;
    int64_t ldb_src, ldh_src, ldb_dst, ldh_dst;
    int in_place;
    uint32_t *err;
};

// The sequence that i takes, or -1: none, or its own in place.
__device__ __forceinline__ int fork_source(const ForkK &a, int i) {
    const int s = ld_dep(a.source + i);
    return s < 0 || s >= a.from || (a.in_place && s == i) ? -1 : s;
}
__device__ __forceinline__ int fork_length(const ForkK &a, int s) {
    return min(max(ld_dep(a.length + s), 0), min(a.cap_src, a.cap_dst));
}

__device__ __forceinline__ const char *fork_from(const ForkK &a, const ForkArray &p, int s, int h) {
    return p.src + (s * a.ldb_src + h * a.ldh_src) * p.row;
}
__device__ __forceinline__ char *fork_to(const ForkK &a, const ForkArray &p, int i, int h) {
    return p.dst + (i * a.ldb_dst + h * a.ldh_dst) * p.row;
}

template <typename V>
__device__ __forceinline__ void fork_load(uint4 &v, const char *p) { *reinterpret_cast<V *>(&v) = ld_dep(reinterpret_cast<const V *>(p)); }
template <typename V>
__device__ __forceinline__ void fork_store(const uint4 &v, char *p) { *reinterpret_cast<V *>(p) = *reinterpret_cast<const V *>(&v); }

// Slots t0 .. of head h of sequence s, of which it has len, to the sequences of the chain that begins with `taker`.
__device__ __forceinline__ void fork_copy(const ForkK &a, int s, int len, int h, int t0, int taker, const int *next) {
    const int total = a.begin[a.parts];
    for (int u0 = threadIdx.x; u0 < total; u0 += kForkSteps * kForkThreads) {
        uint4 v[kForkSteps];
        char *to[kForkSteps];    // in sequence 0
        int row[kForkSteps], bytes[kForkSteps];   // bytes of the step: 0 none, less than its width at a source's end
#pragma unroll
        for (int k = 0; k < kForkSteps; ++k) {
            const int u = u0 + k * kForkThreads;
            bytes[k] = 0;
            if (u >= total) continue;
            int x = 0;
#pragma unroll
            for (int e = 1; e < 6; ++e) x += e < a.parts && u >= a.begin[e];
            const ForkArray &p = a.part[x];
            const int64_t at = (int64_t)t0 * p.row + (int64_t)(u - a.begin[x]) * p.wide;
            bytes[k] = (int)max((int64_t)0, min((int64_t)p.wide, (int64_t)len * p.row - at));
            if (bytes[k] == 0) continue;
            const char *from = fork_from(a, p, s, h) + at;
            to[k] = fork_to(a, p, 0, h) + at;
            row[k] = p.row;
            if (bytes[k] == 16) fork_load<uint4>(v[k], from);
            else if (bytes[k] == 8) fork_load<uint2>(v[k], from);
            else if (bytes[k] == 4) fork_load<uint32_t>(v[k], from);
            else {
                fork_load<uint2>(v[k], from);
                v[k].z = ld_dep(reinterpret_cast<const uint32_t *>(from) + 2);
            }
        }
        for (int i = taker; i >= 0; i = next[i]) {
            const int64_t slots = i * a.ldb_dst;
#pragma unroll
            for (int k = 0; k < kForkSteps; ++k) {
                char *at = to[k] + slots * row[k];
                if (bytes[k] == 16) fork_store<uint4>(v[k], at);
                else if (bytes[k] == 8) fork_store<uint2>(v[k], at);
                else if (bytes[k] == 4) fork_store<uint32_t>(v[k], at);
                else if (bytes[k]) {
                    fork_store<uint2>(v[k], at);
                    reinterpret_cast<uint32_t *>(at)[2] = v[k].z;
                }
            }
        }
    }
}

// In place, a sequence that is read is written, too: what a piece's sequences take is read before any of it is written.
__device__ __forceinline__ void fork_held(const ForkK &a, const ForkArray &p, int h, int t0, int t1, uint32_t *held) {
    const int fit = max(kForkHeld / (a.to * p.row), 1);   // slots of a piece
    for (; t0 < t1; t0 += fit) {
        const int words = min(fit, t1 - t0) * p.row / 4;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t e = threadIdx.x; e < (int64_t)words * a.to; e += kForkThreads) {
                const int i = (int)(e / words), u = (int)(e - (int64_t)i * words);
                const int s = fork_source(a, i);
                if (s < 0 || t0 + u * 4 / p.row >= fork_length(a, s)) continue;
                const int64_t at = (int64_t)t0 * p.row / 4 + u;
                if (pass == 0) held[e] = ld_dep(reinterpret_cast<const uint32_t *>(fork_from(a, p, s, h)) + at);
                else reinterpret_cast<uint32_t *>(fork_to(a, p, i, h))[at] = held[e];
            }
            __syncthreads();
        }
    }
}

__global__ void __launch_bounds__(kForkThreads, 4) fork_kernel(ForkK a) {
    // who takes a source, as chains; the sources that are taken, and their ranges' places in the list.  In place, where
    // sequences are read and written, what is held (kForkHeld bytes, or one slot's rows of all sequences).
    extern __shared__ uint32_t smem[];
    __shared__ int scan[32], active, ranges;
    int *taker = reinterpret_cast<int *>(smem), *next = taker + a.from, *taken = next + a.to, *place = taken + a.from;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    for (int s = tid; s < a.from; s += kForkThreads) taker[s] = -1;
    if (tid == 0) active = ranges = 0;
    __syncthreads();
    bool both = false;   // whether some sequence is read and written
    for (int i = tid; i < a.to; i += kForkThreads) {
        const int x = ld_dep(a.source + i), s = fork_source(a, i);
        if (blockIdx.x == 0) {
            // tell what is wrong
            if (x != -1 && (x < 0 || x >= a.from)) atomicOr(a.err, CS_DEVERR_INDEX);
            else if (x >= 0 && ld_dep(a.length + x) != fork_length(a, x)) atomicOr(a.err, CS_DEVERR_COUNT);
        }
        if (s < 0) continue;
        next[i] = atomicExch(&taker[s], i);
        if (a.in_place) both |= fork_source(a, s) >= 0;
    }
    if (__syncthreads_or(both)) {
        const int parts = (a.cap_src + kForkSlots - 1) / kForkSlots;
        for (int64_t x = blockIdx.x; x < (int64_t)parts * a.heads; x += gridDim.x) {
            const int h = (int)(x / parts), t0 = (int)(x % parts) * kForkSlots;
            for (int p = 0; p < a.parts; ++p) fork_held(a, a.part[p], h, t0, min(t0 + kForkSlots, a.cap_src), smem);
        }
        return;
    }
    for (int s0 = 0; s0 < a.from; s0 += kForkThreads) {
        const int s = s0 + tid;
        const bool some = s < a.from && taker[s] >= 0;
        const int n = some ? (fork_length(a, s) + kForkSlots - 1) / kForkSlots * a.heads : 0;
        int sum, count;
        const int at = block_excl_scan(n, scan, &sum), index = block_excl_scan(some, scan, &count);
        if (some) {
            taken[active + index] = s;
            place[active + index] = ranges + at;
        }
        __syncthreads();
        if (tid == 0) {
            active += count;
            ranges += sum;
        }
        __syncthreads();
    }
    for (int x = blockIdx.x; x < ranges; x += gridDim.x) {
        int lo = 0, hi = active;   // the last source whose ranges do not begin behind x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (place[mid] <= x) lo = mid;
            else hi = mid;
        }
        const int s = taken[lo], len = fork_length(a, s), parts = (len + kForkSlots - 1) / kForkSlots, r = x - place[lo];
        fork_copy(a, s, len, r / parts, r % parts * kForkSlots, taker[s], next);
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
    int widest = 0;
    auto put = [&](const void *src_at, void *dst_at, int row) {
        if (!src_at) return;
        // steps as wide as everything that starts a row of the array allows
        uint64_t bits = reinterpret_cast<uintptr_t>(src_at) | reinterpret_cast<uintptr_t>(dst_at) | 16;
        if (c.batch > 1) bits |= (uint64_t)c.ldb * row;
        if (to.batch > 1) bits |= (uint64_t)to.ldb * row;
        if (c.heads > 1) bits |= (uint64_t)c.ldh * row | (uint64_t)to.ldh * row;
        a.part[a.parts++] = ForkArray{static_cast<const char *>(src_at), static_cast<char *>(dst_at), row, (int)(bits & -bits)};
        widest = row > widest ? row : widest;
    };
    put(c.k, to.k, c.d / 2);
    put(c.v, to.v, c.d / 2);
    put(c.ks, to.ks, c.d / kQGroup * 4);
    put(c.vs, to.vs, c.d / kQGroup * 4);
    put(c.weight, to.weight, 4);
    put(c.pos, to.pos, 4);
    for (int x = 0; x < a.parts; ++x) a.begin[x + 1] = a.begin[x] + kForkSlots * a.part[x].row / a.part[x].wide;
    size_t smem = (3 * (size_t)a.from + a.to) * sizeof(int);
    if (a.in_place) {
        const size_t hold = (size_t)a.to * widest > kForkHeld ? (size_t)a.to * widest : kForkHeld;
        if (hold > 224 * 1024) {
            set_error("%s: %d sequences of d_head %d in place are too many", who, a.to, c.d);
            return CS_ERR_UNSUPPORTED;
        }
        if (hold > smem) smem = hold;
    }
    const int sms = device_sm_count();
    cudaError_t e = cudaSuccess;
    if (smem > 47 * 1024) e = allow_smem(reinterpret_cast<const void *>(&fork_kernel));
    if (e == cudaSuccess)
        e = launch(fork_kernel, dim3(4 * (sms > 0 ? sms : 1)), dim3(kForkThreads), smem, (cudaStream_t)stream, pdl_enabled(), a);
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
