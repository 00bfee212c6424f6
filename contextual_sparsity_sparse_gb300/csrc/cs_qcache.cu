// The KV cache held in 4 bits: writing rows, reading them back, choosing the
// slots to give up, and cutting a cache down.  (Attention: cs_qattn.cu.)
//
// Contextual sparsity keeps what a token needs and leaves the rest; a serving
// process does the same with its cache: the slots that gathered the least
// attention are given up, and the rows that stay are held in 4 bits.
#include <cooperative_groups.h>

#include "cs_qcache.cuh"

namespace cg = cooperative_groups;

namespace cs {

namespace {

// ---------------------------------------------------------------- append, read

struct QRowsCall {
    QCacheK c;
    QRowsK k, v;
    int n;
    const int32_t *start, *slots, *n_new, *pos;
    uint32_t *err;
    uint32_t mul, shift;     // x / n = (x mul) >> shift for x < 2^31
};

// The slot of token t of sequence b in head h, or -1; a slot out of range is flagged.
__device__ __forceinline__ int slot_of(const QRowsCall &a, int b, int h, int t) {
    const int64_t i = a.slots ? ld_dep(a.slots + ((int64_t)b * a.c.heads + h) * a.n + t)
                              : (int64_t)ld_dep(a.start + b) + t;
    if (i >= 0 && i < a.c.cap) return (int)i;
    if (i != -1) atomicOr(a.err, CS_DEVERR_INDEX);
    return -1;
}

__device__ __forceinline__ void load8(const QRowsK &r, int64_t i, float (&x)[8]) {
    if (!r.vec) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = q_load1(r, i + e);
    } else if (r.dt == CS_F32) {
        const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(r.p) + i);
        const float4 lo = p[0], hi = p[1];
        x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
        x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(r.p + 2 * i);
        if (r.dt == CS_F16) unpack16(v, x, static_cast<const __half *>(nullptr));
        else unpack16(v, x, static_cast<const __nv_bfloat16 *>(nullptr));
    }
}

__device__ __forceinline__ void store8(const QRowsK &r, int64_t i, const float (&x)[8]) {
    if (!r.vec) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q_store1(r, i + e, x[e]);
    } else if (r.dt == CS_F32) {
        float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(r.p) + i);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint4 v;
        uint32_t *w = &v.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (r.dt == CS_F16) {
                const __half2 p = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t *>(&p);
            } else {
                const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t *>(&p);
            }
        }
        *reinterpret_cast<uint4 *>(r.p + 2 * i) = v;
    }
}

// A row's part that one thread has: 8 channels, D / 8 threads to a row.  A CTA
// takes kRowSteps x 256 / (D / 8) of a sequence's rows, which are numbered with
// the token running fastest, then the head, so that codes are written (and read)
// in long runs.  All of a thread's loads are issued before it works on any.
constexpr int kRowThreads = 256, kRowSteps = 2;
template <int D>
struct RowPart {
    static constexpr int PER = D / 8, ROWS = kRowThreads / PER;
    int c8, t[kRowSteps], h[kRowSteps], slot[kRowSteps];   // slot -1: no such row, or none for it
    bool row[kRowSteps];

    // limit: how many of the n tokens the sequence has
    __device__ __forceinline__ RowPart(const QRowsCall &a, int b, int limit) {
        const int r = threadIdx.x / PER;
        c8 = threadIdx.x % PER * 8;
        const uint32_t rows = (uint32_t)a.n * a.c.heads;
#pragma unroll
        for (int i = 0; i < kRowSteps; ++i) {
            const uint32_t x = (blockIdx.x * kRowSteps + i) * (uint32_t)ROWS + r;
            h[i] = (int)((uint64_t)x * a.mul >> a.shift);
            t[i] = (int)(x - (uint32_t)h[i] * a.n);
            row[i] = r < ROWS && x < rows && t[i] < limit;
            slot[i] = row[i] ? slot_of(a, b, h[i], t[i]) : -1;
        }
    }
};

// The 8 codes of channels x whose group lies in [lo, hi], beside the group's
// scale and offset: the nearest of (x - z) / s in exact arithmetic.  An fp32
// quotient below 16 is off by less than 1e-5, so only one within 1e-4 of a half
// is divided again in 64 bits.  The group's threads go through this together.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float lo, float hi, __half &sh, __half &zh) {
    sh = __float2half_rn((hi - lo) * (1.f / 15.f));
    zh = __float2half_rn(lo);
    const float s = __half2float(sh), z = __half2float(zh);
    if (s == 0.f) return 0;
    const float inv = 1.f / s;
    // rounded scales and offsets can take the ends past 0 and 15
    const bool past = (lo - z) * inv < -0.499f || (hi - z) * inv > 15.499f;
    float n[8];
    bool half = past;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = (x[e] - z) * inv;
        n[e] = (q + 12582912.f) - 12582912.f;   // 1.5 2^23: rounds to the nearest integer, halves to even
        half |= fabsf(q - n[e]) > 0.4999f;
    }
    if (half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = (x[e] - z) * inv;
            float r = rintf(q);
            if (fabsf(fabsf(q - r) - 0.5f) < 1e-4f) r = (float)rint(((double)x[e] - (double)z) / (double)s);
            n[e] = fminf(fmaxf(r, 0.f), 15.f);
        }
    }
    const float a = fmaf(fmaf(fmaf(n[3], 16.f, n[2]), 16.f, n[1]), 16.f, n[0]);
    const float b = fmaf(fmaf(fmaf(n[7], 16.f, n[6]), 16.f, n[5]), 16.f, n[4]);
    return (uint32_t)a | (uint32_t)b << 16;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) qappend_kernel(QRowsCall a) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y;
    int limit = a.n;
    if (a.n_new) {
        limit = ld_dep(a.n_new + b);
        if (limit < 0 || limit > a.n) {
            atomicOr(a.err, CS_DEVERR_COUNT);
            limit = limit < 0 ? 0 : a.n;
        }
    }
    const RowPart<D> p(a, b, limit);
    float x[kRowSteps][2][8];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][v][e] = 0.f;
            const QRowsK &r = v ? a.v : a.k;
            if (p.slot[i] >= 0) load8(r, b * r.ldb + p.t[i] * r.ldt + p.h[i] * r.ldh + p.c8, x[i][v]);
        }
    const int first = a.pos ? ld_dep(a.pos + b) : 0;
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
        const int64_t at = p.slot[i] >= 0 ? a.c.slot0(b, p.h[i]) + p.slot[i] : 0;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            float lo = INFINITY, hi = -INFINITY;
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                odd |= !(fabsf(x[i][v][e]) <= 65504.f);
                lo = fminf(lo, x[i][v][e]);
                hi = fmaxf(hi, x[i][v][e]);
            }
            if (odd) {
                lo = INFINITY;
                hi = -INFINITY;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &y = x[i][v][e];
                    y = y != y ? 0.f : fminf(fmaxf(y, -65504.f), 65504.f);
                    lo = fminf(lo, y);
                    hi = fmaxf(hi, y);
                }
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
            }
            if (p.slot[i] < 0) continue;
            __half sh, zh;
            const uint32_t codes = quantise8(x[i][v], lo, hi, sh, zh);
            reinterpret_cast<uint32_t *>(v ? a.c.v : a.c.k)[at * (D / 8) + p.c8 / 8] = codes;
            if (p.c8 % kQGroup == 0)
                (v ? a.c.vs : a.c.ks)[at * (D / kQGroup) + p.c8 / kQGroup] =
                    (uint32_t)__half_as_ushort(sh) | (uint32_t)__half_as_ushort(zh) << 16;
        }
        if (p.slot[i] >= 0 && p.c8 == 0) {
            if (a.c.weight) a.c.weight[at] = 0.f;
            if (a.c.pos) a.c.pos[at] = first + p.t[i];
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) qread_kernel(QRowsCall a) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y;
    const RowPart<D> p(a, b, a.n);
    uint32_t codes[kRowSteps][2], sz[kRowSteps][2];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            codes[i][v] = sz[i][v] = 0;
            if (p.slot[i] < 0) continue;
            const int64_t at = a.c.slot0(b, p.h[i]) + p.slot[i];
            codes[i][v] = ld_dep(reinterpret_cast<const uint32_t *>(v ? a.c.v : a.c.k) + at * (D / 8) + p.c8 / 8);
            sz[i][v] = ld_dep((v ? a.c.vs : a.c.ks) + at * (D / kQGroup) + p.c8 / kQGroup);
        }
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (!p.row[i]) continue;
            float s, z, x[8];
            half2x(sz[i][v], s, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // nibbles e and e + 4 as fp16 1024 + n, less 1024
                const uint32_t w = (codes[i][v] >> (4 * e) & 0x000f000fu) | 0x64006400u;
                const float2 n = __half22float2(__hsub2(*reinterpret_cast<const __half2 *>(&w), __float2half2_rn(1024.f)));
                x[e] = fmaf(s, n.x, z);
                x[e + 4] = fmaf(s, n.y, z);
            }
            const QRowsK &r = v ? a.v : a.k;
            store8(r, b * r.ldb + p.t[i] * r.ldt + p.h[i] * r.ldh + p.c8, x);
        }
}

// --------------------------------------------------------------- evict, trim

struct QEvictCall {
    QCacheK c;
    const int32_t *length, *next_pos;
    int limit;               // slots that may be in use
    int n;                   // evict: tokens that need a slot
    int keep;                // trim: slots that stay; -1 for evict
    int sinks, recent;
    int32_t *out;            // evict: [batch, heads, n] slots; trim: [batch, heads, keep] slots that stay
    uint32_t *err;
};

constexpr int kLongThreads = 512;

// A total order on weights as unsigned integers: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0;
    if (u == 0x80000000u) u = 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A slot's class by its token's position: 0 empty, 1 plain, 2 protected.
struct SlotClass {
    int sinks;
    int64_t from;

    __device__ __forceinline__ SlotClass(const QEvictCall &a, int b)
        : sinks(a.sinks), from(a.recent > 0 ? (int64_t)ld_dep(a.next_pos + b) - a.recent : INT64_MAX) {}
    __device__ __forceinline__ int operator()(int p) const { return p < 0 ? 0 : p < sinks || p >= from ? 2 : 1; }
};

// Rows too long for the registers of a cluster: one CTA per (sequence, head) goes
// over the weights once per histogram.  The slots to give up are the first e of the
// order (class, weight, slot), class 0 empty, 1 plain, 2 protected: the class
// and then the weight's four bytes are found one histogram at a time, and a
// last pass in slot order writes the chosen slots (or, for a trim, the others).
__global__ void __launch_bounds__(kLongThreads) qevict_long_kernel(QEvictCall a) {
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    __shared__ int hist[256];
    __shared__ int wsum[32];
    __shared__ int pick[2];
    __shared__ int used_s;
    const int cap = a.keep >= 0 ? a.c.cap : a.limit;
    // one thread reads it: the barriers below need one answer, whatever else writes there meanwhile
    if (tid == 0) used_s = q_length(a.length, b, cap, a.err);
    __syncthreads();
    const int used = used_s;
    const int e = a.keep >= 0 ? max(0, used - a.keep) : max(0, a.n - (cap - used));
    const int64_t slot0 = a.c.slot0(b, h);
    const float *w = a.c.weight + slot0;
    const SlotClass sc(a, b);
    auto cls = [&](int i) { return a.c.pos ? sc(ld_dep(a.c.pos + slot0 + i)) : 1; };
    int want = e;            // still to take at or above the prefix found so far
    int c = -1;
    uint32_t key = 0;
    if (e > 0) {
        for (int i = tid; i < 4; i += kLongThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < used; i += kLongThreads) atomicAdd(&hist[cls(i)], 1);
        __syncthreads();
        for (c = 0; c < 2 && want > hist[c]; ++c) want -= hist[c];
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            for (int i = tid; i < 256; i += kLongThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < used; i += kLongThreads) {
                const uint32_t u = weight_key(ld_dep(w + i));
                if (cls(i) == c && (shift == 24 || u >> (shift + 8) == key >> (shift + 8)))
                    atomicAdd(&hist[u >> shift & 255u], 1);
            }
            __syncthreads();
            int total;
            const int v = tid < 256 ? hist[tid] : 0;
            const int before = block_excl_scan(v, wsum, &total);
            if (v && want > before && want <= before + v) {
                pick[0] = tid;
                pick[1] = before;
            }
            __syncthreads();
            key |= (uint32_t)pick[0] << shift;
            want -= pick[1];
        }
    }
    // `want` of the slots equal to (c, key) go, the first ones; weights that another kernel changes meanwhile
    // must not lead past the list
    const int room = a.keep >= 0 ? a.keep : a.n;
    int32_t *out = a.out + ((int64_t)b * a.c.heads + h) * room;
    int equal = 0, put = 0;
    for (int i0 = 0; i0 < used; i0 += kLongThreads) {
        const int i = i0 + tid;
        bool lower = false, same = false;
        if (e > 0 && i < used) {
            const int ci = cls(i);
            const uint32_t u = weight_key(ld_dep(w + i));
            lower = ci < c || (ci == c && u < key);
            same = ci == c && u == key;
        }
        int n;
        const int eq = equal + block_excl_scan(same, wsum, &n);
        equal += n;
        bool take = lower || (same && eq < want);
        if (a.keep >= 0) take = i < used && !take;
        const int at = put + block_excl_scan(take, wsum, &n);
        put += n;
        if (take && at < room) out[at] = i;
    }
    if (a.keep < 0)
        for (int i = e + tid; i < a.n; i += kLongThreads) out[i] = used + i - e;
}

// A cluster of C CTAs of T threads per (sequence, head), K slots to a thread, all
// in registers: a warp has 32 K consecutive slots.  The slots to give up are the
// first e of the order (class, weight, slot): three histograms find the last
// one's class and key (2 + 10, 11 and 11 bits), each CTA its own slots' counts,
// which the cluster adds up a slice per CTA; then ballots number the chosen
// slots, and the equal ones, in slot order.
constexpr int kBins = 3 * 1024;

template <int T>
struct EvictShared {
    int hist[kBins];
    int red[kBins];
    int wsum[32];
    int tot[8];          // the slices' totals
    int pick[2];         // the bin, and what comes before it
    int lower[T / 32], same[T / 32];
    int2 cta[8];         // the CTAs' chosen and equal slots
    int used;
};

// The bin of the cluster's `want`-th value (from 1) among nb bins, and how many
// lie in lower bins.
template <int T>
__device__ int2 find_bin(EvictShared<T> &sh, cg::cluster_group &cl, int nb, int want) {
    const int C = (int)cl.num_blocks(), me = (int)cl.block_rank(), tid = threadIdx.x;
    const int *counts = sh.hist;
    int slice = nb, lo = 0, before = 0, owner = 0;
    if (C > 1) {
        slice = nb / C;
        lo = me * slice;
        cl.sync();
        int sum = 0;
        for (int i = tid; i < slice; i += T) {
            int v = 0;
            for (int r = 0; r < C; ++r) v += cl.map_shared_rank(sh.hist, r)[lo + i];
            sh.red[i] = v;
            sum += v;
        }
        int total;
        block_excl_scan(sum, sh.wsum, &total);
        if (tid < C) cl.map_shared_rank(sh.tot, tid)[me] = total;
        cl.sync();
        while (owner < C - 1 && want > before + sh.tot[owner]) before += sh.tot[owner++];
        counts = sh.red;
    } else {
        __syncthreads();
    }
    if (me == owner) {
        const int each = (slice + T - 1) / T;
        const int i0 = min(slice, tid * each), i1 = min(slice, i0 + each);
        int sum = 0;
        for (int i = i0; i < i1; ++i) sum += counts[i];
        int total;
        int at = before + block_excl_scan(sum, sh.wsum, &total);
        if (want > at && want <= at + sum)
            for (int i = i0; i < i1; ++i) {
                if (want <= at + counts[i]) {
                    for (int r = 0; r < C; ++r) {
                        int *to = C > 1 ? cl.map_shared_rank(sh.pick, r) : sh.pick;
                        to[0] = lo + i;
                        to[1] = at;
                    }
                    break;
                }
                at += counts[i];
            }
    }
    if (C > 1) cl.sync();
    else __syncthreads();
    return make_int2(sh.pick[0], sh.pick[1]);
}

template <int T, int K>
__global__ void __launch_bounds__(T) qevict_kernel(QEvictCall a) {
    __shared__ EvictShared<T> sh;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
    const int row = blockIdx.x / C, h = row % a.c.heads, b = row / a.c.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kBins; i += T) sh.hist[i] = 0;
    if (C > 1) cl.sync();   // the others' shared memory is there
    pdl_wait();
    pdl_launch_dependents();
    const int cap = a.keep >= 0 ? a.c.cap : a.limit;
    // one thread reads it for the cluster: the barriers below need one answer, whatever else writes there meanwhile
    if (me == 0 && tid == 0) {
        const int n = q_length(a.length, b, cap, a.err);
        for (int r = 0; r < C; ++r) *cl.map_shared_rank(&sh.used, r) = n;
    }
    const int64_t slot0 = a.c.slot0(b, h);
    const SlotClass sc(a, b);
    // slots past the length are loaded, too (they are the cache's), while it is on its way
    const int first = (me * (T / 32) + warp) * 32 * K + lane;
    uint32_t key[K], cls = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int slot = first + 32 * i;
        key[i] = slot < cap ? __float_as_uint(ld_dep(a.c.weight + slot0 + slot)) : 0;
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int slot = first + 32 * i;
        const int c = a.c.pos ? sc(slot < cap ? ld_dep(a.c.pos + slot0 + slot) : 0) : 1;
        cls |= (uint32_t)c << (2 * i);
    }
    if (C > 1) cl.sync();
    else __syncthreads();
    const int used = sh.used;
    const int e = a.keep >= 0 ? max(0, used - a.keep) : max(0, a.n - (cap - used));
#pragma unroll
    for (int i = 0; i < K; ++i) {
        key[i] = weight_key(__uint_as_float(key[i]));
        if (first + 32 * i >= used) cls |= 3u << (2 * i);
    }
    int want = e;
    uint32_t pc = 0, pk = 0;   // the last one's class and key
    if (e > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const uint32_t c = cls >> (2 * i) & 3u;
            if (c < 3) atomicAdd(&sh.hist[c * 1024 + (key[i] >> 22)], 1);
        }
        int2 p = find_bin<T>(sh, cl, kBins, want);
        pc = (uint32_t)p.x >> 10;
        pk = (uint32_t)(p.x & 1023) << 22;
        want -= p.y;
#pragma unroll 1
        for (int shift = 11; shift >= 0; shift -= 11) {
            for (int i = tid; i < 2048; i += T) sh.hist[i] = 0;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < K; ++i)
                if ((cls >> (2 * i) & 3u) == pc && (key[i] ^ pk) >> (shift + 11) == 0) atomicAdd(&sh.hist[key[i] >> shift & 2047u], 1);
            p = find_bin<T>(sh, cl, 2048, want);
            pk |= (uint32_t)p.x << shift;
            want -= p.y;
        }
    }
    // `want` of the slots equal to (pc, pk) go, the first ones
    uint32_t lower = 0, same = 0;
    int nl = 0, ns = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const uint32_t c = cls >> (2 * i) & 3u;
        const bool in = e > 0 && c < 3;
        const bool lo = in && (c < pc || (c == pc && key[i] < pk)), eq = in && c == pc && key[i] == pk;
        lower |= (uint32_t)lo << i;
        same |= (uint32_t)eq << i;
        nl += __popc(__ballot_sync(kFull, lo));
        ns += __popc(__ballot_sync(kFull, eq));
    }
    if (lane == 0) {
        sh.lower[warp] = nl;
        sh.same[warp] = ns;
    }
    __syncthreads();
    int bl = 0, bs = 0, tl = 0, ts = 0;
    for (int w = 0; w < T / 32; ++w) {
        if (w < warp) {
            bl += sh.lower[w];
            bs += sh.same[w];
        }
        tl += sh.lower[w];
        ts += sh.same[w];
    }
    if (C > 1) {
        if (tid < C) cl.map_shared_rank(sh.cta, tid)[me] = make_int2(tl, ts);
        cl.sync();
        for (int r = 0; r < me; ++r) {
            bl += sh.cta[r].x;
            bs += sh.cta[r].y;
        }
    }
    // weights that another kernel changes meanwhile must not lead past the list
    const int room = a.keep >= 0 ? a.keep : a.n;
    int32_t *out = a.out + ((int64_t)b * a.c.heads + h) * room;
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int slot = first + 32 * i;
        const uint32_t wl = __ballot_sync(kFull, lower >> i & 1u), we = __ballot_sync(kFull, same >> i & 1u);
        const int eqs = bs + __popc(we & below);
        const bool gone = (lower >> i & 1u) || ((same >> i & 1u) && eqs < want);
        const int at = bl + __popc(wl & below) + min(eqs, want);   // slots before this one that go
        bl += __popc(wl);
        bs += __popc(we);
        if (a.keep >= 0) {
            if (slot < used && !gone && slot - at < room) out[slot - at] = slot;
        } else if (gone && at < room) {
            out[at] = slot;
        }
    }
    if (a.keep < 0 && me == 0)
        for (int i = e + tid; i < a.n; i += T) out[i] = used + i - e;
}

// Copies the slots that stay.  A CTA takes kTrimSlots of a head's: their codes in
// 16-byte pieces, then their scales, weights and positions word by word.
constexpr int kTrimSlots = 64;
template <int D>
__global__ void __launch_bounds__(256) qtrim_kernel(QEvictCall a, QCacheK dst) {
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.y, b = blockIdx.z, t0 = blockIdx.x * kTrimSlots;
    __shared__ int slots[kTrimSlots];
    const int n = min(kTrimSlots, min(a.keep, q_length(a.length, b, a.c.cap, nullptr)) - t0);
    if (threadIdx.x < kTrimSlots) {
        int s = -1;
        if ((int)threadIdx.x < n) s = ld_dep(a.out + ((int64_t)b * a.c.heads + h) * a.keep + t0 + threadIdx.x);
        slots[threadIdx.x] = s < a.c.cap ? s : -1;
    }
    __syncthreads();
    const int64_t from = a.c.slot0(b, h), to = dst.slot0(b, h) + t0;
    constexpr int CH = D / 32, STEPS = kTrimSlots * CH / 256 > 0 ? (kTrimSlots * CH + 255) / 256 : 1;
    uint4 v[2][STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int x = i * 256 + threadIdx.x, t = x / CH, ch = x % CH;
        const int s = t < kTrimSlots ? slots[t] : -1;
        if (s < 0) continue;
        v[0][i] = ld_dep(reinterpret_cast<const uint4 *>(a.c.k) + (from + s) * CH + ch);
        v[1][i] = ld_dep(reinterpret_cast<const uint4 *>(a.c.v) + (from + s) * CH + ch);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int x = i * 256 + threadIdx.x, t = x / CH, ch = x % CH;
        if (t >= kTrimSlots || slots[t] < 0) continue;
        reinterpret_cast<uint4 *>(dst.k)[(to + t) * CH + ch] = v[0][i];
        reinterpret_cast<uint4 *>(dst.v)[(to + t) * CH + ch] = v[1][i];
    }
    constexpr int G = D / kQGroup;
    for (int x = threadIdx.x; x < kTrimSlots * G; x += 256) {
        const int t = x / G, g = x % G, s = slots[t];
        if (s < 0) continue;
        const uint32_t ks = ld_dep(a.c.ks + (from + s) * G + g), vs = ld_dep(a.c.vs + (from + s) * G + g);
        dst.ks[(to + t) * G + g] = ks;
        dst.vs[(to + t) * G + g] = vs;
    }
    if (threadIdx.x < kTrimSlots && slots[threadIdx.x] >= 0) {
        const int s = slots[threadIdx.x];
        const float w = ld_dep(a.c.weight + from + s);
        const int p = a.c.pos ? ld_dep(a.c.pos + from + s) : 0;
        dst.weight[to + threadIdx.x] = w;
        if (a.c.pos) dst.pos[to + threadIdx.x] = p;
    }
}

// Launches the choice of slots for rows of up to `cap` slots.
template <int T, int K>
cudaError_t launch_evict(const QEvictCall &a, int ctas, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.c.heads * a.c.batch * ctas));
    cfg.blockDim = dim3(T);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, qevict_kernel<T, K>, a);
}

cudaError_t choose_slots(const QEvictCall &a, cudaStream_t s) {
    const int cap = a.keep >= 0 ? a.c.cap : a.limit, sms = device_sm_count();
    const int64_t rows = (int64_t)a.c.heads * a.c.batch;
    // few rows: several CTAs each, as long as the GPU has room and a CTA has at least 2048 slots
    int ctas = 1;
    while (ctas < 8 && ((rows * ctas * 2 <= 2 * sms && cap / (2 * ctas) >= 2048) || cap > 16384 * ctas)) ctas *= 2;
    const int each = (cap + ctas - 1) / ctas;
    if (each <= 2048) return launch_evict<512, 4>(a, ctas, s);
    if (each <= 8192) return launch_evict<512, 16>(a, ctas, s);
    if (each <= 16384) return launch_evict<1024, 16>(a, ctas, s);
    return launch(qevict_long_kernel, dim3(a.c.heads, a.c.batch), dim3(kLongThreads), 0, s, pdl_enabled(), a);
}

// ------------------------------------------------------------------- host side

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#define CS_CHECK(cond, ...)                       \
    do {                                          \
        if (!(cond)) {                            \
            set_error(__VA_ARGS__);               \
            return CS_ERR_INVALID;                \
        }                                         \
    } while (0)

constexpr int kMaxHeads = 1024, kMaxCapacity = 1 << 24, kMaxTokens = 1 << 24;

// codes: whether the call reads or writes k, v and their scales.
cs_status check_cache(const cs_qcache *q, bool codes, const char *who, QCacheK *out) {
    CS_CHECK(q, "%s: cache is null", who);
    CS_CHECK(q->batch >= 1 && q->n_heads >= 1 && q->capacity >= 1, "%s: batch, n_heads and capacity must be >= 1 (%d, %d, %d)",
             who, q->batch, q->n_heads, q->capacity);
    if (q->batch > kQMaxBatch || q->n_heads > kMaxHeads || q->capacity > kMaxCapacity) {
        set_error("%s: batch %d, n_heads %d or capacity %d above %d, %d and %d", who, q->batch, q->n_heads, q->capacity,
                  kQMaxBatch, kMaxHeads, kMaxCapacity);
        return CS_ERR_UNSUPPORTED;
    }
    const int64_t ldh = q->ld_head ? q->ld_head : q->capacity;
    const int64_t ldb = q->ld_batch ? q->ld_batch : ldh * q->n_heads;
    CS_CHECK((q->n_heads == 1 || ldh >= q->capacity) && (q->batch == 1 || ldb >= q->capacity),
             "%s: ld_batch %lld and ld_head %lld must be at least the capacity %d", who, (long long)ldb, (long long)ldh,
             q->capacity);
    CS_CHECK(ldh < (int64_t(1) << 40) && ldb < (int64_t(1) << 40), "%s: ld_batch or ld_head too large", who);
    if (codes) {
        if (q->d_head < kQGroup || q->d_head > 256 || q->d_head % kQGroup) {
            set_error("%s: d_head=%d is not 64, 128, 192 or 256", who, q->d_head);
            return CS_ERR_UNSUPPORTED;
        }
        CS_CHECK(q->k && q->v && q->k_scale && q->v_scale, "%s: the cache's k, v, k_scale and v_scale are required", who);
        const int groups = q->d_head / kQGroup, piece = 4 * (groups & -groups);   // a slot's scales are copied in such pieces
        CS_CHECK(aligned(q->k, 16) && aligned(q->v, 16) && aligned(q->k_scale, piece) && aligned(q->v_scale, piece),
                 "%s: k and v must be 16-byte aligned, their scales %d-byte", who, piece);
    }
    CS_CHECK(aligned(q->weight, 4) && aligned(q->pos, 4), "%s: weight and pos must be 4-byte aligned", who);
    *out = QCacheK{q->k, q->v, static_cast<uint32_t *>(q->k_scale), static_cast<uint32_t *>(q->v_scale), q->weight, q->pos,
                   q->batch, q->n_heads, q->capacity, q->d_head, ldb, ldh};
    return CS_OK;
}

cs_status check_rows(const cs_head_rows *r, const char *name, const char *who, QRowsK *out) {
    CS_CHECK(r && r->data, "%s: %s is null", who, name);
    CS_CHECK(r->dtype == CS_F32 || r->dtype == CS_F16 || r->dtype == CS_BF16, "%s: %s has a bad dtype %d", who, name, (int)r->dtype);
    const int es = (int)dtype_size(r->dtype);
    CS_CHECK(aligned(r->data, es), "%s: %s must be aligned to its elements", who, name);
    const int64_t most = int64_t(1) << 46;
    CS_CHECK(r->ld_batch >= 0 && r->ld_token >= 0 && r->ld_head >= 0 && r->ld_batch < most && r->ld_token < most && r->ld_head < most,
             "%s: %s has a bad stride", who, name);
    *out = QRowsK{static_cast<char *>(r->data), r->ld_batch, r->ld_token, r->ld_head, (int)r->dtype,
                  aligned(r->data, 16) && (r->ld_batch * es) % 16 == 0 && (r->ld_token * es) % 16 == 0 && (r->ld_head * es) % 16 == 0};
    return CS_OK;
}

cs_status check_qws(void *ws, size_t ws_bytes, size_t need, const char *who) {
    if (!ws || !aligned(ws, 256)) {
        set_error("%s: workspace is null or not 256-byte aligned", who);
        return CS_ERR_WORKSPACE;
    }
    if (ws_bytes < need) {
        set_error("%s: workspace too small: %zu bytes given, %zu needed", who, ws_bytes, need);
        return CS_ERR_WORKSPACE;
    }
    return CS_OK;
}

cs_status check_evict(const cs_qcache *q, const int32_t *length, const int32_t *next_pos, int sinks, int recent,
                      const char *who) {
    CS_CHECK(q->weight, "%s: the cache has no weights", who);
    CS_CHECK(length && aligned(length, 4), "%s: length is null or misaligned", who);
    CS_CHECK(sinks >= 0 && recent >= 0, "%s: sinks and recent must be >= 0 (%d, %d)", who, sinks, recent);
    CS_CHECK((sinks == 0 && recent == 0) || q->pos, "%s: sinks and recent need a cache with positions", who);
    CS_CHECK(recent == 0 || (next_pos && aligned(next_pos, 4)), "%s: recent needs next_pos", who);
    return CS_OK;
}

size_t trim_scratch(int batch, int heads, int keep) { return align256((size_t)batch * heads * keep * sizeof(int32_t)); }

// Launches append's or read's kernel of the cache's d_head.
template <typename F>
cudaError_t by_d(int d, F f) {
    switch (d) {
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    case 192: return f(std::integral_constant<int, 192>());
    default: return f(std::integral_constant<int, 256>());
    }
}
template <int D>
dim3 rows_grid(const QRowsCall &a) {
    const int64_t rows = (int64_t)a.n * a.c.heads, each = RowPart<D>::ROWS * kRowSteps;
    return dim3((unsigned)((rows + each - 1) / each), a.c.batch);
}

cs_status rows_call(const cs_qcache *cache, const cs_head_rows *k, const cs_head_rows *v, int n, const int32_t *start,
                    const int32_t *slots, void *ws, size_t ws_bytes, const char *who, QRowsCall *a) {
    cs_status st = check_cache(cache, true, who, &a->c);
    if (st == CS_OK) st = check_rows(k, "k", who, &a->k);
    if (st == CS_OK) st = check_rows(v, "v", who, &a->v);
    if (st != CS_OK) return st;
    CS_CHECK(k->dtype == v->dtype, "%s: k and v differ in dtype", who);
    CS_CHECK(n >= 0 && n <= kMaxTokens, "%s: n=%d outside [0, %d]", who, n, kMaxTokens);
    CS_CHECK((start != nullptr) != (slots != nullptr), "%s: exactly one of start and slots is required", who);
    CS_CHECK(aligned(start, 4) && aligned(slots, 4), "%s: start and slots must be 4-byte aligned", who);
    if ((int64_t)n * cache->n_heads >= (int64_t(1) << 31) - 4096) {
        set_error("%s: n x n_heads = %lld is too large", who, (long long)n * cache->n_heads);
        return CS_ERR_UNSUPPORTED;
    }
    // with 2^s >= n, 2^(31 + s) / n rounded up is off by at most 1, which x < 2^31 times 2^-(31 + s) keeps below 1 / n
    a->shift = 31;
    while ((int64_t(1) << (a->shift - 31)) < n) ++a->shift;
    a->mul = n > 0 ? (uint32_t)((uint64_t(1) << a->shift) / n + (n > 1)) : 0;
    a->n = n;
    a->start = start;
    a->slots = slots;
    a->n_new = a->pos = nullptr;
    a->err = static_cast<uint32_t *>(ws);
    return check_qws(ws, ws_bytes, kControlBytes, who);
}

}  // namespace

}  // namespace cs

using namespace cs;

extern "C" {

size_t cs_qcache_workspace_size(int batch, int kv_heads, int capacity, int d_head, int n_heads, int n_q) {
    if (batch < 1 || batch > kQMaxBatch || kv_heads < 1 || kv_heads > kMaxHeads || capacity < 1 || capacity > kMaxCapacity ||
        d_head < kQGroup || d_head > 256 || d_head % kQGroup || n_heads < kv_heads || n_heads % kv_heads || n_q < 1 ||
        (int64_t)n_heads / kv_heads * n_q > kQMaxRows)
        return 0;
    const size_t attn = qattn_scratch(batch, kv_heads, capacity, d_head, n_heads, n_q, device_sm_count());
    const size_t trim = trim_scratch(batch, kv_heads, capacity);
    return kControlBytes + (attn > trim ? attn : trim);
}

cs_status cs_qcache_append(const cs_qcache *cache, const cs_head_rows *k, const cs_head_rows *v, int n,
                           const int32_t *start, const int32_t *slots, const int32_t *n_new, const int32_t *pos,
                           void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_qcache_append";
    QRowsCall a;
    const cs_status st = rows_call(cache, k, v, n, start, slots, ws, ws_bytes, who, &a);
    if (st != CS_OK) return st;
    CS_CHECK((pos != nullptr) == (cache->pos != nullptr), "%s: pos is required if and only if the cache has positions", who);
    CS_CHECK(aligned(pos, 4) && aligned(n_new, 4), "%s: pos and n_new must be 4-byte aligned", who);
    a.n_new = n_new;
    a.pos = pos;
    if (n == 0) return CS_OK;
    const cudaError_t e = by_d(a.c.d, [&](auto d) {
        return launch(qappend_kernel<d()>, rows_grid<d()>(a), dim3(kRowThreads), 0, (cudaStream_t)stream, pdl_enabled(), a);
    });
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

cs_status cs_qcache_read(const cs_qcache *cache, const cs_head_rows *k, const cs_head_rows *v, int n,
                         const int32_t *start, const int32_t *slots, void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_qcache_read";
    QRowsCall a;
    const cs_status st = rows_call(cache, k, v, n, start, slots, ws, ws_bytes, who, &a);
    if (st != CS_OK) return st;
    if (n == 0) return CS_OK;
    const cudaError_t e = by_d(a.c.d, [&](auto d) {
        return launch(qread_kernel<d()>, rows_grid<d()>(a), dim3(kRowThreads), 0, (cudaStream_t)stream, pdl_enabled(), a);
    });
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

cs_status cs_qcache_attention(const cs_qcache *cache, const cs_head_rows *q, int n_heads, int n_q,
                              const int32_t *length, const int32_t *q_pos, const uint32_t *mask, float scale,
                              float decay, float *weight, const cs_head_rows *out, void *ws, size_t ws_bytes,
                              cs_stream_t stream) {
    const char *who = "cs_qcache_attention";
    QAttnArgs a;
    cs_status st = check_cache(cache, true, who, &a.c);
    if (st == CS_OK) st = check_rows(q, "q", who, &a.q);
    if (st == CS_OK) st = check_rows(out, "out", who, &a.out);
    if (st != CS_OK) return st;
    CS_CHECK(q->dtype == out->dtype, "%s: q and out differ in dtype", who);
    CS_CHECK(q->data != out->data, "%s: out must not be q", who);
    CS_CHECK(n_heads >= 1 && n_heads % cache->n_heads == 0, "%s: n_heads=%d is not a multiple of the cache's %d", who, n_heads,
             cache->n_heads);
    CS_CHECK(n_q >= 0, "%s: n_q=%d is negative", who, n_q);
    if ((int64_t)n_heads / cache->n_heads * n_q > kQMaxRows) {
        set_error("%s: %d query rows per cache head, above %d", who, n_heads / cache->n_heads * n_q, kQMaxRows);
        return CS_ERR_UNSUPPORTED;
    }
    if ((int64_t)cache->batch * cache->n_heads * ((cache->capacity + 15) / 16 + 16) >= INT32_MAX) {
        set_error("%s: batch x n_heads x capacity is too large", who);
        return CS_ERR_UNSUPPORTED;
    }
    CS_CHECK(length && aligned(length, 4), "%s: length is null or misaligned", who);
    CS_CHECK(!q_pos || cache->pos, "%s: q_pos needs a cache with positions", who);
    CS_CHECK(aligned(q_pos, 4) && aligned(mask, 4) && aligned(weight, 4), "%s: q_pos, mask and weight must be 4-byte aligned", who);
    CS_CHECK(scale == scale && scale - scale == 0.f && decay - decay == 0.f, "%s: scale and decay must be finite", who);
    CS_CHECK(!weight || decay == 0.f || cache->weight, "%s: decay != 0 needs a cache with weights", who);
    a.heads = n_heads;
    a.n_q = n_q;
    a.length = length;
    a.q_pos = q_pos;
    a.mask = mask;
    a.scale = scale != 0.f ? scale : 1.f / sqrtf((float)cache->d_head);
    a.decay = decay;
    a.weight = weight;
    a.sms = device_sm_count();
    st = check_qws(ws, ws_bytes,
                   kControlBytes + qattn_scratch(a.c.batch, a.c.heads, a.c.cap, a.c.d, n_heads, n_q, a.sms), who);
    if (st != CS_OK) return st;
    a.err = static_cast<uint32_t *>(ws);
    a.scratch = static_cast<char *>(ws) + kControlBytes;
    if (n_q == 0) return CS_OK;
    const cudaError_t e = launch_qattn(a, (cudaStream_t)stream);
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

cs_status cs_qcache_evict(const cs_qcache *cache, const int32_t *length, int limit, int n, const int32_t *next_pos,
                          int sinks, int recent, int32_t *slots, void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_qcache_evict";
    QEvictCall a;
    cs_status st = check_cache(cache, false, who, &a.c);
    if (st == CS_OK) st = check_evict(cache, length, next_pos, sinks, recent, who);
    if (st != CS_OK) return st;
    CS_CHECK(n >= 1 && n <= limit && limit <= cache->capacity, "%s: needs 1 <= n <= limit <= capacity (%d, %d, %d)", who, n, limit,
             cache->capacity);
    CS_CHECK(slots && aligned(slots, 4), "%s: slots is null or misaligned", who);
    st = check_qws(ws, ws_bytes, kControlBytes, who);
    if (st != CS_OK) return st;
    a.length = length;
    a.next_pos = next_pos;
    a.limit = limit;
    a.n = n;
    a.keep = -1;
    a.sinks = sinks;
    a.recent = recent;
    a.out = slots;
    a.err = static_cast<uint32_t *>(ws);
    const cudaError_t e = choose_slots(a, (cudaStream_t)stream);
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

cs_status cs_qcache_trim(const cs_qcache *src, const int32_t *length, int keep, const int32_t *next_pos, int sinks,
                         int recent, const cs_qcache *dst, void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_qcache_trim";
    QEvictCall a;
    QCacheK to;
    cs_status st = check_cache(src, true, who, &a.c);
    if (st == CS_OK) st = check_evict(src, length, next_pos, sinks, recent, who);
    if (st == CS_OK) st = check_cache(dst, true, who, &to);
    if (st != CS_OK) return st;
    CS_CHECK(dst->batch == src->batch && dst->n_heads == src->n_heads && dst->d_head == src->d_head,
             "%s: dst and src differ in batch, n_heads or d_head", who);
    CS_CHECK(keep >= 1 && keep <= dst->capacity, "%s: keep=%d outside [1, dst's capacity %d]", who, keep, dst->capacity);
    CS_CHECK(dst->weight && (dst->pos != nullptr) == (src->pos != nullptr),
             "%s: dst needs weights, and positions if and only if src has them", who);
    CS_CHECK(dst->k != src->k && dst->v != src->v && dst->k_scale != src->k_scale && dst->v_scale != src->v_scale &&
                 dst->weight != src->weight && (!dst->pos || dst->pos != src->pos),
             "%s: dst must not share memory with src", who);
    // no more than the source's slots can stay
    a.keep = keep < src->capacity ? keep : src->capacity;
    st = check_qws(ws, ws_bytes, kControlBytes + trim_scratch(a.c.batch, a.c.heads, a.keep), who);
    if (st != CS_OK) return st;
    a.length = length;
    a.next_pos = next_pos;
    a.limit = a.n = 0;
    a.sinks = sinks;
    a.recent = recent;
    a.out = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + kControlBytes);
    a.err = static_cast<uint32_t *>(ws);
    cudaError_t e = choose_slots(a, (cudaStream_t)stream);
    if (e == cudaSuccess)
        e = by_d(a.c.d, [&](auto d) {
            return launch(qtrim_kernel<d()>, dim3((a.keep + kTrimSlots - 1) / kTrimSlots, a.c.heads, a.c.batch), dim3(256), 0,
                          (cudaStream_t)stream, pdl_enabled(), a, to);
        });
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
