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

// 8 elements of a row as they lie in memory.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];

    __device__ __forceinline__ void load(const QRowsK &r, int64_t i) {
        const T *p = reinterpret_cast<const T *>(r.p) + i;
        if (r.vec) {
#pragma unroll
            for (int e = 0; e < (int)sizeof(T) / 2; ++e) v[e] = ld_dep(reinterpret_cast<const uint4 *>(p) + e);
        } else {
            T x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = ld_dep(p + e);
            memcpy(v, x, sizeof x);
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        constexpr int N = Vec<T>::N;
#pragma unroll
        for (int e = 0; e < 8 / N; ++e) {
            float y[N];
            unpack<T>(v[e], y);
#pragma unroll
            for (int i = 0; i < N; ++i) x[e * N + i] = y[i];
        }
    }
};

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

// The part of a sequence's rows that one thread has: N channels of a key row and
// of its value row, D / N threads to a row.  Rows are numbered with the token
// running fastest, then the head, so that codes are written (and read) in long runs.
constexpr int kRowThreads = 256, kPart = 16;
template <int D, int N>
struct RowPart {
    static constexpr int PER = D / N, ROWS = kRowThreads / PER;   // rows of a CTA
    int c, t, h;   // first channel
    bool row;      // there is such a row

    // limit: how many of the n tokens the sequence has; step: rows of how many CTAs come before
    __device__ __forceinline__ RowPart(const QRowsCall &a, int limit, uint32_t step) {
        const int r = threadIdx.x / PER;
        c = threadIdx.x % PER * N;
        const uint32_t x = step * (uint32_t)ROWS + r;
        h = (int)((uint64_t)x * a.mul >> a.shift);
        t = (int)(x - (uint32_t)h * a.n);
        row = r < ROWS && x < (uint32_t)a.n * a.c.heads && t < limit;
    }
};

__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The least and the largest of N values; NaN if one of them is.
template <int N>
__device__ __forceinline__ void bounds(const float (&x)[N], float &lo, float &hi) {
    lo = hi = x[0];
#pragma unroll
    for (int e = 1; e < N; e += 2) {
        lo = min_nan(lo, x[e], x[e + 1 < N ? e + 1 : e]);
        hi = max_nan(hi, x[e], x[e + 1 < N ? e + 1 : e]);
    }
}

// The codes of channels x whose group lies in [lo, hi], beside the group's scale
// and offset: the nearest of (x - z) / s in exact arithmetic.  An fp32 quotient
// below 16 is off by three roundings, 3 x 2^-24 x 16 < 3e-6; one within 8e-6 of a
// half m + 1/2 is decided by the sign of x - z - (m + 1/2) s.  There x - z is
// taken as an unevaluated sum of two fp32 numbers, (m + 1/2) s has 17 bits, and
// the difference of the two near numbers is exact.  (In 64 bits these divisions
// took a quarter of the kernel's time: bf16 rows often hit a half exactly.)
__device__ __forceinline__ uint2 quantise(const float (&x)[kPart], float lo, float hi, __half &sh, __half &zh) {
    sh = __float2half_rn((hi - lo) * (1.f / 15.f));
    zh = __float2half_rn(lo);
    const float s = __half2float(sh), z = __half2float(zh);
    if (s == 0.f) return make_uint2(0, 0);
    const float inv = 1.f / s;
    float n[kPart], far = 0.f;
#pragma unroll
    for (int e = 0; e < kPart; e += 2) {
        float d[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float q = (x[e + i] - z) * inv;
            n[e + i] = (q + 12582912.f) - 12582912.f;   // 1.5 2^23: rounds to the nearest integer, halves to even
            d[i] = fabsf(q - n[e + i]);
        }
        far = max_nan(far, d[0], d[1]);
    }
    // rounded scales and offsets can take the ends past 0 and 15, too
    if (far > 0.499992f || (lo - z) * inv < -0.499f || (hi - z) * inv > 15.499f) {
#pragma unroll
        for (int e = 0; e < kPart; ++e) {
            const float q = (x[e] - z) * inv;
            float r = rintf(q);
            if (fabsf(fabsf(q - r) - 0.5f) < 1e-5f) {
                const float m = floorf(q), d = x[e] - z, xx = d + z;
                const float rest = (x[e] - xx) + ((xx - d) - z);   // what d lacks of x - z
                const float over = fmaf(-(m + 0.5f), s, d) + rest;
                r = over > 0.f ? m + 1.f : over < 0.f ? m : 2.f * rintf(0.5f * m + 0.25f);
            }
            n[e] = fminf(fmaxf(r, 0.f), 15.f);
        }
    }
    // four codes are added up exactly in fp32
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)fmaf(fmaf(fmaf(n[4 * e + 3], 16.f, n[4 * e + 2]), 16.f, n[4 * e + 1]), 16.f, n[4 * e]);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// 7,999 tokens of 8 heads of 128, bf16: 21 us alone, issuing in 57% of its cycles, with DRAM at 23% of a copy's rate, so
// bound by neither: a thread loads its rows, waits, quantises and stores once (fp32 20.9 us, fp16 20.4).  With the
// read-back, in a graph: three CTAs per SM 25.5 us, two 28.8, four (64 registers) 26.5, five 35.7.
template <int D, typename T>
__global__ void __launch_bounds__(kRowThreads, 3) qappend_kernel(QRowsCall a) {
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
    // the rows' loads do not wait for their slots
    const RowPart<D, kPart> p(a, limit, blockIdx.x);
    Raw8<T> raw[2][2] = {};
    if (p.row) {
        const int64_t ki = b * a.k.ldb + p.t * a.k.ldt + p.h * a.k.ldh + p.c, vi = b * a.v.ldb + p.t * a.v.ldt + p.h * a.v.ldh + p.c;
        raw[0][0].load(a.k, ki);
        raw[0][1].load(a.k, ki + 8);
        raw[1][0].load(a.v, vi);
        raw[1][1].load(a.v, vi + 8);
    }
    const int first = a.pos ? ld_dep(a.pos + b) : 0;
    const int slot = p.row ? slot_of(a, b, p.h, p.t) : -1;
    const int64_t at = slot >= 0 ? a.c.slot0(b, p.h) + slot : 0;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float x[kPart], lo, hi;
        raw[v][0].get(*reinterpret_cast<float(*)[8]>(x));
        raw[v][1].get(*reinterpret_cast<float(*)[8]>(x + 8));
        bounds(x, lo, hi);
        if (!(fmaxf(fabsf(lo), fabsf(hi)) <= 65504.f) || lo != lo) {
#pragma unroll
            for (int e = 0; e < kPart; ++e) x[e] = x[e] != x[e] ? 0.f : fminf(fmaxf(x[e], -65504.f), 65504.f);
            bounds(x, lo, hi);
        }
#pragma unroll
        for (int o = 1; o < kQGroup / kPart; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
        }
        if (slot < 0) continue;
        __half sh, zh;
        const uint2 codes = quantise(x, lo, hi, sh, zh);
        reinterpret_cast<uint2 *>(v ? a.c.v : a.c.k)[at * (D / kPart) + p.c / kPart] = codes;
        if (p.c % kQGroup == 0)
            (v ? a.c.vs : a.c.ks)[at * (D / kQGroup) + p.c / kQGroup] =
                (uint32_t)__half_as_ushort(sh) | (uint32_t)__half_as_ushort(zh) << 16;
    }
    if (slot >= 0 && p.c == 0) {
        if (a.c.weight) a.c.weight[at] = 0.f;
        if (a.c.pos) a.c.pos[at] = first + p.t;
    }
}

// 8 channels to a thread here, of two rows: 16-byte stores side by side (with 16
// channels a warp's stores leave gaps, and 8,192 rows of 128 took 12.5 instead of 11.5 us).
constexpr int kReadSteps = 2;
template <int D>
__global__ void __launch_bounds__(kRowThreads) qread_kernel(QRowsCall a) {
    pdl_wait();
    pdl_launch_dependents();
    using Part = RowPart<D, 8>;
    const int b = blockIdx.y;
    const Part p[kReadSteps] = {Part(a, a.n, blockIdx.x * kReadSteps), Part(a, a.n, blockIdx.x * kReadSteps + 1)};
    uint32_t codes[kReadSteps][2], sz[kReadSteps][2];
#pragma unroll
    for (int i = 0; i < kReadSteps; ++i) {
        const int slot = p[i].row ? slot_of(a, b, p[i].h, p[i].t) : -1;
        const int64_t at = a.c.slot0(b, p[i].h) + slot;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            codes[i][v] = slot >= 0 ? ld_dep(reinterpret_cast<const uint32_t *>(v ? a.c.v : a.c.k) + at * (D / 8) + p[i].c / 8) : 0;
            sz[i][v] = slot >= 0 ? ld_dep((v ? a.c.vs : a.c.ks) + at * (D / kQGroup) + p[i].c / kQGroup) : 0;
        }
    }
#pragma unroll
    for (int i = 0; i < kReadSteps; ++i) {
        if (!p[i].row) continue;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const QRowsK &r = v ? a.v : a.k;
            float s, z, x[8];
            half2x(sz[i][v], s, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // nibbles e and e + 4 as fp16 1024 + n, less 1024 (Kim et al., "Who Says Elephants Can't Run", 2022)
                const uint32_t w = (codes[i][v] >> (4 * e) & 0x000f000fu) | 0x64006400u;
                const float2 n = __half22float2(__hsub2(*reinterpret_cast<const __half2 *>(&w), __float2half2_rn(1024.f)));
                x[e] = fmaf(s, n.x, z);
                x[e + 4] = fmaf(s, n.y, z);
            }
            store8(r, b * r.ldb + p[i].t * r.ldt + p[i].h * r.ldh + p[i].c, x);
        }
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
// first e of the order (class, weight, slot).  One reduction gives the classes'
// sizes and the keys' range, which a histogram of 2048 bins cuts up (weights
// spread over many powers of two, so bins by leading bits would be few and
// crowded); each CTA counts its own slots and the cluster adds a slice of the
// bins per CTA.  The bin of the last slot to go holds few keys: they are gathered
// and ranked against one another, or, if they are many (equal weights), cut up
// again.  Then ballots number the chosen slots, and the equal ones, in slot order.
constexpr int kBins = 2048, kRank = 256;

template <int T>
struct EvictShared {
    int hist[kBins];
    int red[kBins];
    int wsum[32];
    uint32_t stat[T / 32][4];
    uint32_t cstat[8][4];    // the CTAs'
    int tot[8];              // the slices' totals
    int pick[3];             // the bin, what comes before it, and its own count
    uint32_t list[kRank];    // the first CTA's: keys to rank
    int listed;
    uint32_t last;           // the last key to go, and how many equal to it go
    int ties;
    int lower[T / 32], same[T / 32];
    int2 cta[8];             // the CTAs' chosen and equal slots
    int used;
};

// The bin of the cluster's `want`-th value (from 1), how many lie in lower bins, and in it.
template <int T>
__device__ int3 find_bin(EvictShared<T> &sh, cg::cluster_group &cl, int want) {
    const int C = (int)cl.num_blocks(), me = (int)cl.block_rank(), tid = threadIdx.x;
    int *counts = sh.hist;
    const int slice = kBins / C;
    int lo = 0, before = 0, owner = 0;
    if (C > 1) {
        lo = me * slice;
        cl.sync();
        int sum = 0;
        for (int i = tid; i < slice; i += T) {
            int v = 0;
#pragma unroll 8
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
                        to[2] = counts[i];
                    }
                    break;
                }
                at += counts[i];
            }
    }
    if (C > 1) cl.sync();
    else __syncthreads();
    return make_int3(sh.pick[0], sh.pick[1], sh.pick[2]);
}

// Over the cluster: the sums of a and b, the least lo, the largest hi.
template <int T>
__device__ uint4 reduce_stat(EvictShared<T> &sh, cg::cluster_group &cl, uint32_t a, uint32_t b, uint32_t lo, uint32_t hi) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = (int)cl.num_blocks();
    a = __reduce_add_sync(kFull, a);
    b = __reduce_add_sync(kFull, b);
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    if (lane == 0) {
        sh.stat[warp][0] = a;
        sh.stat[warp][1] = b;
        sh.stat[warp][2] = lo;
        sh.stat[warp][3] = hi;
    }
    __syncthreads();
    const bool in = lane < T / 32;
    a = __reduce_add_sync(kFull, in ? sh.stat[lane % (T / 32)][0] : 0u);
    b = __reduce_add_sync(kFull, in ? sh.stat[lane % (T / 32)][1] : 0u);
    lo = __reduce_min_sync(kFull, sh.stat[lane % (T / 32)][2]);
    hi = __reduce_max_sync(kFull, sh.stat[lane % (T / 32)][3]);
    if (C > 1) {
        if ((int)threadIdx.x < C) {
            uint32_t *to = cl.map_shared_rank(&sh.cstat[0][0], threadIdx.x) + 4 * cl.block_rank();
            to[0] = a;
            to[1] = b;
            to[2] = lo;
            to[3] = hi;
        }
        cl.sync();
        const bool at = lane < C;
        a = __reduce_add_sync(kFull, at ? sh.cstat[lane & 7][0] : 0u);
        b = __reduce_add_sync(kFull, at ? sh.cstat[lane & 7][1] : 0u);
        lo = __reduce_min_sync(kFull, at ? sh.cstat[lane & 7][2] : 0xffffffffu);
        hi = __reduce_max_sync(kFull, at ? sh.cstat[lane & 7][3] : 0u);
    } else {
        __syncthreads();
    }
    return make_uint4(a, b, lo, hi);
}

template <int T, int K>
// Two CTAs of 512 per SM: 512 full rows of 8,192 slots give up one slot each in 23.7 us, 37 in 26.3 (with registers for one
// CTA 33.9 and 35.8, for three, spilling, 24.0 and 26.7); rows of 4,096 15.4 and 16.4 (22.4 and 23.5; 14.2 and 15.5).
__global__ void __launch_bounds__(T, 1024 / T) qevict_kernel(QEvictCall a) {
    __shared__ EvictShared<T> sh;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
    const int row = blockIdx.x / C, h = row % a.c.heads, b = row / a.c.heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kBins; i += T) sh.hist[i] = 0;
    if (tid == 0) sh.listed = 0;
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
    if (a.c.pos) {
        int p[K];
#pragma unroll
        for (int i = 0; i < K; ++i) p[i] = first + 32 * i < cap ? ld_dep(a.c.pos + slot0 + first + 32 * i) : 0;
#pragma unroll
        for (int i = 0; i < K; ++i) cls |= (uint32_t)sc(p[i]) << (2 * i);
    } else {
        cls = 0x55555555u;
    }
    if (C > 1) cl.sync();
    else __syncthreads();
    const int used = sh.used;
    const int e = a.keep >= 0 ? max(0, used - a.keep) : max(0, a.n - (cap - used));
    if (a.keep < 0 && e == 0) {
        // there is room: the next free slots
        int32_t *free = a.out + ((int64_t)b * a.c.heads + h) * a.n;
        for (int i = me * T + tid; i < a.n; i += C * T) free[i] = used + i;
        return;
    }
    uint32_t n0 = 0, n2 = 0, lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        key[i] = weight_key(__uint_as_float(key[i]));
        if (first + 32 * i >= used) cls |= 3u << (2 * i);
        const uint32_t c = cls >> (2 * i) & 3u;
        n0 += c == 0;
        n2 += c == 2;
        if (c == 1) {
            lo = min(lo, key[i]);
            hi = max(hi, key[i]);
        }
    }
    int want = e;
    uint32_t pc = 1, pk = 0;   // the last one's class and key
    if (e > 0) {
        uint4 st = reduce_stat(sh, cl, n0, n2, lo, hi);
        const int plain = used - (int)st.x - (int)st.y;
        if (want <= (int)st.x || want > (int)st.x + plain) {
            // it is an empty slot, or a protected one
            pc = want <= (int)st.x ? 0 : 2;
            want -= pc ? (int)st.x + plain : 0;
            lo = 0xffffffffu;
            hi = 0;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if ((cls >> (2 * i) & 3u) == pc) {
                    lo = min(lo, key[i]);
                    hi = max(hi, key[i]);
                }
            if (C > 1) cl.sync();   // the others have read the first answer
            st = reduce_stat(sh, cl, 0, 0, lo, hi);
        } else {
            want -= (int)st.x;
        }
        lo = st.z;
        hi = st.w;
        for (;;) {
            const int shift = max(0, 21 - __clz(hi - lo));   // (hi - lo) >> shift < 2048
#pragma unroll
            for (int i = 0; i < K; ++i)
                if ((cls >> (2 * i) & 3u) == pc && key[i] >= lo && key[i] <= hi) atomicAdd(&sh.hist[(key[i] - lo) >> shift], 1);
            const int3 p = find_bin<T>(sh, cl, want);
            want -= p.y;
            lo += (uint32_t)p.x << shift;
            hi = min(hi, lo + ((1u << shift) - 1u));
            pk = lo;
            if (shift == 0) break;
            if (p.z <= kRank) {
                uint32_t *list = C > 1 ? cl.map_shared_rank(sh.list, 0) : sh.list;
                int *listed = C > 1 ? cl.map_shared_rank(&sh.listed, 0) : &sh.listed;
#pragma unroll
                for (int i = 0; i < K; ++i)
                    if ((cls >> (2 * i) & 3u) == pc && key[i] >= lo && key[i] <= hi) list[atomicAdd(listed, 1)] = key[i];
                if (C > 1) cl.sync();
                else __syncthreads();
                if (me == 0 && tid < p.z) {
                    const uint32_t mine = sh.list[tid];
                    int less = 0, equal = 0;
                    for (int i = 0; i < p.z; ++i) {
                        less += sh.list[i] < mine;
                        equal += sh.list[i] == mine;
                    }
                    if (want > less && want <= less + equal)   // equal keys write the same
                        for (int r = 0; r < C; ++r) {
                            *cl.map_shared_rank(&sh.last, r) = mine;
                            *cl.map_shared_rank(&sh.ties, r) = want - less;
                        }
                }
                if (C > 1) cl.sync();
                else __syncthreads();
                pk = sh.last;
                want = sh.ties;
                break;
            }
            for (int i = tid; i < kBins; i += T) sh.hist[i] = 0;
            __syncthreads();
        }
    }
    // `want` of the slots equal to (pc, pk) go, the first ones
    uint32_t lower = 0, same = 0;
    int nl = 0, ns = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const uint32_t c = cls >> (2 * i) & 3u;
        const bool in = e > 0 && c < 3;
        const bool lt = in && (c < pc || (c == pc && key[i] < pk)), eq = in && c == pc && key[i] == pk;
        lower |= (uint32_t)lt << i;
        same |= (uint32_t)eq << i;
        nl += __popc(__ballot_sync(kFull, lt));
        ns += __popc(__ballot_sync(kFull, eq));
    }
    if (lane == 0) {
        sh.lower[warp] = nl;
        sh.same[warp] = ns;
    }
    __syncthreads();
    const int vl = lane < T / 32 ? sh.lower[lane % (T / 32)] : 0, vs = lane < T / 32 ? sh.same[lane % (T / 32)] : 0;
    int bl = __reduce_add_sync(kFull, lane < warp ? vl : 0), bs = __reduce_add_sync(kFull, lane < warp ? vs : 0);
    if (C > 1) {
        const int tl = __reduce_add_sync(kFull, vl), ts = __reduce_add_sync(kFull, vs);
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
    if (a.keep >= 0 || nl + ns > 0) {
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
    // all loads first: codes, then (one word per thread at the most) scales, weights and positions
    constexpr int CH = D / 32, STEPS = (kTrimSlots * CH + 255) / 256, G = D / kQGroup;
    static_assert(kTrimSlots * G <= 256, "a thread has one group's scales");
    uint4 v[2][STEPS];
    uint32_t ks = 0, vs = 0;
    float weight = 0.f;
    int pos = 0;
    const int tid = threadIdx.x, sg = tid < kTrimSlots * G ? slots[tid / G] : -1, sw = tid < kTrimSlots ? slots[tid] : -1;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int x = i * 256 + tid, t = x / CH, ch = x % CH;
        const int s = t < kTrimSlots ? slots[t] : -1;
        if (s < 0) continue;
        v[0][i] = ld_dep(reinterpret_cast<const uint4 *>(a.c.k) + (from + s) * CH + ch);
        v[1][i] = ld_dep(reinterpret_cast<const uint4 *>(a.c.v) + (from + s) * CH + ch);
    }
    if (sg >= 0) {
        ks = ld_dep(a.c.ks + (from + sg) * G + tid % G);
        vs = ld_dep(a.c.vs + (from + sg) * G + tid % G);
    }
    if (sw >= 0) {
        weight = ld_dep(a.c.weight + from + sw);
        if (a.c.pos) pos = ld_dep(a.c.pos + from + sw);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int x = i * 256 + tid, t = x / CH, ch = x % CH;
        if (t >= kTrimSlots || slots[t] < 0) continue;
        reinterpret_cast<uint4 *>(dst.k)[(to + t) * CH + ch] = v[0][i];
        reinterpret_cast<uint4 *>(dst.v)[(to + t) * CH + ch] = v[1][i];
    }
    if (sg >= 0) {
        dst.ks[(to + tid / G) * G + tid % G] = ks;
        dst.vs[(to + tid / G) * G + tid % G] = vs;
    }
    if (sw >= 0) {
        dst.weight[to + tid] = weight;
        if (a.c.pos) dst.pos[to + tid] = pos;
    }
}

// The weights of a step without query tokens: nothing is added to what the slots had.
constexpr int kDecayThreads = 256, kDecaySlots = 4096;
__global__ void __launch_bounds__(kDecayThreads) qdecay_kernel(QAttnArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.y, b = blockIdx.z;
    const int used = q_length(a.length, b, a.c.cap, a.err), t0 = blockIdx.x * kDecaySlots, t1 = min(used, t0 + kDecaySlots);
    const int64_t slot0 = a.c.slot0(b, h);
    for (int t = t0 + threadIdx.x; t < t1; t += kDecayThreads)
        a.weight[slot0 + t] = a.decay == 0.f ? 0.f : a.decay * ld_dep(a.c.weight + slot0 + t);
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

constexpr int kMinSlots = 2048;   // (a cluster's barriers cost more than halving fewer: 40 rows of 2,048 in two CTAs each took 8.1, not 5.1 us)
cudaError_t choose_slots(const QEvictCall &a, cudaStream_t s) {
    const int cap = a.keep >= 0 ? a.c.cap : a.limit, sms = device_sm_count();
    const int64_t rows = (int64_t)a.c.heads * a.c.batch;
    // few rows: several CTAs each, as long as the GPU has room and a CTA has at least 2048 slots
    int ctas = 1;
    while (ctas < 8 && ((rows * ctas * 2 <= 2 * sms && cap / (2 * ctas) >= kMinSlots) || cap > 16384 * ctas)) ctas *= 2;
    const int each = (cap + ctas - 1) / ctas;
    if (each <= 2048) return launch_evict<512, 4>(a, ctas, s);
    if (each <= 4096) return launch_evict<512, 8>(a, ctas, s);
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

// empty: no tokens, so no data
cs_status check_rows(const cs_head_rows *r, bool empty, const char *name, const char *who, QRowsK *out) {
    CS_CHECK(r && (r->data || empty), "%s: %s is null", who, name);
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
dim3 rows_grid(const QRowsCall &a, int each) {
    const int64_t rows = (int64_t)a.n * a.c.heads;
    return dim3((unsigned)((rows + each - 1) / each), a.c.batch);
}

cs_status rows_call(const cs_qcache *cache, const cs_head_rows *k, const cs_head_rows *v, int n, const int32_t *start,
                    const int32_t *slots, void *ws, size_t ws_bytes, const char *who, QRowsCall *a) {
    cs_status st = check_cache(cache, true, who, &a->c);
    if (st == CS_OK) st = check_rows(k, n == 0, "k", who, &a->k);
    if (st == CS_OK) st = check_rows(v, n == 0, "v", who, &a->v);
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
        d_head < kQGroup || d_head > 256 || d_head % kQGroup)
        return 0;
    const size_t trim = trim_scratch(batch, kv_heads, capacity);
    if (n_heads == 0) return kControlBytes + trim;
    if (n_heads < kv_heads || n_heads % kv_heads || n_q < 1 || (int64_t)n_heads / kv_heads * n_q > kQMaxRows) return 0;
    const size_t attn = qattn_scratch(batch, kv_heads, capacity, d_head, n_heads, n_q, true, device_sm_count());
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
        auto go = [&](auto kernel) {
            return launch(kernel, rows_grid(a, RowPart<d(), kPart>::ROWS), dim3(kRowThreads), 0, (cudaStream_t)stream, pdl_enabled(), a);
        };
        return a.k.dt == CS_F32   ? go(qappend_kernel<d(), float>)
               : a.k.dt == CS_F16 ? go(qappend_kernel<d(), __half>)
                                  : go(qappend_kernel<d(), __nv_bfloat16>);
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
        return launch(qread_kernel<d()>, rows_grid(a, RowPart<d(), 8>::ROWS * kReadSteps), dim3(kRowThreads), 0, (cudaStream_t)stream, pdl_enabled(), a);
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
    if (st == CS_OK) st = check_rows(q, n_q == 0, "q", who, &a.q);
    if (st == CS_OK) st = check_rows(out, n_q == 0, "out", who, &a.out);
    if (st != CS_OK) return st;
    CS_CHECK(q->dtype == out->dtype, "%s: q and out differ in dtype", who);
    CS_CHECK(n_q == 0 || q->data != out->data, "%s: out must not be q", who);
    CS_CHECK(n_heads >= 1 && n_heads % cache->n_heads == 0, "%s: n_heads=%d is not a multiple of the cache's %d", who, n_heads,
             cache->n_heads);
    CS_CHECK(n_q >= 0, "%s: n_q=%d is negative", who, n_q);
    if ((int64_t)n_heads / cache->n_heads * n_q > kQMaxRows) {
        set_error("%s: %d query rows per cache head, above %d", who, n_heads / cache->n_heads * n_q, kQMaxRows);
        return CS_ERR_UNSUPPORTED;
    }
    if ((int64_t)cache->batch * cache->n_heads * ((cache->capacity + 15) / 16 + 32) >= INT32_MAX) {
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
                   kControlBytes + qattn_scratch(a.c.batch, a.c.heads, a.c.cap, a.c.d, n_heads, n_q, weight != nullptr, a.sms), who);
    if (st != CS_OK) return st;
    a.err = static_cast<uint32_t *>(ws);
    a.scratch = static_cast<char *>(ws) + kControlBytes;
    if (n_q == 0 && !weight) return CS_OK;
    const cudaError_t e = n_q > 0 ? launch_qattn(a, (cudaStream_t)stream)
                                  : launch(qdecay_kernel, dim3((a.c.cap + kDecaySlots - 1) / kDecaySlots, a.c.heads, a.c.batch),
                                           dim3(kDecayThreads), 0, (cudaStream_t)stream, pdl_enabled(), a);
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
