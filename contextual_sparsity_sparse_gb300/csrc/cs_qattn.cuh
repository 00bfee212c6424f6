// Attention over the 4-bit KV cache: the kernels, a translation unit per
// d_head (cs_qattn64.cu ...); cs_qattn.cu holds the host side.
//
// Per query row r (a query head of a cache head's group, at one query token):
//     x_i = q_r . k_i (q scaled),   p_i = 2^((x_i - m) c1),   out = sum p_i v_i / sum p_i.
// With k = z + s n and v = z + s n per group of 64 channels (n = 0 .. 15):
//     q . k = sum_g s_g (q . (n - 8))_g + (z_g + 8 s_g) (sum q)_g
//     sum_i p_i v_i = sum_i (p_i s_i) (n_i - 8) + sum_i p_i (z_i + 8 s_i)
// so the codes go into matrix products as they are and the scales meet only
// sums (keys) or probabilities (values).
//
// Two kernels.  In the first the slots of all sequences and heads, cut into
// units of UT slots, are one long axis that is split evenly over the CTAs,
// whatever the lengths: a CTA may take the end of one head's slots, some whole
// heads, and the start of another.  Its warps take the units of a head in
// turn, each with its own running maximum and sums, fed by its own ring of
// asynchronous copies, which runs on across heads; at a head's end the warps'
// sums are joined.  A head that lies in one CTA is finished there; else the CTA
// leaves a partial record, and the second kernel joins the records and
// finishes (for every CTA of the first a few small ones, so that uneven
// leavings even out; each adds up a share of the records' sums and of the weights).
// Starting and joining a head costs a CTA about as long as kHeadCost units, so
// a head is that much longer on the axis.
//
// Products.  mma.sync m16n8k16 with fp32 sums: the query rows are the
// 8 columns, so a batch-1 head wastes little, and the codes are the A operand
// straight from their packed words.  For the keys, in fp16, 16 slots x 16 channels: a
// nibble ANDed out of a word is an fp16 subnormal n 2^-24 (or, four bits up,
// n 2^-20), exact in the product; the factor 16 goes into q, and the sums start
// at -8 (sum q); where n - 8 itself is the operand, n is ORed into the fraction of 1024 and 1032 subtracted (Kim, Henry,
// Fahim and Awadalla, "Who Says Elephants Can't Run", 2022).  For the values, in bf16, 16 channels x 16 slots: two slots' words are
// interleaved by byte permutes, and a nibble ANDed out is bf16's n 2^-133 (four bits
// up n 2^-129: the bit that leaves the fraction is the exponent's lowest, and the least
// exponent has the subnormals' steps); one multiply-add by 2^127 takes it to (n - 8) / 64 (or / 4).
// The tensor-memory path of the newer matrix instructions needs 128 rows and
// operands in shared memory; with at most 16 query rows per head the products
// are not what bounds this kernel, the instructions around them are.
//
// Precision.  q is scaled by a power of two and split into two fp16 parts (22
// bits, or steps of 2^-35 of the row's largest channel; the second is zero for 16-bit inputs).  p s goes in bf16 parts of 8 bits each:
// two for 16-bit outputs (what is left out is 2^-17 of a term or less, beside output roundings of 2^-8 and
// 2^-11), three for fp32 ones (2^-26).  bf16 has fp32's range, so a term keeps its bits however
// small it is beside others: fp16 parts under one power of two for a warp's slots, rows and groups cost the others
// up to 13 bits where one slot's or one group's scale was 2^15 of theirs, with no weight at all on it (fp32 outputs off by 6e-5).
// With at most 4 rows the first two parts sit in the same 8 columns.  All sums and the softmax statistics are fp32; for
// fp32 outputs (TWO) the keys' codes are taken as n - 8 outright and a unit's value
// products are summed apart (see there).  Logits of size X (64 channels in eight products, each cut off
// after 24 bits) move fp32 outputs by 2^-21 X of the terms at most.
//
// Bound (64 ragged sequences of up to 8,192 slots, 64 over 8 heads of 128, bf16:
// 107 us of which the bytes need 47): 900 instructions per unit of 32 slots, of which some
// 200 are for the keys, 360 for p and the values, 80 for the maxima and x, 250 for
// copies, heads' starts and joins.  The first kernel issues in 62% of its cycles, keeps
// the tensor pipe busy for 27% and moves 374 MB in 90 us (62% of a copy's rate, the
// logits that it leaves included).  When the call took 100 us, its
// copies and joins alone, with all of a unit's arithmetic left out, took 81, and of one long sequence's 47 us 36.
// What else was tried then: four warps to a CTA,
// four CTAs to an SM, 126 us; one CTA of 8, 12 or 16 warps per SM with more
// registers, 118, 114, 119 us; keys and values of a stage replaced one after
// the other as they are used, 109 us.
#pragma once

#include "cs_qcache.cuh"

namespace cs {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxPerSm = 2;   // CTAs of the first kernel
// A head's fixed cost on the axis in units: 8, 16, 24, 32, 48 for
//   64 ragged sequences of up to 8,192 slots (8 rows, 128 channels, bf16): 129, 116, 106, 107, 111 us
//   the same in fp32: 144, 128, 129, 131, 135; without weights: 107, 93, 86, 87, 91; 4 rows: 116, 100, 93, 93, 97
//   32 of up to 4,096 of 64 channels, 16 rows: 63, 47, 43, 44, 47; 16 of 128 channels, 16 rows: 55, 45, 42, 44, 46
//   16 of 192 channels: 57, 49, 41, 41, 37; of 256: 67, 57, 49, 46, 43, 16 rows: 102, 88, 80, 73, 73
//   40 heads of 2,048 slots: 14.0, 14.0, 13.9, 14.4, 15.0; one sequence of 131,001: 49.5, 48.5, 48.3, 48.4, 46.0
// So 24 is the best or near it up to 128 channels; wide rows (one CTA per SM) would take 10% less with 48.
constexpr int kHeadCost = 24;

struct QAttnK {
    QAttnArgs a;
    int group, rows;     // query heads per cache head; rows of this pass
    int row0;            // its first row: row r is head r % group of the group, token r / group
    int grid;            // CTAs of the first kernel
    int subs;            // CTAs of the second kernel for each of them
    int4 *left;          // [grid, 2, 2] what the first kernel left to finish (Left)
    float *part;         // [grid, 2] records: per column its maximum, sum and c1, then the sums of p v
    float *logit;        // [grid, area / RP, RP] x, for the weights (null without weights)
    int64_t area;        // floats of one CTA's part of logit: a head's end in front, if it has one, then one head at a time
    float c2, sign;      // |scale| log2(e), and the scale's sign
};

// CTAs of the first kernel where `most` fit the GPU, for an axis of `cost` units at the most.
inline int qattn_grid(int64_t cost, int64_t most) {
    const int64_t useful = (cost + kWarps - 1) / kWarps;
    return (int)(useful < most ? useful : most);
}
// The most units whose x one CTA keeps at a time, of heads of up to `head` units: one piece of a head as long as its
// part of the axis, or the end of one and a piece of another, which has a head's cost in front of it.
inline int64_t qattn_area(int64_t cost, int grid, int64_t head) {
    int64_t part = (cost + grid - 1) / grid;
    if (part < kWarps) part = kWarps;
    const int64_t one = part < head ? part : head, two = part - kHeadCost < 2 * head ? part - kHeadCost : 2 * head;
    return one > two ? one : two;
}

// Query columns per pass and how they sit in the 8 columns of a product.
enum QMode { PACK4 = 0, ONE8 = 1, TWO8 = 2 };

// Launches both kernels of one d_head.
template <int D>
cudaError_t run_qattn(QAttnK k, int mode, int64_t cost, cudaStream_t s);

#ifdef CS_QATTN_KERNELS

namespace {

template <int D, int MODE>
struct Cfg {
    static constexpr int NT = MODE == TWO8 ? 2 : 1;          // tiles of 8 columns
    static constexpr int RP = MODE == PACK4 ? 4 : 8 * NT;    // query rows
    static constexpr int PARTS = MODE == PACK4 ? 1 : 2;      // q's two parts: same or separate products
    static constexpr int G = D / kQGroup;
    static constexpr int UT = D <= 128 ? 32 : 16;            // slots per unit
    static constexpr int SUB = UT / 16;
    static constexpr int RB = D / 2;                         // bytes of a row
    static constexpr int STAGE = UT * (2 * RB + 8 * G + 4);  // one unit: keys, values, their scales, positions
    static constexpr int MINB = D * NT <= 128 ? kMaxPerSm : 1;   // CTAs per SM
    static constexpr int ST = D == 64 ? 4 : MINB == 2 ? 2 : 3;
    static constexpr int RS = D + 4;                         // floats of a joined column (conflict-free)
    static constexpr int QF = NT * PARTS * (D / 32) * 32;    // uint4 fragments of q, two products each
    static constexpr int CP = RP < 8 || 8 * RS * 4 > STAGE ? 4 : 8;   // columns that are joined at a time: a warp's go into a stage
    static constexpr int CS = 3 + G;                         // floats of a column: c1, last position, on, sums of q
    static constexpr int STAT = kWarps * RP * 2 + 3 * RP;    // floats: the warps' maxima (then factors) and sums, then the joined ones
    static constexpr int REC = RP * (D + 3);                 // floats of a record
    static_assert(CP * RS * 4 <= STAGE && RP % CP == 0, "a pass of the join fits a stage");
    static constexpr size_t smem_fixed = (size_t)kWarps * ST * STAGE + 2 * (QF * 16 + RP * CS * 4) + STAT * 4;
};

template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    if (N == 16) asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_or0(uint32_t dst, const void *src, bool on) {
    if (N == 16) asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(on ? N : 0) : "memory");
}
template <typename T>
__device__ __forceinline__ T lds(const char *p) { return *reinterpret_cast<const T *>(p); }
// A slot's G scale words.
template <int G>
__device__ __forceinline__ void lds_scales(const char *p, uint32_t (&w)[G]) {
    if (G == 2) {
        const uint2 v = lds<uint2>(p);
        w[0] = v.x;
        w[1 % G] = v.y;
    } else if (G == 4) {
        const uint4 v = lds<uint4>(p);
        w[0] = v.x;
        w[1 % G] = v.y;
        w[2 % G] = v.z;
        w[3 % G] = v.w;
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = lds<uint32_t>(p + 4 * g);
    }
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_bf(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (x & mask) | or
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t o) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(o));
    return r;
}
__device__ __forceinline__ uint32_t hsub2u(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// a b + c of two bf16 pairs
__device__ __forceinline__ uint32_t bfma2u(uint32_t a, uint32_t b, uint32_t c) {
    using P = const __nv_bfloat162 *;
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<P>(&a), *reinterpret_cast<P>(&b), *reinterpret_cast<P>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Where a 16-byte chunk of a unit's row lies: pairs of chunks (the 32 bytes of a
// group) are permuted so that the four slots of which a half warp reads the
// keys, or a warp the values, lie in different banks.  Rows of 32 and 96 bytes
// need nothing.
template <int D>
__device__ __forceinline__ int swizzle(int tok) { return D == 128 ? tok & 2 : D == 256 ? (tok & 3) << 1 : 0; }
// The slot within 16 that is row i of a product.  Of any four in the above, no
// two are alike modulo 4; slot_of_row(i + 1) = slot_of_row(i) ^ 2 for even i.
__device__ __forceinline__ int slot_of_row(int i) {
    return (i & 8) | (i & 4) | (((i & 1) ^ ((i >> 2) & 1)) << 1) | ((i >> 1) & 1);
}

// ------------------------------------------------------------ the split axis

// Whether a cache head has a chosen query head.
__device__ __forceinline__ bool kv_on(const QAttnK &k, int b, int h) {
    if (!k.a.mask) return true;
    const uint32_t *m = k.a.mask + (int64_t)b * ((k.a.heads + 31) / 32);
    for (int j = h * k.group; j < (h + 1) * k.group;) {
        const int bit = j & 31, n = min(32 - bit, (h + 1) * k.group - j);
        const uint32_t w = ld_dep(m + (j >> 5)) >> bit;
        if (n == 32 ? w : w & ((1u << n) - 1u)) return true;
        j += n;
    }
    return false;
}

__device__ __forceinline__ bool row_on(const QAttnK &k, int b, int h, int r) {
    if (r >= k.rows) return false;
    if (!k.a.mask) return true;
    const int j = h * k.group + (k.row0 + r) % k.group;
    return ld_dep(k.a.mask + (int64_t)b * ((k.a.heads + 31) / 32) + (j >> 5)) >> (j & 31) & 1u;
}

// The last position that a row sees; past the largest there is, that.
__device__ __forceinline__ int last_seen(const QAttnK &k, int b, int r) {
    if (!k.a.q_pos) return INT_MAX;
    const int t = (k.row0 + r) / k.group;
    return min(ld_dep(k.a.q_pos + b), INT_MAX - t) + t;
}

// How many cache heads have a chosen query head; the whole warp asks together.
__device__ __forceinline__ int heads_on(const QAttnK &k, int b) {
    if (!k.a.mask) return k.a.c.heads;
    int n = 0;
    for (int h0 = 0; h0 < k.a.c.heads; h0 += 32) {
        const int h = h0 + (threadIdx.x & 31);
        n += __popc(__ballot_sync(kFull, h < k.a.c.heads && kv_on(k, b, h)));
    }
    return n;
}

// The cache head that is the sequence's n-th with a chosen query head; the whole warp asks together.
__device__ __forceinline__ int chosen_head(const QAttnK &k, int b, int n) {
    if (!k.a.mask) return n;
    for (int h0 = 0; h0 < k.a.c.heads; h0 += 32) {
        const int h = h0 + (threadIdx.x & 31);
        const uint32_t on = __ballot_sync(kFull, h < k.a.c.heads && kv_on(k, b, h));
        const int c = __popc(on);
        if (n < c) {
            const bool it = (on >> (threadIdx.x & 31) & 1u) && __popc(on & ((1u << (threadIdx.x & 31)) - 1u)) == n;
            return h0 + __ffs(__ballot_sync(kFull, it)) - 1;
        }
        n -= c;
    }
    return k.a.c.heads - 1;   // not reached while the mask stays as it was counted
}

// In shared memory per sequence: its length, and where it starts on the axis (one more at the end).
struct Axis {
    int *len, *pre;
    int per;          // a CTA's length of the axis
    int begin, end;   // this CTA's part

    template <int UT>
    __device__ __forceinline__ int cost(int n, int heads) {
        return n ? ((n + UT - 1) / UT + kHeadCost) * heads : 0;
    }

    template <int UT>
    __device__ void build(const QAttnK &k, int *smem, int *wsum, bool flag) {
        len = smem;
        pre = smem + k.a.c.batch;
        const int B = k.a.c.batch, lane = threadIdx.x & 31;
        uint32_t *err = flag ? k.a.err : nullptr;
        int total;
        if (B <= 32) {
            // every warp writes the same values, so no warp waits for another
            const int n = lane < B ? q_length(k.a.length, lane, k.a.c.cap, err) : 0;
            int heads = k.a.c.heads;
            if (k.a.mask) {
#pragma unroll 4
                for (int b = 0; b < B; ++b) {
                    const int on = heads_on(k, b);
                    if (lane == b) heads = on;
                }
            }
            const int v = cost<UT>(n, heads);
            int inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int m = __shfl_up_sync(kFull, inc, o);
                if (lane >= o) inc += m;
            }
            total = __shfl_sync(kFull, inc, 31);
            if (lane < B) {
                len[lane] = n;
                pre[lane] = inc - v;
            }
            if (lane == 0) pre[B] = total;
            __syncwarp();
        } else {
            if (k.a.mask) {
                for (int b = threadIdx.x >> 5; b < B; b += kWarps) {
                    const int on = heads_on(k, b);
                    if (lane == 0) pre[b] = on;
                }
                __syncthreads();
            }
            const int each = (B + kThreads - 1) / kThreads;
            const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
            int sum = 0;
            for (int b = b0; b < b1; ++b) {
                const int n = q_length(k.a.length, b, k.a.c.cap, err);
                const int v = cost<UT>(n, k.a.mask ? pre[b] : k.a.c.heads);
                len[b] = n;
                pre[b] = v;   // not yet summed
                sum += v;
            }
            int at = block_excl_scan(sum, wsum, &total);
            for (int b = b0; b < b1; ++b) {
                const int v = pre[b];
                pre[b] = at;
                at += v;
            }
            if (threadIdx.x == 0) pre[B] = total;
            __syncthreads();
        }
        // a warp without a unit saves nothing, so a CTA takes at least one for each
        per = max((total + k.grid - 1) / k.grid, kWarps);
        begin = (int)min((int64_t)total, (int64_t)blockIdx.x * per);
        end = (int)min((int64_t)total, (int64_t)begin + per);
    }
};

// A CTA's share of one head's units.
struct Seg {
    int b, h;         // sequence, and which of its chosen heads
    int u0, u1;       // units [u0, u1) ...
    int nu;           // ... of nu
    int first;        // the first unit's place on the axis

    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == nu; }
    __device__ __forceinline__ int next() const { return first + nu; }
    template <int UT>
    __device__ __forceinline__ void seek(const Axis &x, int at, int from_b) {
        b = from_b;
        while (x.pre[b + 1] <= at) ++b;
        nu = (x.len[b] + UT - 1) / UT;
        const int rel = at - x.pre[b];
        h = rel / (nu + kHeadCost);
        first = x.pre[b] + h * (nu + kHeadCost) + kHeadCost;
        u0 = max(0, at - first);
        u1 = max(u0, min(nu, x.end - first));   // none, if this CTA's part ends before them
    }
};

__device__ __forceinline__ int first_seq(const Axis &x, int B, int at) {
    int lo = 0, hi = B;   // the last b with pre[b] <= at; empty ones before it are passed over by seek
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (x.pre[mid] <= at) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A row's statistics: m and l of its pass, m in units of 1 / c1.
__device__ __forceinline__ void put_stat(const QAttnK &k, int b, int head, int row, float m, float l, float c1) {
    const int r = k.row0 + row;
    k.a.stat[((int64_t)b * k.a.n_q + r / k.group) * k.a.heads + head * k.group + r % k.group] =
        make_float2(m == -INFINITY ? -INFINITY : m * c1, l);
}

__device__ __forceinline__ int64_t out_at(const QAttnK &k, int b, int head, int row) {
    const int r = k.row0 + row;
    return b * k.a.out.ldb + r / k.group * k.a.out.ldt + (int64_t)(head * k.group + r % k.group) * k.a.out.ldh;
}

// The weights of n slots from slot0 on, from the x that were left at lg: RP / 4
// threads to a slot, each four columns.  base, c1, inv: per column.
template <int RP, int U, bool AHEAD>
__device__ __forceinline__ void weigh(const QAttnK &k, const float *lg, int n, int64_t slot0, const float *base, const float *c1,
                                      const float *inv) {
    constexpr int L = RP / 4;
    const int c = threadIdx.x % L * 4;
    float bb[4], cc[4], ii[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bb[i] = base[c + i];
        cc[i] = c1[c + i];
        ii[i] = inv[c + i];
    }
    // U slots a round, loads first (the compiler may not move them over stores); whole warps go round, so that the
    // shuffles have all their lanes.  AHEAD: the next round's loads are under way while this one is worked on.
    constexpr int STEP = kThreads / L;
    struct Round {
        float4 x[U];
        float old[U];
    };
    auto load = [&](Round &d, int t0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int t = t0 + i * STEP + threadIdx.x / L;
            d.x[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            d.old[i] = 0.f;
            if (t < n) {
                d.x[i] = ld_dep(reinterpret_cast<const float4 *>(lg + (int64_t)t * RP + c));
                if (c == 0 && k.a.decay != 0.f) d.old[i] = ld_dep(k.a.c.weight + slot0 + t);
            }
        }
    };
    Round now, next;
    if (AHEAD) load(now, 0);
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += U * STEP) {
        if (AHEAD) load(next, t0 + U * STEP);
        else load(now, t0);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int t = t0 + i * STEP + threadIdx.x / L;
            float w = exp2_approx((now.x[i].x - bb[0]) * cc[0]) * ii[0];
            w = fmaf(exp2_approx((now.x[i].y - bb[1]) * cc[1]), ii[1], w);
            w = fmaf(exp2_approx((now.x[i].z - bb[2]) * cc[2]), ii[2], w);
            w = fmaf(exp2_approx((now.x[i].w - bb[3]) * cc[3]), ii[3], w);
#pragma unroll
            for (int o = 1; o < L; o <<= 1) w += __shfl_xor_sync(kFull, w, o);
            if (t < n && c == 0) k.a.weight[slot0 + t] = fmaf(k.a.decay, now.old[i], w);
        }
        if (AHEAD) now = next;
    }
}

// ------------------------------------------------------------- first kernel

// A row's m moves only when an x leads it by more than 2^kLead in p (moving it
// scales all sums): most rows keep the m of their first unit.
constexpr float kLead = 8.f;

template <int D, int MODE>
struct Tile {
    using C = Cfg<D, MODE>;
    float o[C::G * 4][C::NT][4];     // channels 8 (lane / 4) + 2 t (+ 1) of group g in o[4 g + t], columns 2 (lane % 4) (+ 1)
    float z[C::G][C::NT][2];         // sums of p (z + 8 s), this lane's slots
    float l[C::NT][2];               // sums of p, this lane's slots
    float m[C::NT][2];               // largest x so far
    float ms[C::NT][2];              // the same, 0 for -inf
    float t[C::NT][2];               // an x beyond this one moves m

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
#pragma unroll
            for (int x = 0; x < C::G * 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[x][n][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = -INFINITY;
                ms[n][i] = 0.f;
                t[n][i] = -INFINITY;
                l[n][i] = 0.f;
#pragma unroll
                for (int g = 0; g < C::G; ++g) z[g][n][i] = 0.f;
            }
        }
    }
};

// Starts the copies of one unit of a head, n slots or more, into a stage of the warp's ring.
template <int D, int MODE>
__device__ __forceinline__ void fetch(const QAttnK &k, uint32_t stage, int64_t slot0, int n) {
    using C = Cfg<D, MODE>;
    constexpr int CH = C::RB / 16, N = C::UT * CH;
    // a slot's scales go in one piece, or (12 bytes) word by word
    constexpr int SP = C::G == 3 ? 4 : 4 * C::G, SN = C::UT * C::G * 4 / SP;
    const int lane = threadIdx.x & 31;
    const QCacheK &c = k.a.c;
    const uint8_t *kp = c.k + slot0 * C::RB + lane * 16, *vp = c.v + slot0 * C::RB + lane * 16;
    const char *ks = reinterpret_cast<const char *>(c.ks + slot0 * C::G) + lane * SP;
    const char *vs = reinterpret_cast<const char *>(c.vs + slot0 * C::G) + lane * SP;
    const uint32_t sc = stage + 2 * C::UT * C::RB + lane * SP;
    if (n >= C::UT) {
#pragma unroll
        for (int i = 0; i < N; i += 32) {
            const int tok = (i + lane) / CH;
            const uint32_t at = stage + tok * C::RB + (((i + lane) % CH ^ swizzle<D>(tok)) << 4);
            cp_async<16>(at, kp + i * 16);
            cp_async<16>(at + C::UT * C::RB, vp + i * 16);
        }
#pragma unroll
        for (int i = 0; i < SN; i += 32)
            if (SN % 32 == 0 || i + lane < SN) {
                cp_async<SP>(sc + i * SP, ks + i * SP);
                cp_async<SP>(sc + C::UT * C::G * 4 + i * SP, vs + i * SP);
            }
    } else {
        // what lies past the head's slots is not read; zeros stand in the ring
        for (int i = 0; i < N; i += 32) {
            const int tok = (i + lane) / CH;
            const uint32_t at = stage + tok * C::RB + (((i + lane) % CH ^ swizzle<D>(tok)) << 4);
            const bool on = tok < n;
            cp_async_or0<16>(at, on ? kp + i * 16 : c.k, on);
            cp_async_or0<16>(at + C::UT * C::RB, on ? vp + i * 16 : c.v, on);
        }
        for (int i = 0; i < SN; i += 32)
            if (i + lane < SN) {
                const bool on = (i + lane) * SP < n * C::G * 4;
                cp_async_or0<SP>(sc + i * SP, on ? ks + i * SP : reinterpret_cast<const char *>(c.ks), on);
                cp_async_or0<SP>(sc + C::UT * C::G * 4 + i * SP, on ? vs + i * SP : reinterpret_cast<const char *>(c.vs), on);
            }
    }
    if ((k.a.q_pos || k.a.taken) && lane < C::UT)
        cp_async_or0<4>(stage + C::UT * (2 * C::RB + C::G * 8) + lane * 4, lane < n ? c.pos + slot0 + lane : c.pos, lane < n);
}

// Slots that 16-bit outputs sum up in one chain of cut off products per warp (an eighth of them each).  Over 131,072 slots
// of one head and CTA a chain lost 2e-5 to 6e-5 of a flat average, an eighth of fp16's half step at the most; over 2^24 it
// would lose bf16's.  Longer pieces take the fp32 outputs' kernel, which loses nothing.
constexpr int64_t kChain = 131072;

// TWO: q has a second part, p s a third, and sums are kept to fp32's precision.
template <int D, int MODE, bool TWO>
__global__ void __launch_bounds__(kThreads, Cfg<D, MODE>::MINB) qattn_kernel(QAttnK k) {
    using C = Cfg<D, MODE>;
    extern __shared__ __align__(16) char smem[];
    // this head's query fragments and column data, and the next one's
    uint4 *qf = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * C::ST * C::STAGE), *qf_next = qf + C::QF;
    float *cols = reinterpret_cast<float *>(qf_next + C::QF), *cols_next = cols + C::RP * C::CS;
    float *stat = cols_next + C::RP * C::CS;
    int *axis_mem = reinterpret_cast<int *>(stat + C::STAT);
    __shared__ int wsum[32];
    __shared__ int woff[kWarps];
    __shared__ int64_t outs[2][C::RP];
    int64_t *out_row = outs[0], *out_next = outs[1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, j = lane & 3;
    const QCacheK &c = k.a.c;
    pdl_wait();
    pdl_launch_dependents();
    if (tid < 2) k.left[blockIdx.x * 4 + tid] = k.left[blockIdx.x * 4 + 2 + tid] = make_int4(0, 0, 0, 0);
    Axis ax{};
    ax.build<C::UT>(k, axis_mem, wsum, blockIdx.x == 0);
    if (ax.begin >= ax.end) return;

    const char *ring = smem + warp * C::ST * C::STAGE;
    const uint32_t ring_at = smem_addr(ring);
    const bool by_pos = k.a.q_pos || k.a.taken, weighing = k.a.weight != nullptr;

    // the fetching side runs ahead of the computing side, on across heads
    Seg s{};
    s.template seek<C::UT>(ax, ax.begin, first_seq(ax, c.batch, ax.begin));
    Seg f = s;
    int fu = f.u0 + warp, fstage = 0;
    int fhead = chosen_head(k, f.b, f.h);
    bool more = true;
    auto fetch_next = [&]() {
        while (more && fu >= f.u1) {
            if (f.next() >= ax.end) {
                more = false;
            } else {
                f.template seek<C::UT>(ax, f.next(), f.b);
                fu = f.u0 + warp;
                fhead = chosen_head(k, f.b, f.h);
            }
        }
        if (more) {
            fetch<D, MODE>(k, ring_at + fstage * C::STAGE, c.slot0(f.b, fhead) + (int64_t)fu * C::UT, ax.len[f.b] - fu * C::UT);
            fu += kWarps;
        }
        fstage = fstage + 1 == C::ST ? 0 : fstage + 1;
        cp_async_commit();
    };

    // what this lane reads of a unit, from the start of a stage
    const int tok0 = slot_of_row(r), vtok = slot_of_row(2 * j);
    int kat[C::G], vat[2][C::G];   // of sub-unit 0; 8 rows and sub-units further, only the row differs
#pragma unroll
    for (int g = 0; g < C::G; ++g) {
        kat[g] = tok0 * C::RB + (((2 * g) ^ swizzle<D>(tok0)) << 4) + j * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tok = vtok ^ (2 * i);
            vat[i][g] = C::UT * C::RB + tok * C::RB + (((2 * g) ^ swizzle<D>(tok)) << 4) + r * 4;
        }
    }

    int stage = 0;
    Tile<D, MODE> T;
    // a warp's query rows (rows warp, warp + 8) of a head, fetched ahead of their use
    constexpr int QR = (C::RP + kWarps - 1) / kWarps;
    float qv[QR][D / 32];
    auto fetch_q = [&](int b, int h) {
#pragma unroll
        for (int i = 0; i < QR; ++i) {
            const int row = warp + i * kWarps, t = (k.row0 + row) / k.group;
            const bool on = row < C::RP && row_on(k, b, h, row);
            const int64_t src = b * k.a.q.ldb + t * k.a.q.ldt + (int64_t)(h * k.group + (k.row0 + row) % k.group) * k.a.q.ldh;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) qv[i][e] = on ? k.sign * q_load1(k.a.q, src + e * 32 + lane) : 0.f;
        }
    };
    // ... turned into fragments, and the columns' data, of head h of sequence b, in the `next` buffers
    auto put_q = [&](int b, int h) {
        __half *qh = reinterpret_cast<__half *>(qf_next);
#pragma unroll
        for (int qi = 0; qi < QR; ++qi) {
            const int row = warp + qi * kWarps;
            if (row >= C::RP) break;
            float (&q)[D / 32] = qv[qi];
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) big = fmaxf(big, fabsf(q[i]));
            big = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(big)));
            // the power of two that takes the largest to [2^14, 2^15); infinities stay what they are
            const int eb = (int)(__float_as_uint(big) >> 23);
            const int up = big > 0.f && eb < 255 ? min(141 - eb, 127) : 0;
            const float f1 = __uint_as_float((uint32_t)(127 + up / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                // channel 32 i + lane of the row is nibble `nib` of word `w` of lane jj's two words of its group
                const int jj = (i & 1) * 2 + (lane >> 4), w = (i & ~1) + ((lane >> 3) & 1), nib = lane & 7;
                q[i] = q[i] * f1 * f2;
                const float v = nib & 1 ? q[i] * 0.0625f : q[i];
                const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
                const int col = row & 7, nt = row >> 3;
                auto put = [&](int tile, int cc, __half x) {
                    qh[((tile * (D / 32) + w) * 32 + cc * 4 + jj) * 8 + ((nib & 3) >> 1) * 4 + (nib & 1) * 2 + (nib >> 2)] = x;
                };
                put(nt * C::PARTS, col, hi);
                if (C::PARTS == 1) put(0, col + 4, lo);
                else if (TWO) put(nt * 2 + 1, col, lo);
            }
            float sum[C::G];
#pragma unroll
            for (int g = 0; g < C::G; ++g) sum[g] = warp_sum(q[2 * g] + q[2 * g + 1]);
            if (lane == 0) {
                float *cc = cols_next + row * C::CS;
                out_next[row] = out_at(k, b, h, row);
                // takes the products back; kept where x c1 stays in fp32's range (beyond, one slot takes all as well)
                cc[0] = fminf(fmaxf(k.c2 * exp2f((float)((TWO ? 0 : 24) - up)), 1.2e-38f), 1.2e30f);
                cc[1] = __int_as_float(by_pos ? last_seen(k, b, row) : INT_MAX);
                cc[2] = row_on(k, b, h, row) ? 1.f : 0.f;
#pragma unroll
                for (int g = 0; g < C::G; ++g) cc[3 + g] = sum[g] * (TWO ? 1.f : 5.9604644775390625e-8f);   // 2^-24, as the products
            }
        }
    };
    auto turn = [&]() {
        uint4 *t = qf;
        qf = qf_next;
        qf_next = t;
        float *u = cols;
        cols = cols_next;
        cols_next = u;
        int64_t *v = out_row;
        out_row = out_next;
        out_next = v;
    };
    if (s.u0 >= s.u1) return;   // only the last head of a CTA's part can have no unit in it
    // the x of the head's end that this CTA's part begins with stay; the heads after it follow one another behind them
    const int front = s.u0 == 0 ? 0 : s.u1 - s.u0;
    int head = fhead;
    fetch_q(s.b, head);   // ahead of the ring's first copies, behind which it would wait
#pragma unroll 1
    for (int i = 0; i < C::ST - 1; ++i) fetch_next();
    put_q(s.b, head);
    turn();
    __syncthreads();
    for (;;) {
        constexpr bool two = TWO && C::PARTS == 2;
        float c1[C::NT][2], inv1[C::NT][2], zq[C::NT][2][C::G];
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *cc = cols + (MODE == PACK4 ? (j & 1) * 2 + i : n * 8 + j * 2 + i) * C::CS;
                c1[n][i] = cc[0];
                inv1[n][i] = 1.f / cc[0];
#pragma unroll
                for (int g = 0; g < C::G; ++g) zq[n][i][g] = MODE == PACK4 && j >= 2 ? 0.f : cc[3 + g];
            }
        T.clear();
        const int newest = by_pos ? last_seen(k, s.b, k.rows - 1) : 0;
        const int len = ax.len[s.b];
        float *lg = k.logit + blockIdx.x * k.area + (s.u0 == 0 ? front : 0) * (int64_t)(C::UT * C::RP);

        Seg nx = s;
        bool last = s.next() >= ax.end;
        if (!last) {
            nx.template seek<C::UT>(ax, s.next(), s.b);
            last = nx.u0 >= nx.u1;
        }
        const int nhead = last ? 0 : chosen_head(k, nx.b, nx.h);
        bool asked = last;   // whether the next head's query rows are on their way: from the warp's last unit on

        for (int u = s.u0 + warp; u < s.u1; u += kWarps) {
            if (!asked && u + kWarps >= s.u1) {
                fetch_q(nx.b, nhead);
                asked = true;
            }
            __syncwarp();
            fetch_next();
            cp_async_wait<C::ST - 1>();
            __syncwarp();
            const char *ub = ring + stage * C::STAGE, *sb = ub + 2 * C::UT * C::RB;
            stage = stage + 1 == C::ST ? 0 : stage + 1;

            // ---- x = sum_g s_g (q . (n - 8))_g + (z_g + 8 s_g) (sum q)_g
            float x[C::SUB][C::NT][4];
            uint32_t ks[C::SUB][2][C::G];
#pragma unroll
            for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                for (int i = 0; i < 2; ++i) lds_scales<C::G>(sb + (sub * 16 + 8 * i + tok0) * C::G * 4, ks[sub][i]);
#pragma unroll
            for (int g = 0; g < C::G; ++g) {
                float acc[C::SUB][C::NT][4];
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float a0 = TWO ? 0.f : -8.f * zq[n][q][g];
#pragma unroll
                        for (int sub = 0; sub < C::SUB; ++sub) acc[sub][n][q] = acc[sub][n][2 + q] = a0;
                    }
                uint2 kw[C::SUB][2];
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                    for (int i = 0; i < 2; ++i) kw[sub][i] = lds<uint2>(ub + kat[g] + (sub * 16 + 8 * i) * C::RB);
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        const uint4 *qa = qf + (n * C::PARTS * (D / 32) + 2 * g + w) * 32 + lane;
                        const uint4 b = *qa;
                        uint4 b2 = make_uint4(0, 0, 0, 0);
                        if (two) b2 = qa[(D / 32) * 32];
#pragma unroll
                        for (int step = 0; step < 2; ++step)
#pragma unroll
                            for (int sub = 0; sub < C::SUB; ++sub) {
                                uint32_t a[4];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    uint32_t v = w ? kw[sub][i].y : kw[sub][i].x;
                                    if (step) v >>= 8;
                                    if (TWO) {
                                        // a product's 16 terms are cut off alike, after the largest: n - 8 itself is nearer 0
                                        a[i] = hsub2u(and_or(v, 0x000f000fu, 0x64006400u), 0x64086408u);
                                        a[i + 2] = hsub2u(and_or(v, 0x00f000f0u, 0x64006400u), 0x64806480u);
                                    } else {
                                        a[i] = v & 0x000f000fu;
                                        a[i + 2] = v & 0x00f000f0u;
                                    }
                                }
                                mma16816(acc[sub][n], a, step ? b.z : b.x, step ? b.w : b.y);
                                if (two) mma16816(acc[sub][n], a, step ? b2.z : b2.x, step ? b2.w : b2.y);
                            }
                    }
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float sc, zo;
                        half2x(ks[sub][i][g], sc, zo);
                        zo = fmaf(8.f, sc, zo);
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const float v = g == 0 ? zo * zq[n][q][g] : fmaf(zo, zq[n][q][g], x[sub][n][2 * i + q]);
                                x[sub][n][2 * i + q] = fmaf(acc[sub][n][2 * i + q], sc, v);
                            }
                    }
            }
            if (MODE == PACK4) {
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[sub][0][i] += __shfl_xor_sync(kFull, x[sub][0][i], 2);
            }
            uint32_t vs[C::SUB][2][C::G];
#pragma unroll
            for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    lds_scales<C::G>(sb + C::UT * C::G * 4 + (sub * 16 + 8 * i + tok0) * C::G * 4, vs[sub][i]);
            // ---- what is not seen is -inf, and the value scales of slots that no row sees count as 0
            if (by_pos || (u + 1) * C::UT > len) {
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int tok = sub * 16 + 8 * i + tok0;
                        int p = 0;
                        bool there = u * C::UT + tok < len;
                        if (by_pos) {
                            p = lds<int>(sb + C::UT * C::G * 8 + tok * 4);
                            there = there && p >= 0 && p <= newest;
                        }
#pragma unroll
                        for (int g = 0; g < C::G; ++g) vs[sub][i][g] = there ? vs[sub][i][g] : 0u;
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int col = MODE == PACK4 ? (j & 1) * 2 + q : n * 8 + j * 2 + q;
                                if (!there || p > __float_as_int(cols[col * C::CS + 1])) x[sub][n][2 * i + q] = -INFINITY;
                            }
                    }
            }
            if (weighing && (MODE != PACK4 || j < 2)) {
                float *to = lg + ((u - s.u0) * C::UT + tok0) * (int64_t)C::RP + 2 * j;
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
                            *reinterpret_cast<float2 *>(to + (sub * 16 + 8 * i) * C::RP + n * 8) =
                                make_float2(x[sub][n][2 * i], x[sub][n][2 * i + 1]);
            }
            // ---- the running maxima
            float mx[C::NT][2];
            bool grow = false;
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    mx[n][q] = fmaxf(x[0][n][q], x[0][n][2 + q]);
                    if (C::SUB == 2) mx[n][q] = fmaxf(mx[n][q], fmaxf(x[C::SUB - 1][n][q], x[C::SUB - 1][n][2 + q]));
                    grow |= mx[n][q] > T.t[n][q];
                }
            if (__any_sync(kFull, grow)) {
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float m = fmaxf(mx[n][q], T.m[n][q]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                        // a column that need not move stays, and so do its sums
                        m = m > T.t[n][q] ? m : T.m[n][q];
                        // nothing but zeros, or NaN, came before the first finite x
                        const float al = T.m[n][q] == -INFINITY ? 0.f : exp2_approx((T.m[n][q] - m) * c1[n][q]);
                        T.m[n][q] = m;
                        T.ms[n][q] = m == -INFINITY ? 0.f : m;
                        T.t[n][q] = fmaf(kLead, inv1[n][q], m);
                        T.l[n][q] *= al;
#pragma unroll
                        for (int g = 0; g < C::G; ++g) T.z[g][n][q] *= al;
#pragma unroll
                        for (int t = 0; t < C::G * 4; ++t) {
                            T.o[t][n][q] *= al;
                            T.o[t][n][2 + q] *= al;
                        }
                    }
            }
            // ---- p, its sums, and p s as fragments
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &v = x[sub][n][2 * i + q];
                            v = exp2_approx((v - T.ms[n][q]) * c1[n][q]);
                            T.l[n][q] += v;
                        }
            // p s of one group and 16 slots as fragments, in two parts of 8 bits, for fp32 outputs three
            auto weights = [&](int g, int sub, uint32_t (&ph)[C::NT][2], uint32_t (&pl)[C::NT][2], uint32_t (&p3)[C::NT][2]) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float sc, zo;
                    half2x(vs[sub][i][g], sc, zo);
                    zo = fmaf(8.f, sc, zo);
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        const float p0 = x[sub][n][2 * i], p1 = x[sub][n][2 * i + 1];
                        T.z[g][n][0] = fmaf(p0, zo, T.z[g][n][0]);
                        T.z[g][n][1] = fmaf(p1, zo, T.z[g][n][1]);
                        const float a0 = p0 * sc, a1 = p1 * sc;
                        float h0, h1, l0, l1;
                        const uint32_t h = pack_bf2(a0, a1);
                        bf2x(h, h0, h1);
                        const uint32_t lo = pack_bf2(a0 - h0, a1 - h1);
                        uint32_t third = 0;
                        if (TWO) {
                            bf2x(lo, l0, l1);
                            third = pack_bf2((a0 - h0) - l0, (a1 - h1) - l1);
                        }
                        if (MODE == PACK4) {
                            ph[n][i] = transpose8x8(j >= 2 ? lo : h);
                            if (TWO) p3[n][i] = transpose8x8(j >= 2 ? third : 0u);   // beside lo: h's sums stay exact
                        } else {
                            ph[n][i] = transpose8x8(h);
                            pl[n][i] = transpose8x8(lo);
                            if (TWO) p3[n][i] = transpose8x8(third);
                        }
                    }
                }
            };
            // the values' words of one group and 16 slots, and of them the fragment of channels 2 t, 2 t + 1 (of 8) of
            // every lane row: rows of a product are channels, its columns the slots' order of the keys' rows
            auto words = [&](int g, int sub, uint32_t (&w)[4]) {
                uint32_t vw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) vw[i] = lds<uint32_t>(ub + vat[i & 1][g] + (sub * 16 + 8 * (i >> 1)) * C::RB);
                w[0] = __byte_perm(vw[0], vw[1], 0x5410);
                w[1] = __byte_perm(vw[2], vw[3], 0x5410);
                w[2] = __byte_perm(vw[0], vw[1], 0x7632);
                w[3] = __byte_perm(vw[2], vw[3], 0x7632);
            };
            auto fragment = [&](const uint32_t (&w)[4], int t, uint32_t (&fr)[4]) {
                const uint32_t av = t & 1 ? w[t & 2] >> 8 : w[t & 2], bv = t & 1 ? w[(t & 2) + 1] >> 8 : w[(t & 2) + 1];
                fr[0] = bfma2u(av & 0x000f000fu, 0x7f007f00u, 0xbe00be00u);
                fr[1] = bfma2u(av & 0x00f000f0u, 0x7f007f00u, 0xc000c000u);
                fr[2] = bfma2u(bv & 0x000f000fu, 0x7f007f00u, 0xbe00be00u);
                fr[3] = bfma2u(bv & 0x00f000f0u, 0x7f007f00u, 0xc000c000u);
            };
            if (TWO) {
                // A product's sum is cut off, not rounded, so long chains drift: for fp32 outputs a unit's products are
                // summed from zero and added to the others with a rounding.
#pragma unroll
                for (int g = 0; g < C::G; ++g) {
                    uint32_t ph[C::SUB][C::NT][2], pl[C::SUB][C::NT][2], p3[C::SUB][C::NT][2], w[C::SUB][4];
#pragma unroll
                    for (int sub = 0; sub < C::SUB; ++sub) {
                        weights(g, sub, ph[sub], pl[sub], p3[sub]);
                        words(g, sub, w[sub]);
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float sum[C::NT][4] = {};
#pragma unroll
                        for (int sub = 0; sub < C::SUB; ++sub) {
                            uint32_t fr[4];
                            fragment(w[sub], t, fr);
#pragma unroll
                            for (int n = 0; n < C::NT; ++n) {
                                mma16816_bf(sum[n], fr, p3[sub][n][0], p3[sub][n][1]);
                                if (MODE != PACK4) mma16816_bf(sum[n], fr, pl[sub][n][0], pl[sub][n][1]);
                                mma16816_bf(sum[n], fr, ph[sub][n][0], ph[sub][n][1]);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) T.o[g * 4 + t][n][i] += sum[n][i];
                    }
                }
            } else {
#pragma unroll
                for (int g = 0; g < C::G; ++g)
#pragma unroll
                    for (int sub = 0; sub < C::SUB; ++sub) {
                        uint32_t ph[C::NT][2], pl[C::NT][2], p3[C::NT][2], w[4];
                        weights(g, sub, ph, pl, p3);
                        words(g, sub, w);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            uint32_t fr[4];
                            fragment(w, t, fr);
#pragma unroll
                            for (int n = 0; n < C::NT; ++n) {
                                mma16816_bf(T.o[g * 4 + t][n], fr, ph[n][0], ph[n][1]);
                                if (MODE != PACK4) mma16816_bf(T.o[g * 4 + t][n], fr, pl[n][0], pl[n][1]);
                            }
                        }
                    }
            }
        }

        if (!last) {
            if (!asked) fetch_q(nx.b, nhead);
            put_q(nx.b, nhead);
        }
        // ---- the warps' sums become one: each leaves its own in the stage of its ring that is free
        const bool whole = s.whole();
        float *rec = k.part + ((int64_t)blockIdx.x * 2 + (s.u0 == 0)) * C::REC;
        float *base = stat + 2 * kWarps * C::RP, *sum = base + C::RP, *cc1 = sum + C::RP;
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    T.l[n][q] += __shfl_xor_sync(kFull, T.l[n][q], o);
#pragma unroll
                    for (int g = 0; g < C::G; ++g) T.z[g][n][q] += __shfl_xor_sync(kFull, T.z[g][n][q], o);
                }
                if (r == 0 && (MODE != PACK4 || j < 2)) {
                    const int col = n * 8 + 2 * j + q;
                    stat[warp * C::RP + col] = T.m[n][q];
                    stat[(kWarps + warp) * C::RP + col] = T.l[n][q];
                }
            }
        if (lane == 0) woff[warp] = (warp * C::ST + fstage) * C::STAGE;
        float *mine = reinterpret_cast<float *>(smem + (warp * C::ST + fstage) * C::STAGE);
#pragma unroll
        for (int pass = 0; pass < C::RP / C::CP; ++pass) {
            if (pass > 0) __syncthreads();   // the last pass has been read
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int t = 0; t < C::G * 4; ++t) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = T.o[t][n][i];
                        if (MODE == PACK4) v[i] += __shfl_xor_sync(kFull, v[i], 2);
                    }
                    const int col = n * 8 + 2 * j - pass * C::CP;   // the first of this lane's two columns
                    if (col >= 0 && col < C::CP && (MODE != PACK4 || j < 2)) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            *reinterpret_cast<float2 *>(mine + (col + q) * C::RS + t * 16 + r * 2) =
                                make_float2(fmaf(v[q], 64.f, T.z[t / 4][n][q]), fmaf(v[2 + q], 4.f, T.z[t / 4][n][q]));
                    }
                }
            __syncthreads();
            if (pass == 0) {
                // a warp to a column, a lane to a warp's sums
                for (int row = warp; row < C::RP; row += kWarps) {
                    const float c = cols[row * C::CS];
                    const float mw = lane < kWarps ? stat[lane * C::RP + row] : -INFINITY;
                    float m = mw;
#pragma unroll
                    for (int o = 1; o < kWarps; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                    float l = 0.f;
                    if (lane < kWarps) {
                        const float f = exp2f((mw - (m == -INFINITY ? 0.f : m)) * c);
                        stat[lane * C::RP + row] = f;
                        l = f * stat[(kWarps + lane) * C::RP + row];
                    }
#pragma unroll
                    for (int o = 1; o < kWarps; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
                    if (lane == 0) {
                        base[row] = m;
                        sum[row] = cols[row * C::CS + 2] != 0.f ? l : 0.f;   // a row that is not asked for has no sum
                        cc1[row] = c;
                        if (k.a.stat && whole && row < k.rows) put_stat(k, s.b, head, row, m, sum[row], c);
                    }
                }
                __syncthreads();
            }
            for (int i = tid; i < C::CP * D; i += kThreads) {
                const int col = i / D, e = i % D, row = pass * C::CP + col;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    v = fmaf(stat[w * C::RP + row], reinterpret_cast<const float *>(smem + woff[w])[col * C::RS + e], v);
                const int ch = (e >> 6) * 64 + ((e >> 1) & 7) * 8 + ((e >> 4) & 3) * 2 + (e & 1);
                if (!whole) {
                    rec[3 * C::RP + row * D + ch] = v;
                } else if (row < k.rows) {
                    const float l = sum[row];
                    q_store1(k.a.out, out_row[row] + ch, l == 0.f ? 0.f : v / l);
                }
            }
        }
        __syncthreads();   // the stages may be filled again
        if (!whole) {
            if (tid < 3 * C::RP) rec[tid] = base[tid];   // maximum, sum and c1 lie side by side
            if (tid < 2) {
                // by the threads that cleared the entry
                const int p0 = s.first / ax.per;
                k.left[blockIdx.x * 4 + 2 * (s.u0 == 0) + tid] =
                    tid == 0 ? make_int4(s.b, head, s.u0 * C::UT, min(len, s.u1 * C::UT))
                             : make_int4(p0, (s.first + s.nu - 1) / ax.per - p0 + 1, 0, 0);
            }
        } else if (weighing) {
            if (tid < C::RP) {
                base[tid] = base[tid] == -INFINITY ? 0.f : base[tid];
                sum[tid] = sum[tid] == 0.f ? 0.f : 1.f / sum[tid];
            }
            __syncthreads();
            weigh<C::RP, 8, true>(k, lg, len, c.slot0(s.b, head), base, cc1, sum);
        }
        if (last) break;
        s = nx;
        head = nhead;
        turn();
        __syncthreads();
    }
}

// ------------------------------------------------------------ second kernel

// What a CTA of the first kernel left of a head that others have parts of, too.
struct Left {
    int b, head, t0, t1;   // its slots [t0, t1)
    int p0, n;             // the head's n records (0: nothing left) are of CTAs p0, p0 + 1, ...
};

// Finishes the heads that lie in more than one CTA, and writes what no CTA came
// by: zero rows (and decayed weights) of empty sequences and heads not chosen.
// A CTA has up to two heads of one CTA of the first kernel, and a share of each.
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 4) qattn_join_kernel(QAttnK k) {
    using C = Cfg<D, MODE>;
    constexpr int RP = C::RP, REC = C::REC;
    extern __shared__ __align__(16) float factor[];   // [2, grid, RP]
    __shared__ float base[2][RP], inv[2][RP], cc1[2][RP];
    __shared__ float red[kThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x / k.subs, sub = blockIdx.x % k.subs;
    const QCacheK &c = k.a.c;
    pdl_wait();
    pdl_launch_dependents();
    Left s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int4 x = ld_dep(k.left + cta * 4 + 2 * i), y = ld_dep(k.left + cta * 4 + 2 * i + 1);
        s[i] = Left{x.x, x.y, x.z, x.w, y.x, y.y};
    }
    // the heads that no CTA came by, of this CTA's share of all
    const int64_t heads = (int64_t)c.batch * c.heads, each = (heads + gridDim.x - 1) / gridDim.x;
    const int64_t h0 = min(heads, blockIdx.x * each), h1 = min(heads, h0 + each);
    auto idle = [&](int64_t i) {
        const int b = (int)(i / c.heads), n = ld_dep(k.a.length + b);
        return n <= 0 || !kv_on(k, b, (int)(i % c.heads));
    };
    bool some = false;
    for (int64_t i = h0 + tid; i < h1; i += kThreads) some |= idle(i);
    if (__syncthreads_or(some)) {
        for (int64_t i = h0; i < h1; ++i) {
            if (!idle(i)) continue;
            const int b = (int)(i / c.heads), h = (int)(i % c.heads);
            for (int e = tid; e < k.rows * D; e += kThreads) q_store1(k.a.out, out_at(k, b, h, e / D) + e % D, 0.f);
            if (k.a.stat && tid < k.rows) put_stat(k, b, h, tid, -INFINITY, 0.f, 1.f);
            if (k.a.weight)
                for (int e = tid; e < q_length(k.a.length, b, c.cap, nullptr); e += kThreads) {
                    const int64_t slot = c.slot0(b, h) + e;
                    k.a.weight[slot] = k.a.decay == 0.f ? 0.f : k.a.decay * ld_dep(c.weight + slot);
                }
        }
    }
    if (s[0].n == 0 && s[1].n == 0) return;
    auto rec = [&](const Left &x, int p) { return k.part + ((int64_t)(x.p0 + p) * 2 + (p == 0)) * REC; };
    // a warp to a column of a head: its maximum and sum over the n records
    for (int i = warp; i < 2 * RP; i += kWarps) {
        const Left x = i < RP ? s[0] : s[1];
        const int row = i % RP, n = x.n;
        float *f = factor + (int64_t)(i / RP) * k.grid * RP + row;
        if (n == 0) continue;
        const float c1 = ld_dep(rec(x, 0) + 2 * RP + row);
        float m = lane < n ? ld_dep(rec(x, lane) + row) : -INFINITY, l = lane < n ? ld_dep(rec(x, lane) + RP + row) : 0.f;
        const float m0 = m, l0 = l;
        for (int p = lane + 32; p < n; p += 32) m = fmaxf(m, ld_dep(rec(x, p) + row));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        if (m == -INFINITY) m = 0.f;
        const float g0 = exp2f((m0 - m) * c1);
        if (lane < n) f[lane * RP] = g0;
        l = lane < n ? g0 * l0 : 0.f;
        for (int p = lane + 32; p < n; p += 32) {
            const float g = exp2f((ld_dep(rec(x, p) + row) - m) * c1);
            f[p * RP] = g;
            l = fmaf(g, ld_dep(rec(x, p) + RP + row), l);
        }
        l = warp_sum(l);
        if (lane == 0) {
            base[i / RP][row] = m;
            inv[i / RP][row] = l == 0.f ? 0.f : 1.f / l;
            cc1[i / RP][row] = c1;
            // m is 0 for a row that saw nothing, whose l is 0 as well
            if (k.a.stat && row < k.rows && sub == 0) put_stat(k, x.b, x.head, row, l == 0.f ? -INFINITY : m, l, c1);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Left &x = s[i];
        if (x.n == 0) continue;
        const float *f = factor + (int64_t)i * k.grid * RP;
        // this CTA's share of the output values: many records are added up by 8 warps, few by one thread
        const int64_t total = k.rows * D, part = (int64_t)(cta - x.p0) * k.subs + sub, parts = (int64_t)x.n * k.subs;
        const int e0 = (int)(total * part / parts), e1 = (int)(total * (part + 1) / parts);
        if (x.n > kWarps) {
            for (int a = e0; a < e1; a += 32) {
                const int e = a + lane;
                float v = 0.f;
                if (e < e1) {
#pragma unroll 4
                    for (int p = warp; p < x.n; p += kWarps) v = fmaf(f[p * RP + e / D], ld_dep(rec(x, p) + 3 * RP + e), v);
                }
                red[tid] = v;
                __syncthreads();
                if (warp == 0 && e < e1) {
                    v = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v += red[w * 32 + lane];
                    q_store1(k.a.out, out_at(k, x.b, x.head, e / D) + e % D, v * inv[i][e / D]);
                }
                __syncthreads();
            }
        } else {
            for (int e = e0 + tid; e < e1; e += kThreads) {
                float v = 0.f;
#pragma unroll
                for (int p = 0; p < kWarps; ++p)
                    if (p < x.n) v = fmaf(f[p * RP + e / D], ld_dep(rec(x, p) + 3 * RP + e), v);
                q_store1(k.a.out, out_at(k, x.b, x.head, e / D) + e % D, v * inv[i][e / D]);
            }
        }
        if (k.a.weight) {
            const int n = x.t1 - x.t0, a0 = (int)((int64_t)n * sub / k.subs), a1 = (int)((int64_t)n * (sub + 1) / k.subs);
            // behind the units of the CTA's first piece, as they were left
            const int64_t at = i == 0 ? 0 : (s[0].t1 - s[0].t0 + C::UT - 1) / C::UT * C::UT;
            weigh<RP, 4, false>(k, k.logit + cta * k.area + (at + a0) * RP, a1 - a0, c.slot0(x.b, x.head) + x.t0 + a0, base[i],
                                cc1[i], inv[i]);
        }
    }
}

template <int D, int MODE, bool TWO>
cudaError_t run(QAttnK k, int64_t cost, cudaStream_t s) {
    using C = Cfg<D, MODE>;
    const size_t axis = (2 * (size_t)k.a.c.batch + 1) * sizeof(int), smem = C::smem_fixed + axis;
    static_assert(C::smem_fixed + (2 * kQMaxBatch + 1) * 4 <= 226 * 1024, "shared memory of one CTA");
    // 228 KB per SM, of which 1 KB per CTA and its static variables are spoken for
    const int fit = (int)(228 * 1024 / (smem + 2048));
    k.grid = qattn_grid(cost, (int64_t)(k.a.sms > 0 ? k.a.sms : 1) * (fit < C::MINB ? fit : C::MINB));
    k.area = qattn_area(cost, k.grid, (k.a.c.cap + C::UT - 1) / C::UT) * C::UT * C::RP;
    const size_t join = 2 * (size_t)k.grid * C::RP * sizeof(float);
    k.subs = 2;   // one wave of four per SM (64 ragged sequences of up to 8,192 slots: 108, 101, 104 us with 1, 2, 3)
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(&qattn_kernel<D, MODE, TWO>));
    if (e == cudaSuccess && join > 48 * 1024) e = allow_smem(reinterpret_cast<const void *>(&qattn_join_kernel<D, MODE>));
    if (e == cudaSuccess) e = launch(qattn_kernel<D, MODE, TWO>, dim3(k.grid), dim3(kThreads), smem, s, pdl_enabled(), k);
    if (e == cudaSuccess) e = launch(qattn_join_kernel<D, MODE>, dim3(k.grid * k.subs), dim3(kThreads), join, s, pdl_enabled(), k);
    return e;
}

}  // namespace

template <int D>
cudaError_t run_qattn(QAttnK k, int mode, int64_t cost, cudaStream_t s) {
    // with one CTA per SM, the longest piece of a head that a CTA can have
    constexpr int UT = Cfg<D, TWO8>::UT;
    const int64_t head = (k.a.c.cap + UT - 1) / UT, part = cost / (k.a.sms > 0 ? k.a.sms : 1), piece = part < head ? part : head;
    const bool two = k.a.q.dt == CS_F32 || piece * UT > kChain;
    if (mode == PACK4) return two ? run<D, PACK4, true>(k, cost, s) : run<D, PACK4, false>(k, cost, s);
    if (mode == ONE8) return two ? run<D, ONE8, true>(k, cost, s) : run<D, ONE8, false>(k, cost, s);
    return two ? run<D, TWO8, true>(k, cost, s) : run<D, TWO8, false>(k, cost, s);
}

#endif  // CS_QATTN_KERNELS

}  // namespace cs
