// Attention over the 4-bit KV cache.
//
// Per query row r (a query head of a cache head's group, at one query token):
//     x_i = scale log2(e) q_r . k_i,   p_i = 2^(x_i - m),   out = sum p_i v_i / sum p_i.
// With k = z + s n and v = z + s n per group of 64 channels (n = 0 .. 15):
//     q . k = sum_g s_g (q . n)_g + z_g (sum q)_g
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
// finishes (with the same split, every CTA a share of the record sums).
//
// Products.  mma.sync m16n8k16 in fp16 with fp32 sums: the query rows are the
// 8 columns, so a batch-1 head wastes little, and the codes are the A operand
// straight from their packed words.  For the keys, 16 slots x 16 channels: a
// nibble ANDed out of a word is an fp16 subnormal n 2^-24 (or, four bits up,
// n 2^-20), exact in the product; the factor 16 goes into q.  For the values, 16
// channels x 16 slots: two slots' words are interleaved by byte permutes, n is
// ORed into 1024 + n and 1032 subtracted.  The tensor memory path of the newer
// matrix instructions needs 128 rows and operands in shared memory; with at
// most 16 query rows per head the products are not what bounds this kernel.
//
// Precision.  q is scaled by a power of two and split into two fp16 parts
// (22 bits; the second is zero for 16-bit inputs), p s likewise (scaled so that
// the largest stays below 2^15).  With at most 4 rows the two parts sit in the
// same 8 columns.  All sums and the softmax statistics are fp32.
#include "cs_qcache.cuh"

namespace cs {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct QAttnK {
    QAttnArgs a;
    int group, rows;     // query heads per cache head; rows of this pass
    int row0;            // its first row: row r is head r % group of the group, token r / group
    int grid;            // CTAs of both kernels
    float *part;         // [grid, 2, RP * (D + 2)]: per column m and sum, then the sums of p v
    float *logit;        // [grid, 2, per, UT, RP] x, for the weights
    int64_t area;        // floats of one CTA's half of logit
    float c2;            // scale log2(e)
};

// Query columns per pass and how they sit in the 8 columns of a product.
enum Mode { PACK4 = 0, ONE8 = 1, TWO8 = 2 };

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
    static constexpr int MINB = D * NT <= 128 ? 2 : 1;       // CTAs per SM
    static constexpr int ST = D == 64 ? 4 : MINB == 2 ? 2 : 3;
    static constexpr int RS = D + 4;                         // floats of a joined column (conflict-free)
    static constexpr int QF = NT * PARTS * (D / 32) * 2 * 32;    // uint2 fragments of q
    static constexpr int RED = kWarps * 4 * RS;              // floats: four columns of every warp
    static constexpr int COLS = RP * (3 + G);                // floats: per column c1, last position, on, sums of q
    static constexpr int STAT = kWarps * RP * 2 + 2 * RP;    // floats: the warps' m and l, then the joined ones
    static constexpr size_t smem_fixed = (size_t)kWarps * ST * STAGE + QF * 8 + (RED + COLS + STAT) * 4;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
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
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Where a 16-byte chunk of a unit's row lies: chunks are permuted so that eight
// slots' same chunk, and four slots' same pair of chunks, lie in different banks.
template <int D>
__device__ __forceinline__ int swizzle(int tok) {
    if (D == 128) return ((tok >> 1) & 1) * 2 + ((tok >> 2) & 1);
    if (D == 256) return ((tok & 3) << 1) | ((tok >> 2) & 1);
    return (tok >> 2) & 1;
}
// The slot within 16 that is row i of a product: with this order both the keys'
// rows and the values' columns of a warp are read without bank conflicts.
__device__ __forceinline__ int slot_of_row(int i) { return (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3); }

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

// In shared memory per sequence: its length, and the units before it (one more at the end).
struct Axis {
    int *len, *pre;
    int per;          // units of a CTA
    int begin, end;   // this CTA's

    template <int UT>
    __device__ void build(const QAttnK &k, int *smem, int *wsum, bool flag) {
        len = smem;
        pre = smem + k.a.c.batch;
        const int B = k.a.c.batch, each = (B + kThreads - 1) / kThreads;
        const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = q_length(k.a.length, b, k.a.c.cap, flag ? k.a.err : nullptr);
            int heads = k.a.c.heads;
            if (k.a.mask) {
                heads = 0;
                for (int h = 0; h < k.a.c.heads; ++h) heads += kv_on(k, b, h);
            }
            len[b] = n;
            const int units = (n + UT - 1) / UT * heads;
            pre[b] = units;   // not yet summed
            sum += units;
        }
        int total;
        int at = block_excl_scan(sum, wsum, &total);
        for (int b = b0; b < b1; ++b) {
            const int units = pre[b];
            pre[b] = at;
            at += units;
        }
        if (threadIdx.x == 0) pre[B] = total;
        __syncthreads();
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
    int at;           // u0 on the split axis

    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == nu; }
    template <int UT>
    __device__ __forceinline__ void seek(const Axis &x, int unit, int from_b) {
        b = from_b;
        while (x.pre[b + 1] <= unit) ++b;
        nu = (x.len[b] + UT - 1) / UT;
        const int rel = unit - x.pre[b];
        h = rel / nu;
        u0 = rel - h * nu;
        u1 = min(nu, u0 + x.end - unit);
        at = unit;
    }
};

__device__ __forceinline__ int first_seq(const Axis &x, int B, int unit) {
    int lo = 0, hi = B;   // the last b with pre[b] <= unit; empty ones before it are passed over by seek
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (x.pre[mid] <= unit) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The cache head that is the sequence's n-th chosen one.
__device__ __forceinline__ int chosen_head(const QAttnK &k, int b, int n) {
    if (!k.a.mask) return n;
    int h = 0;
    for (; h < k.a.c.heads - 1; ++h)
        if (kv_on(k, b, h) && n-- == 0) break;
    return h;
}

// ------------------------------------------------------------- first kernel

template <int D, int MODE>
struct Tile {
    using C = Cfg<D, MODE>;
    float o[C::G * 4][C::NT][4];     // channels 8 (lane / 4) + 2 t (+ 1) of group g in o[4 g + t], columns 2 (lane % 4) (+ 1)
    float z[C::G][C::NT][2];         // sums of p (z + 8 s), this lane's slots
    float m[C::NT][2], l[C::NT][2];
    int e;                           // exponent field of the largest value scale so far

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
#pragma unroll
            for (int t = 0; t < C::G * 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][n][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = -INFINITY;
                l[n][i] = 0.f;
#pragma unroll
                for (int g = 0; g < C::G; ++g) z[g][n][i] = 0.f;
            }
        }
        e = 1;
    }
};

// Starts the copies of one unit of a head into a stage of the warp's ring.
template <int D, int MODE>
__device__ __forceinline__ void fetch(const QAttnK &k, uint32_t stage, int64_t slot0, int n) {
    using C = Cfg<D, MODE>;
    constexpr int CH = C::RB / 16;
    const int lane = threadIdx.x & 31;
    const QCacheK &c = k.a.c;
    const uint8_t *kp = c.k + slot0 * C::RB, *vp = c.v + slot0 * C::RB;
#pragma unroll
    for (int i0 = 0; i0 < C::UT * CH; i0 += 32) {
        const int i = i0 + lane, tok = i / CH, ch = i % CH;
        const uint32_t at = stage + tok * C::RB + ((ch ^ swizzle<D>(tok)) << 4);
        const bool on = tok < n;
        const int off = on ? i * 16 : 0;
        cp16(at, kp + off, on);
        cp16(at + C::UT * C::RB, vp + off, on);
    }
    const uint32_t *ks = c.ks + slot0 * C::G, *vs = c.vs + slot0 * C::G;
    const uint32_t sc = stage + 2 * C::UT * C::RB;
#pragma unroll
    for (int i0 = 0; i0 < C::UT * C::G; i0 += 32) {
        const int i = i0 + lane;
        if (C::UT * C::G % 32 == 0 || i < C::UT * C::G) {
            const bool on = i < n * C::G;
            const int off = on ? i : 0;
            cp4(sc + i * 4, ks + off, on);
            cp4(sc + C::UT * C::G * 4 + i * 4, vs + off, on);
        }
    }
    if (k.a.q_pos && lane < C::UT) cp4(sc + C::UT * C::G * 8 + lane * 4, c.pos + slot0 + (lane < n ? lane : 0), lane < n);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, Cfg<D, MODE>::MINB) qattn_kernel(QAttnK k) {
    using C = Cfg<D, MODE>;
    extern __shared__ __align__(16) char smem[];
    uint2 *qf = reinterpret_cast<uint2 *>(smem + (size_t)kWarps * C::ST * C::STAGE);
    float *red = reinterpret_cast<float *>(qf + C::QF);
    float *cols = red + C::RED;
    float *stat = cols + C::COLS;
    int *axis_mem = reinterpret_cast<int *>(stat + C::STAT);
    __shared__ int wsum[32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, j = lane & 3;
    const QCacheK &c = k.a.c;
    pdl_wait();
    pdl_launch_dependents();
    Axis ax{};
    ax.build<C::UT>(k, axis_mem, wsum, blockIdx.x == 0);
    if (ax.begin >= ax.end) return;

    const uint32_t ring = smem_addr(smem) + warp * C::ST * C::STAGE;
    const bool by_pos = k.a.q_pos != nullptr, weigh = k.a.weight != nullptr;

    // the fetching side runs ahead of the computing side, on across heads
    Seg f{};
    f.template seek<C::UT>(ax, ax.begin, first_seq(ax, c.batch, ax.begin));
    int fu = f.u0 + warp, fstage = 0;
    int fhead = chosen_head(k, f.b, f.h);
    bool more = true;
    auto fetch_next = [&]() {
        while (more && fu >= f.u1) {
            const int next = f.at + f.u1 - f.u0;
            if (next >= ax.end) {
                more = false;
            } else {
                f.template seek<C::UT>(ax, next, f.b);
                fu = f.u0 + warp;
                fhead = chosen_head(k, f.b, f.h);
            }
        }
        if (more) {
            fetch<D, MODE>(k, ring + fstage * C::STAGE, c.slot0(f.b, fhead) + (int64_t)fu * C::UT, ax.len[f.b] - fu * C::UT);
            fu += kWarps;
        }
        fstage = fstage + 1 == C::ST ? 0 : fstage + 1;
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < C::ST - 1; ++i) fetch_next();

    int stage = 0;
    Seg s{};
    s.template seek<C::UT>(ax, ax.begin, first_seq(ax, c.batch, ax.begin));
    Tile<D, MODE> T;
    for (;;) {
        const int head = chosen_head(k, s.b, s.h);
        // ---- this head's query rows as fragments, a warp to a row
        {
            __half *qh = reinterpret_cast<__half *>(qf);
            for (int row = warp; row < C::RP; row += kWarps) {
                const bool on = row_on(k, s.b, head, row);
                const int t = (k.row0 + row) / k.group;
                const int64_t src = s.b * k.a.q.ldb + t * k.a.q.ldt + (int64_t)(head * k.group + (k.row0 + row) % k.group) * k.a.q.ldh;
                float q[D / 32];
                float big = 0.f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    q[i] = on ? q_load1(k.a.q, src + i * 32 + lane) : 0.f;
                    big = fmaxf(big, fabsf(q[i]));
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
                // the power of two that takes the largest to [2^14, 2^15); infinities stay what they are
                const int eb = (int)(__float_as_uint(big) >> 23);
                const int up = big > 0.f && eb < 255 ? min(141 - eb, 127) : 0;
                const float f1 = __uint_as_float((uint32_t)(127 + up / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int jj = lane >> 3, nib = lane & 7;
                    const float v = q[i] * f1 * f2 * (nib & 1 ? 0.0625f : 1.f);
                    const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
                    const int col = row & 7, nt = row >> 3;
                    auto put = [&](int tile, int cc, __half h) {
                        qh[(((tile * (D / 32) + i) * 2 + ((nib & 3) >> 1)) * 32 + cc * 4 + jj) * 4 + (nib & 1) * 2 + (nib >> 2)] = h;
                    };
                    put(nt * C::PARTS, col, hi);
                    if (C::PARTS == 1) put(0, col + 4, lo);
                    else put(nt * 2 + 1, col, lo);
                }
                float sum[C::G];
#pragma unroll
                for (int g = 0; g < C::G; ++g) sum[g] = warp_sum(q[2 * g] + q[2 * g + 1]);
                if (lane == 0) {
                    float *cc = cols + row * (3 + C::G);
                    cc[0] = k.c2 * exp2f((float)-up);
                    cc[1] = __int_as_float(by_pos ? ld_dep(k.a.q_pos + s.b) + t : INT_MAX);
                    cc[2] = __int_as_float(on ? 1 : 0);
#pragma unroll
                    for (int g = 0; g < C::G; ++g) cc[3 + g] = k.c2 * sum[g];
                }
            }
        }
        __syncthreads();
        const bool two = C::PARTS == 2 && k.a.q.dt == CS_F32;
        float c1[C::NT][2], zq[C::NT][2][C::G];
        int last[C::NT][2], newest = INT_MIN;
        bool on[C::NT][2];
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = MODE == PACK4 ? (j & 1) * 2 + i : n * 8 + j * 2 + i;
                const float *cc = cols + col * (3 + C::G);
                c1[n][i] = cc[0];
                last[n][i] = __float_as_int(cc[1]);
                on[n][i] = __float_as_int(cc[2]) != 0;
#pragma unroll
                for (int g = 0; g < C::G; ++g) zq[n][i][g] = MODE == PACK4 && j >= 2 ? 0.f : cc[3 + g];
            }
        if (by_pos) newest = ld_dep(k.a.q_pos + s.b) + (k.row0 + k.rows - 1) / k.group;
        T.clear();
        const int len = ax.len[s.b];
        float *lg = k.logit + ((int64_t)blockIdx.x * 2 + (s.u0 == 0)) * k.area;

        for (int u = s.u0 + warp; u < s.u1; u += kWarps) {
            __syncwarp();
            fetch_next();
            cp_async_wait<C::ST - 1>();
            __syncwarp();
            const uint32_t kb = ring + stage * C::STAGE, vb = kb + C::UT * C::RB, sb = vb + C::UT * C::RB;
            stage = stage + 1 == C::ST ? 0 : stage + 1;

            // ---- x = c1 sum_g s_g (q . n)_g + sum_g z_g zq_g
            float x[C::SUB][C::NT][4];
#pragma unroll
            for (int g = 0; g < C::G; ++g) {
                float acc[C::SUB][C::NT][4];
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                    for (int n = 0; n < C::NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[sub][n][i] = 0.f;
#pragma unroll
                for (int w = 2 * g; w < 2 * g + 2; ++w) {
                    uint32_t kw[C::SUB][2];
#pragma unroll
                    for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int tok = sub * 16 + slot_of_row(r + 8 * i);
                            kw[sub][i] = lds32(kb + tok * C::RB + ((w ^ swizzle<D>(tok)) << 4) + j * 4);
                        }
#pragma unroll
                    for (int step = 0; step < 2; ++step) {
                        uint32_t a[C::SUB][4];
#pragma unroll
                        for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t v = step ? kw[sub][i] >> 8 : kw[sub][i];
                                a[sub][i] = v & 0x000f000fu;
                                a[sub][i + 2] = v & 0x00f000f0u;
                            }
#pragma unroll
                        for (int n = 0; n < C::NT; ++n) {
                            const uint32_t qa = smem_addr(qf) + ((((n * C::PARTS) * (D / 32) + w) * 2 + step) * 32 + lane) * 8;
                            const uint2 b = lds64(qa);
#pragma unroll
                            for (int sub = 0; sub < C::SUB; ++sub) mma16816(acc[sub][n], a[sub], b.x, b.y);
                            if (two) {
                                const uint2 b2 = lds64(qa + (D / 32) * 2 * 32 * 8);
#pragma unroll
                                for (int sub = 0; sub < C::SUB; ++sub) mma16816(acc[sub][n], a[sub], b2.x, b2.y);
                            }
                        }
                    }
                }
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float sc, zo;
                        half2x(lds32(sb + ((sub * 16 + slot_of_row(r + 8 * i)) * C::G + g) * 4), sc, zo);
                        sc *= 16777216.f;   // n was 2^-24 n
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const float v = fmaf(acc[sub][n][2 * i + q] * sc, c1[n][q], zo * zq[n][q][g]);
                                x[sub][n][2 * i + q] = g == 0 ? v : x[sub][n][2 * i + q] + v;
                            }
                    }
            }
            // ---- what is not seen is -inf; the first part of each value scale
            uint32_t vs[C::SUB][2][C::G];
            uint32_t top = 0;
            bool grow = false;
#pragma unroll
            for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = sub * 16 + slot_of_row(r + 8 * i);
                    int p = 0;
                    bool there = u * C::UT + tok < len;
                    if (by_pos) {
                        p = (int)lds32(sb + C::UT * C::G * 8 + tok * 4);
                        there = there && p >= 0 && p <= newest;
                    }
#pragma unroll
                    for (int g = 0; g < C::G; ++g) {
                        const uint32_t v = lds32(sb + C::UT * C::G * 4 + (tok * C::G + g) * 4);
                        vs[sub][i][g] = there ? v : 0u;
                        top = max(top, vs[sub][i][g] & 0x7fffu);
                    }
#pragma unroll
                    for (int n = 0; n < C::NT; ++n)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float &v = x[sub][n][2 * i + q];
                            if (MODE == PACK4) v += __shfl_xor_sync(kFull, v, 2);
                            if (!there || !on[n][q] || p > last[n][q]) v = -INFINITY;
                            grow |= v > T.m[n][q];
                        }
                    if (weigh && there && (MODE != PACK4 || j < 2)) {
                        const int64_t at = (int64_t)(u - s.u0) * C::UT + tok;
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
                            *reinterpret_cast<float2 *>(lg + at * C::RP + n * 8 + 2 * j) =
                                make_float2(x[sub][n][2 * i], x[sub][n][2 * i + 1]);
                    } else if (weigh && u * C::UT + tok < len && (MODE != PACK4 || j < 2)) {
                        const int64_t at = (int64_t)(u - s.u0) * C::UT + tok;
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
                            *reinterpret_cast<float2 *>(lg + at * C::RP + n * 8 + 2 * j) = make_float2(-INFINITY, -INFINITY);
                    }
                }
            const int e = max((int)(__reduce_max_sync(kFull, top) >> 10), 1);
            if (__any_sync(kFull, grow) || e > T.e) {
                const int en = max(e, T.e);
                const float fe = __uint_as_float((uint32_t)(127 + T.e - en) << 23);
                T.e = en;
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float m = T.m[n][q];
#pragma unroll
                        for (int sub = 0; sub < C::SUB; ++sub) m = fmaxf(m, fmaxf(x[sub][n][q], x[sub][n][2 + q]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                        const float al = m > T.m[n][q] ? exp2_approx(T.m[n][q] - m) : 1.f;
                        T.m[n][q] = m;
                        T.l[n][q] *= al;
#pragma unroll
                        for (int g = 0; g < C::G; ++g) T.z[g][n][q] *= al;
#pragma unroll
                        for (int t = 0; t < C::G * 4; ++t) {
                            T.o[t][n][q] *= al * fe;
                            T.o[t][n][2 + q] *= al * fe;
                        }
                    }
            }
            // ---- p, its sums, and p s as fragments
            const float up = __uint_as_float((uint32_t)(127 + 29 - T.e) << 23);
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float m = T.m[n][q] == -INFINITY ? 0.f : T.m[n][q];
#pragma unroll
                    for (int sub = 0; sub < C::SUB; ++sub)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &v = x[sub][n][2 * i + q];
                            v = exp2_approx(v - m);
                            T.l[n][q] += v;
                        }
                }
#pragma unroll
            for (int g = 0; g < C::G; ++g)
#pragma unroll
                for (int sub = 0; sub < C::SUB; ++sub) {
                    uint32_t ph[C::NT][2], pl[C::NT][2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float sc, zo;
                        half2x(vs[sub][i][g], sc, zo);
                        zo = fmaf(8.f, sc, zo);
                        sc *= up;
#pragma unroll
                        for (int n = 0; n < C::NT; ++n) {
                            const float p0 = x[sub][n][2 * i], p1 = x[sub][n][2 * i + 1];
                            T.z[g][n][0] = fmaf(p0, zo, T.z[g][n][0]);
                            T.z[g][n][1] = fmaf(p1, zo, T.z[g][n][1]);
                            const float a0 = p0 * sc, a1 = p1 * sc;
                            uint32_t h = pack_h2(a0, a1);
                            float h0, h1;
                            half2x(h, h0, h1);
                            const uint32_t lo = pack_h2(a0 - h0, a1 - h1);
                            if (MODE == PACK4) {
                                ph[n][i] = transpose8x8(j >= 2 ? lo : h);
                            } else {
                                ph[n][i] = transpose8x8(h);
                                pl[n][i] = transpose8x8(lo);
                            }
                        }
                    }
                    // the values' words: rows of a product are channels, its columns the slots' order of the keys' rows
                    uint32_t vw[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = sub * 16 + slot_of_row(2 * j + (i & 1) + 8 * (i >> 1));
                        vw[i] = lds32(vb + tok * C::RB + (((2 * g + (r >> 2)) ^ swizzle<D>(tok)) << 4) + (r & 3) * 4);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t a = __byte_perm(vw[0], vw[1], half ? 0x7632 : 0x5410);
                        const uint32_t b = __byte_perm(vw[2], vw[3], half ? 0x7632 : 0x5410);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const uint32_t av = t ? a >> 8 : a, bv = t ? b >> 8 : b;
                            uint32_t fr[4];
                            fr[0] = hsub2u(and_or(av, 0x000f000fu, 0x64006400u), 0x64086408u);
                            fr[1] = hsub2u(and_or(av, 0x00f000f0u, 0x64006400u), 0x64806480u);
                            fr[2] = hsub2u(and_or(bv, 0x000f000fu, 0x64006400u), 0x64086408u);
                            fr[3] = hsub2u(and_or(bv, 0x00f000f0u, 0x64006400u), 0x64806480u);
#pragma unroll
                            for (int n = 0; n < C::NT; ++n) {
                                mma16816(T.o[g * 4 + half * 2 + t][n], fr, ph[n][0], ph[n][1]);
                                if (MODE != PACK4) mma16816(T.o[g * 4 + half * 2 + t][n], fr, pl[n][0], pl[n][1]);
                            }
                        }
                    }
                }
        }

        // ---- the warps' sums become one
        const bool lanes = MODE != PACK4 || j < 2;
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
                if (r == 0 && lanes) {
                    stat[warp * C::RP + n * 8 + 2 * j + q] = T.m[n][q];
                    stat[(kWarps + warp) * C::RP + n * 8 + 2 * j + q] = T.l[n][q];
                }
            }
        __syncthreads();
        float *mj = stat + 2 * kWarps * C::RP, *lj = mj + C::RP;
        if (tid < C::RP) {
            float m = -INFINITY, l = 0.f;
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stat[w * C::RP + tid]);
            const float base = m == -INFINITY ? 0.f : m;
            for (int w = 0; w < kWarps; ++w) {
                float &mw = stat[w * C::RP + tid];
                mw = exp2f(mw - base);
                l = fmaf(mw, stat[(kWarps + w) * C::RP + tid], l);
            }
            mj[tid] = m;
            lj[tid] = l;
        }
        const bool whole = s.whole();
        float *rec = k.part + ((int64_t)blockIdx.x * 2 + (s.u0 == 0)) * (C::RP * (D + 2));
        const float down = __uint_as_float((uint32_t)(127 + T.e - 29) << 23);
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
#pragma unroll
            for (int hf = 0; hf < (MODE == PACK4 ? 1 : 2); ++hf) {   // columns 4 hf .. 4 hf + 3 of the tile
                float *mine = red + warp * 4 * C::RS;
#pragma unroll
                for (int t = 0; t < C::G * 4; ++t) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = T.o[t][n][i];
                        if (MODE == PACK4) v[i] += __shfl_xor_sync(kFull, v[i], 2);
                    }
                    if (j >> 1 == hf) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            *reinterpret_cast<float2 *>(mine + (2 * (j & 1) + q) * C::RS + t * 16 + r * 2) =
                                make_float2(fmaf(v[q], down, T.z[t / 4][n][q]), fmaf(v[2 + q], down * 0.0625f, T.z[t / 4][n][q]));
                    }
                }
                __syncthreads();
                for (int i = tid; i < 4 * D; i += kThreads) {
                    const int col = i / D, e = i % D, row = n * 8 + hf * 4 + col;
                    float v = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v = fmaf(stat[w * C::RP + row], red[(w * 4 + col) * C::RS + e], v);
                    const int ch = (e >> 6) * 64 + ((e >> 1) & 7) * 8 + ((e >> 4) & 3) * 2 + (e & 1);
                    if (!whole) {
                        rec[2 * C::RP + row * D + ch] = v;
                    } else if (row < k.rows) {
                        const float l = lj[row];
                        const int rr = k.row0 + row;
                        q_store1(k.a.out, s.b * k.a.out.ldb + rr / k.group * k.a.out.ldt + (int64_t)(head * k.group + rr % k.group) * k.a.out.ldh + ch,
                                 l == 0.f ? 0.f : v / l);
                    }
                }
                __syncthreads();
            }
        }
        if (!whole) {
            if (tid < C::RP) {
                rec[tid] = mj[tid];
                rec[C::RP + tid] = lj[tid];
            }
        } else if (weigh) {
            // every slot's share, from the x that the warps left behind
            const int64_t slot0 = c.slot0(s.b, head);
            for (int i = tid; i < len; i += kThreads) {
                float w = 0.f;
#pragma unroll
                for (int q = 0; q < C::RP; ++q)
                    if (lj[q] != 0.f) w += exp2_approx(lg[(int64_t)i * C::RP + q] - (mj[q] == -INFINITY ? 0.f : mj[q])) / lj[q];
                const float old = k.a.decay == 0.f ? 0.f : k.a.decay * ld_dep(c.weight + slot0 + i);
                k.a.weight[slot0 + i] = old + w;
            }
        }
        const int next = s.at + s.u1 - s.u0;
        if (next >= ax.end) break;
        s.template seek<C::UT>(ax, next, s.b);
        __syncthreads();
    }
}

// ------------------------------------------------------------ second kernel

// Finishes the heads that lie in more than one CTA, and writes what no CTA came
// by: zero rows (and decayed weights) of empty sequences and heads not chosen.
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads) qattn_join_kernel(QAttnK k) {
    using C = Cfg<D, MODE>;
    extern __shared__ __align__(16) int axis_mem[];
    __shared__ int wsum[32];
    __shared__ float mj[C::RP], lj[C::RP];
    constexpr int REC = C::RP * (D + 2);
    const int tid = threadIdx.x;
    const QCacheK &c = k.a.c;
    pdl_wait();
    pdl_launch_dependents();
    Axis ax{};
    ax.build<C::UT>(k, axis_mem, wsum, false);
    auto out_at = [&](int b, int head, int row) {
        const int rr = k.row0 + row;
        return b * k.a.out.ldb + rr / k.group * k.a.out.ldt + (int64_t)(head * k.group + rr % k.group) * k.a.out.ldh;
    };
    if (ax.begin < ax.end) {
        Seg s{};
        s.template seek<C::UT>(ax, ax.begin, first_seq(ax, c.batch, ax.begin));
        for (;;) {
            const int next = s.at + s.u1 - s.u0;
            if (!s.whole()) {
                const int head = chosen_head(k, s.b, s.h);
                const int start = s.at - s.u0;                    // the head's first unit on the axis
                const int c0 = start / ax.per, c1 = (start + s.nu - 1) / ax.per, n = c1 - c0 + 1;
                auto rec = [&](int i) { return k.part + ((int64_t)(c0 + i) * 2 + (i == 0)) * REC; };
                // a warp to a column: its maximum and sum over the n records
                for (int row = tid >> 5; row < C::RP; row += kWarps) {
                    float m = -INFINITY, l = 0.f;
                    for (int i = tid & 31; i < n; i += 32) m = fmaxf(m, ld_dep(rec(i) + row));
#pragma unroll
                    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                    if (m == -INFINITY) m = 0.f;
                    for (int i = tid & 31; i < n; i += 32) l = fmaf(exp2f(ld_dep(rec(i) + row) - m), ld_dep(rec(i) + C::RP + row), l);
                    l = warp_sum(l);
                    if ((tid & 31) == 0) {
                        mj[row] = m;
                        lj[row] = l;
                    }
                }
                __syncthreads();
                // this CTA's share of the output values
                const int mine = blockIdx.x - c0, total = k.rows * D;
                const int e0 = (int)((int64_t)total * mine / n), e1 = (int)((int64_t)total * (mine + 1) / n);
                for (int i = e0 + tid; i < e1; i += kThreads) {
                    const int row = i / D;
                    float v = 0.f;
#pragma unroll 4
                    for (int p = 0; p < n; ++p) v = fmaf(exp2f(ld_dep(rec(p) + row) - mj[row]), ld_dep(rec(p) + 2 * C::RP + i), v);
                    q_store1(k.a.out, out_at(s.b, head, row) + i % D, lj[row] == 0.f ? 0.f : v / lj[row]);
                }
                if (k.a.weight) {
                    const float *lg = k.logit + ((int64_t)blockIdx.x * 2 + (s.u0 == 0)) * k.area;
                    const int t0 = s.u0 * C::UT, t1 = min(ax.len[s.b], s.u1 * C::UT);
                    const int64_t slot0 = c.slot0(s.b, head);
                    for (int i = t0 + tid; i < t1; i += kThreads) {
                        float w = 0.f;
#pragma unroll
                        for (int q = 0; q < C::RP; ++q)
                            if (lj[q] != 0.f) w += exp2_approx(ld_dep(lg + (int64_t)(i - t0) * C::RP + q) - mj[q]) / lj[q];
                        const float old = k.a.decay == 0.f ? 0.f : k.a.decay * ld_dep(c.weight + slot0 + i);
                        k.a.weight[slot0 + i] = old + w;
                    }
                }
                __syncthreads();
            }
            if (next >= ax.end) break;
            s.template seek<C::UT>(ax, next, s.b);
        }
    }
    for (int64_t i = blockIdx.x; i < (int64_t)c.batch * c.heads; i += gridDim.x) {
        const int b = (int)(i / c.heads), h = (int)(i % c.heads);
        if (ax.len[b] > 0 && kv_on(k, b, h)) continue;
        for (int e = tid; e < k.rows * D; e += kThreads) q_store1(k.a.out, out_at(b, h, e / D) + e % D, 0.f);
        if (k.a.weight)
            for (int e = tid; e < ax.len[b]; e += kThreads) {
                const int64_t slot = c.slot0(b, h) + e;
                k.a.weight[slot] = k.a.decay == 0.f ? 0.f : k.a.decay * ld_dep(c.weight + slot);
            }
    }
}

// ----------------------------------------------------------------- host side

int mode_of(int rows) { return rows <= 4 ? PACK4 : rows <= 8 ? ONE8 : TWO8; }
int cols_of(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }
int unit_of(int d) { return d <= 128 ? 32 : 16; }

// The CTAs of a call (two per SM at most) and the most units that one may take.
void split(int batch, int kv_heads, int cap, int d, int sms, int *grid, int64_t *per) {
    const int64_t units = (int64_t)batch * kv_heads * ((cap + unit_of(d) - 1) / unit_of(d));
    const int64_t most = (units + kWarps - 1) / kWarps, ctas = 2 * (int64_t)(sms > 0 ? sms : 1);
    *grid = (int)(most < ctas ? most : ctas);
    *per = (units + *grid - 1) / *grid;
    if (*per < kWarps) *per = kWarps;
}

// Floats of a CTA's half of the logits: no more than its units, or a whole head.
int64_t area_floats(int batch, int kv_heads, int cap, int d, int rows, int sms) {
    int grid;
    int64_t per;
    split(batch, kv_heads, cap, d, sms, &grid, &per);
    // fewer CTAs per SM may run than `split` counts: then each takes more
    const int64_t own = 2 * per, head = (cap + unit_of(d) - 1) / unit_of(d);
    return (own < head ? own : head) * unit_of(d) * cols_of(rows);
}

template <int D, int MODE>
cudaError_t run(QAttnK k, int64_t units, cudaStream_t s) {
    using C = Cfg<D, MODE>;
    const size_t axis = (2 * (size_t)k.a.c.batch + 1) * sizeof(int), smem = C::smem_fixed + axis;
    static_assert(C::smem_fixed + (2 * kQMaxBatch + 1) * 4 <= 227 * 1024, "shared memory of one CTA");
    int64_t grid = (int64_t)k.a.sms * (smem * C::MINB <= 226 * 1024 ? C::MINB : 1);
    if (grid < 1) grid = 1;
    const int64_t most = (units + kWarps - 1) / kWarps;
    k.grid = (int)(most < grid ? most : grid);
    cudaError_t e = cudaFuncSetAttribute(qattn_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch(qattn_kernel<D, MODE>, dim3(k.grid), dim3(kThreads), smem, s, pdl_enabled(), k);
    if (e == cudaSuccess) e = launch(qattn_join_kernel<D, MODE>, dim3(k.grid), dim3(kThreads), axis, s, pdl_enabled(), k);
    return e;
}

template <int D>
cudaError_t run_mode(const QAttnK &k, int64_t units, cudaStream_t s) {
    switch (mode_of(k.rows)) {
    case PACK4: return run<D, PACK4>(k, units, s);
    case ONE8: return run<D, ONE8>(k, units, s);
    default: return run<D, TWO8>(k, units, s);
    }
}

size_t part_bytes(int d, int rows, int sms) {
    return align256((size_t)2 * (sms > 0 ? sms : 1) * 2 * cols_of(rows) * (d + 2) * sizeof(float));
}

}  // namespace

size_t qattn_scratch(int batch, int kv_heads, int cap, int d, int heads, int n_q, int sms) {
    const int rows = heads / kv_heads * n_q;
    return part_bytes(d, rows, sms) +
           align256((size_t)2 * (sms > 0 ? sms : 1) * 2 * area_floats(batch, kv_heads, cap, d, rows, sms) * sizeof(float));
}

cudaError_t launch_qattn(const QAttnArgs &a, cudaStream_t s) {
    QAttnK k{a, a.heads / a.c.heads, 0, 0, 0, nullptr, nullptr, 0, a.scale * 1.44269504088896341f};
    const int rows = k.group * a.n_q;
    k.part = reinterpret_cast<float *>(a.scratch);
    k.logit = reinterpret_cast<float *>(a.scratch + part_bytes(a.c.d, rows, a.sms));
    const int64_t units = (int64_t)a.c.batch * a.c.heads * ((a.c.cap + unit_of(a.c.d) - 1) / unit_of(a.c.d));
    // up to 16 rows in a pass; a later pass adds its weights to an earlier one's
    for (k.row0 = 0; k.row0 < rows; k.row0 += 16) {
        k.rows = rows - k.row0 < 16 ? rows - k.row0 : 16;
        k.area = area_floats(a.c.batch, a.c.heads, a.c.cap, a.c.d, k.rows, a.sms);
        if (k.row0 > 0 && a.weight) {
            k.a.decay = 1.f;
            k.a.c.weight = a.weight;
        }
        const cudaError_t e = a.c.d == 64    ? run_mode<64>(k, units, s)
                              : a.c.d == 128 ? run_mode<128>(k, units, s)
                              : a.c.d == 192 ? run_mode<192>(k, units, s)
                                             : run_mode<256>(k, units, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace cs
