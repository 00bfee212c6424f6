// Attention of many query rows over one head's keys and values on the tensor
// cores: what the packed prompts (cs_prompt.cu) and the drafted trees over the
// 4-bit cache (cs_qtree.cu) share.
//
// The query heads that share a key/value head are rows of one matrix product:
// a row tile has 128 rows, token by token and within a token head by head, and
// a CTA works on a pair of row tiles, so that every key and value tile in
// shared memory is used for 256 rows.  Per tile of 128 keys and row tile t
//     S_t = Q_t K^T   (tcgen05, operands in shared memory, S in tensor memory),
//     P_t = 2^(c (S_t - m) + shift)     by the 128 threads of warpgroup t,
//     O_t += P_t V    (tcgen05, P_t from tensor memory, where it takes S_t's place).
// One warp issues all products, in the order
//     S_0(0) S_1(0) | P_0(0)V S_0(1) | P_1(0)V S_1(1) | P_0(1)V S_0(2) ...
// so that one row tile's products run while the other one's P is worked out.
// A thread has a whole row: no shuffles, and its statistics stay in registers.
//
// A row's m follows its maximum only when that leads by more than 2^kLead in p;
// then the thread scales its row of O, which the order above leaves alone: S_t's
// commit covers the product with V before it.
//
// Work that is cut along the keys leaves records (each row's m, sum of p and
// sums of p v, in 32 bits); the CTA that finishes a row tile pair's last piece adds
// them up in the pieces' order, whoever comes last.
#pragma once

#include <cuda.h>

#include "cs_qcache.cuh"

namespace cs {

namespace {

constexpr int kTile = 128;            // rows of a row tile, keys of a step
constexpr int kPair = 2 * kTile;      // rows of a pair
constexpr int kBlock = 16384;         // bytes of 128 rows x 64 channels of 16 bits
constexpr float kLead = 8.f;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kTmemCols = 512;        // S_0, S_1 (128 each), O_0, O_1 (d each)

// ------------------------------------------------------------------- PTX forms

// Shared-memory matrix descriptor: address, leading and stride byte offsets in
// 16 bytes, descriptor version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t mat_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// kind::f16 instruction descriptor: fp32 sums, A K-major, B K-major or (b_mn) N-major, 128 x n.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, bool b_mn, int n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTile >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(desc), "r"(acc ? 1u : 0u));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(desc), "r"(acc ? 1u : 0u));
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tm_alloc(uint32_t *dst) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_free(uint32_t t) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(kTmemCols) : "memory");
}
// 32 columns of this thread's lane; the registers hold after tm_wait_ld.
__device__ __forceinline__ void tm_ld32(uint32_t t, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                   "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
                   "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
                   "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(t));
}
__device__ __forceinline__ void tm_st32(uint32_t t, const float *v) {
    const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
                 "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
                 "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
                 "r"(t)
                 : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
                 "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
                 : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A warpgroup's registers per thread, out of what the block was launched with.
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b) {   // (x, y) = (x, y) a + b
    asm("{\n\t.reg .b64 v, f, s;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 f, {%2, %2};\n\tmov.b64 s, {%3, %3};\n\t"
        "fma.rn.f32x2 v, v, f, s;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {   // (x, y) += (a, b)
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tadd.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------------------ work

// A piece of the keys of one pair of row tiles, for every head alike.
struct Work {
    int tok0, toks;   // first query token (a row of q, or a token of the tree), and how many
    int seq;          // sequence
    int lim0;         // keys that the first token may see, not yet cut to [0, n_k]; causal: one more for each further token
    int n_k, k0;      // the sequence's keys (slots), and the first one's row
    int j0, j1;       // key tiles of this piece
    int pieces, p;    // the pair's pieces, and which this is
    int rec;          // the first piece's place among one head's records
    int spare;
};
static_assert(sizeof(Work) == 48, "three 16-byte loads");

struct Plan {
    int *count;          // [0] works, [1] records of a head, [2] records that are planned so far
    Work *work;
    unsigned *arrived;   // [records] finished pieces, by the first record's place
    float *rec;          // [records] per row m and l, then [d][256] sums of p v
    int recs;            // how many records there is room for
};
__host__ __device__ constexpr size_t rec_floats(int d) { return (size_t)kPair * (d + 2); }

__device__ __forceinline__ Work load_work(const Work *w) {
    int4 v[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = ld_dep(reinterpret_cast<const int4 *>(w) + i);
    Work r;
    memcpy(&r, v, sizeof r);
    return r;
}

// This CTA's i-th work of `total`, which are in the order of falling size: there and back over the CTAs.
__device__ __forceinline__ int nth_work(int i) {
    const int g = gridDim.x, c = blockIdx.x;
    return i * g + (i & 1 ? g - 1 - c : c);
}

// Barriers of a CTA's roles.
template <int STAGES>
struct Bars {
    uint64_t q_full, q_empty;
    uint64_t full[STAGES], empty[STAGES];   // a stage holds one key or one value tile
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t written, told;                 // a record is written; whether it was the last
    uint64_t drain;
};
template <int STAGES>
__device__ __forceinline__ void init_bars(Bars<STAGES> &b, int q_writers, int writers) {
    mbar_init(&b.q_full, q_writers);
    mbar_init(&b.q_empty, 1);
    for (int i = 0; i < STAGES; ++i) {
        mbar_init(&b.full[i], writers);
        mbar_init(&b.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
        mbar_init(&b.s_full[t], 1);
        mbar_init(&b.p_full[t], kTile);
        mbar_init(&b.o_full[t], 1);
    }
    mbar_init(&b.written, kPair);
    mbar_init(&b.told, 1);
    mbar_init(&b.drain, 1);
    mbar_fence_init();
}

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint32_t *err) {
    if (mbar_wait(bar, parity, kWaitNs)) return true;
    atomicOr(err, CS_DEVERR_TIMEOUT);
    return false;
}

// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, uint32_t *err) {
    return __all_sync(kFull, wait(bar, parity, err));
}

// The key tiles of row tile t in this piece end where its last token's keys do.
struct Span {
    int toks, end;   // tokens of the tile; key tiles [j0, end), none if end <= j0
};
__device__ __forceinline__ Span span_of(const Work &w, int t, int per, int step) {
    Span s;
    s.toks = min(per, w.toks - t * per);
    const int lim = s.toks > 0 ? min(max(w.lim0 + step * (t * per + s.toks - 1), 0), w.n_k) : 0;
    s.end = min(w.j1, (lim + kTile - 1) / kTile);
    return s;
}

// ------------------------------------------------------------- the products' warp

// Issues a work's products; one thread.  it: key and value tiles so far (a ring of STAGES), n_p: P tiles so far.
struct MmaState {
    uint32_t it = 0, n_q = 0, n_p[2] = {0, 0};
};
template <int D, bool BF16, int STAGES>
__device__ __forceinline__ bool issue_work(const Work &w, const int (&end)[2], Bars<STAGES> &b, uint32_t tmem, uint32_t q_at, uint32_t ring,
                                           MmaState &st, uint32_t *err) {
    constexpr uint32_t kS = mma_desc(BF16, false, kTile), kO = mma_desc(BF16, true, D);
    constexpr int DB = D / 64;
    const int last = max(end[0], end[1]);
    if (last <= w.j0) return true;
    auto scores = [&](int t, uint32_t stage) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t in = (kk >> 2) * kBlock + (kk & 3) * 32;
            mma_ss(tmem + t * kTile, mat_desc(q_at + t * DB * kBlock + in, 16, 1024), mat_desc(ring + stage * DB * kBlock + in, 16, 1024),
                   kS, kk > 0);
        }
        mma_commit(&b.s_full[t]);
    };
    if (!wait(&b.q_full, st.n_q & 1, err)) return false;
    ++st.n_q;
    uint32_t ks = st.it % STAGES;
    if (!wait(&b.full[ks], st.it / STAGES & 1, err)) return false;
    tc_after();
#pragma unroll
    for (int t = 0; t < 2; ++t)
        if (w.j0 < end[t]) scores(t, ks);
    mma_commit(&b.empty[ks]);
    if (w.j0 + 1 == last) mma_commit(&b.q_empty);
    ++st.it;
    for (int j = w.j0; j < last; ++j) {
        const uint32_t vs = st.it % STAGES, vp = st.it / STAGES & 1;
        ++st.it;
        const bool more = j + 1 < last;
        uint32_t kp = 0;
        if (more) {
            ks = st.it % STAGES;
            kp = st.it / STAGES & 1;
            ++st.it;
        }
        if (!wait(&b.full[vs], vp, err)) return false;
        if (more && !wait(&b.full[ks], kp, err)) return false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (j >= end[t]) continue;
            if (!wait(&b.p_full[t], st.n_p[t] & 1, err)) return false;
            ++st.n_p[t];
            tc_after();
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
                mma_ts(tmem + 2 * kTile + t * D, tmem + t * kTile + kk * 8,
                       mat_desc(ring + vs * DB * kBlock + kk * 2048, kBlock, 1024), kO, j > w.j0 || kk > 0);
            if (j + 1 == end[t]) mma_commit(&b.o_full[t]);
            if (j + 1 < end[t]) scores(t, ks);
        }
        mma_commit(&b.empty[vs]);
        if (more) {
            mma_commit(&b.empty[ks]);
            if (j + 2 == last) mma_commit(&b.q_empty);
        }
    }
    return true;
}

// -------------------------------------------------------------- a row's softmax

struct RowState {
    float m, l;   // the maximum that p is taken against (-inf: none yet), the sum of p
    uint32_t n_s = 0, n_o = 0, n_rec = 0;   // waits so far
};

// fp16's p are taken 2^7 larger, so that those of 2^-31 of the largest are still there: with m following
// the maximum by 2^8 they stay below 2^16.  bf16 has fp32's range.
template <bool BF16>
constexpr float kShift = BF16 ? 0.f : 7.f;

// A row tile's key tiles [j0, end): its rows' statistics in r, their sums of p v in tensor memory.  mask(j, s): what the
// row does not see becomes -inf.
template <int D, bool BF16, int STAGES, typename Mask>
__device__ __forceinline__ bool softmax_rows(RowState &r, int j0, int end, int t, Bars<STAGES> &b, uint32_t tmem, float c, bool neg,
                                             uint32_t *err, Mask mask) {
    const uint32_t lane = ((threadIdx.x & 127) & ~31u) << 16;
    const uint32_t s_at = tmem + lane + t * kTile, o_at = tmem + lane + 2 * kTile + t * D;
    r.m = -INFINITY;
    r.l = 0.f;
    float base = 0.f, lead = -INFINITY;   // m, or 0 where that is -inf; a score beyond `lead` moves m
    for (int j = j0; j < end; ++j) {
        if (!wait_warp(&b.s_full[t], r.n_s & 1, err)) return false;
        ++r.n_s;
        tc_after();
        float s[kTile];
#pragma unroll
        for (int i = 0; i < 4; ++i) tm_ld32(s_at + 32 * i, s + 32 * i);
        tm_wait_ld();
        if (neg) {
#pragma unroll
            for (int i = 0; i < kTile; ++i) s[i] = -s[i];
        }
        mask(j, s);
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(s[i], s[4 + i], s[8 + i]);
#pragma unroll
        for (int i = 12; i + 8 <= kTile; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[i + e], s[i + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[kTile - 4 + e]);
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        if (__any_sync(kFull, top > lead)) {
            const float m = top > lead ? top : r.m;
            const float keep = r.m == -INFINITY ? 0.f : ex2((r.m - m) * c);
            r.m = m;
            base = m == -INFINITY ? 0.f : m;
            lead = m == -INFINITY ? -INFINITY : m + kLead / c;
            r.l *= keep;
            if (j > j0) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float o[32];
                    tm_ld32(o_at + 32 * i, o);
                    tm_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= keep;
                    tm_st32(o_at + 32 * i, o);
                }
            }
        }
        const float add = fmaf(-base, c, kShift<BF16>);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float &x = s[32 * i + 2 * e], &y = s[32 * i + 2 * e + 1];
                fma2(x, y, c, add);
                x = ex2(x);
                y = ex2(y);
                p[e] = pack2<BF16>(x, y);
                add2(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], x, y);
            }
            tm_st16(s_at + 16 * i, p);
        }
        r.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tm_wait_st();
        tc_before();
        mbar_arrive(&b.p_full[t]);
    }
    if (j0 < end) {
        if (!wait_warp(&b.o_full[t], r.n_o & 1, err)) return false;
        ++r.n_o;
        tc_after();
    }
    return true;
}

// After a piece's record is written: whether this CTA's is the pair's last piece (-1: a wait gave up).  All 256 threads of
// the row tiles; n: how often they have asked before.
template <int STAGES>
__device__ __forceinline__ int last_piece(Bars<STAGES> &b, unsigned *arrived, int pieces, volatile int *flag, uint32_t n, uint32_t *err) {
    __threadfence();
    mbar_arrive(&b.written);
    if (threadIdx.x == 0) {
        if (wait(&b.written, n & 1, err)) {
            *flag = atomicAdd(arrived, 1u) == (unsigned)pieces - 1;
            mbar_arrive(&b.told);
        }
    }
    __syncwarp();
    if (!wait_warp(&b.told, n & 1, err)) return -1;
    const int last = *flag;
    if (last) __threadfence();
    return last;
}

// A row's sums over its pieces: 1 / l in l, and put(i, o) for every 32 channels.
template <int D, typename Put>
__device__ __forceinline__ void join_pieces(const float *rec, int pieces, int row, float c, Put put) {
    float m = -INFINITY, l = 0.f;
    for (int p = 0; p < pieces; ++p) m = fmaxf(m, __ldcg(rec + p * rec_floats(D) + row));
    if (m == -INFINITY) m = 0.f;
    for (int p = 0; p < pieces; ++p) {
        const float *r = rec + p * rec_floats(D) + row;
        l = fmaf(ex2((__ldcg(r) - m) * c), __ldcg(r + kPair), l);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = 0; i < D / 32; ++i) {
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
        for (int p = 0; p < pieces; ++p) {
            const float *r = rec + p * rec_floats(D) + row;
            const float mp = __ldcg(r);
            if (mp == -INFINITY && __ldcg(r + kPair) == 0.f) continue;   // saw nothing, wrote nothing
            const float f = ex2((mp - m) * c) * inv;
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(f, __ldcg(r + (2 + 32 * i + e) * kPair), o[e]);
        }
        put(i, o);
    }
}

// 32 values of a row as 16 bits, its start on a 16-byte boundary.
template <bool BF16>
__device__ __forceinline__ void store32(char *at, const float *v) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint4 *>(at)[i] = make_uint4(pack2<BF16>(v[8 * i], v[8 * i + 1]), pack2<BF16>(v[8 * i + 2], v[8 * i + 3]),
                                                      pack2<BF16>(v[8 * i + 4], v[8 * i + 5]), pack2<BF16>(v[8 * i + 6], v[8 * i + 7]));
}

}  // namespace

}  // namespace cs
