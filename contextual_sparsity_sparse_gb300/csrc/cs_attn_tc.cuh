// Attention of many query rows over one head's keys and values on the tensor
// cores: what the packed prompts (cs_prompt.cu) and the drafted trees over the
// 4-bit cache (cs_qtree.cu) share.
//
// The query heads that share a key/value head are rows of one matrix product:
// a row tile has 128 rows, token by token and within a token head by head.  A
// CTA works on two streams of key tiles of 128 keys, each with a warpgroup of its
// own, whose threads have a row each, and 128 + d columns of tensor memory:
//     S_t = Q_t K^T   (tcgen05, operands in shared memory, S in tensor memory),
//     P_t = 2^(c (S_t - m) + shift)     by the threads of warpgroup t,
//     O_t += P_t V    (tcgen05, P_t from tensor memory, where it takes S_t's place).
// Wide work is a pair of row tiles: the streams are the two tiles, over the same
// keys, and every key and value tile in shared memory serves 256 rows.  Narrow
// work is one row tile: the streams take its keys in turn, and at the end
// warpgroup 0 adds up both.  One warp issues all products, in the order
//     S_0 S_1 | P_0 V  S_0 | P_1 V  S_1 | P_0 V  S_0 ...
// so that one stream's products run while the other one's P is worked out.
//
// A thread has a whole row: no shuffles, and its statistics stay in registers.
// It reads its scores twice, for the maximum and for P, rather than hold 128 of
// them.  m follows the maximum only when that leads by more than 2^kLead in p;
// then the thread scales its row of O, which the order above leaves alone: S_t's
// commit covers the product with V before it.
//
// Work that is cut along the keys leaves records (what each row's p are taken
// against, the sum of p and the sums of p v, in 32 bits), which another kernel
// adds up in the pieces' order.
//
// Bound (8,192 tokens, 64 over 8 heads of 128, causal, bf16: 683 us, 1,610
// TFLOP/s): a pair of key tile and row tiles takes 2,800 cycles, of which the products need 2,048.  A
// stream's next scores come 1,000 to 1,300 cycles after its last P (the product with V 512, the scores 512, barriers),
// and a row's work on 128 scores takes 1,450 (the maximum 480, P 900; exponentials at 4 cycles a warp 512).  Products with both
// operands in shared memory take all of its bandwidth, so every barrier and load costs 100 to 200 cycles beside them.
// Tried and not kept (packed prompts of up to 5,000 tokens, 64 over 8 heads, about 1,590 us then): a warp for
// each stream's products 2,111 instead of 1,708; P in one or four parts 1,764 and 1,957 instead of 1,718;
// a warpgroup of its own for the outputs, with 128 registers for the rows, 1,668 instead of 1,582; masked
// tiles 32 keys at a time inside the loop 1,668 instead of 1,590; works placed by half a tile's cost for narrow ones, no gain;
// outputs' loads from tensor memory ahead of their use 1,597 instead of 1,574.
#pragma once

#include <cuda.h>

#include "cs_qcache.cuh"

namespace cs {

namespace {

constexpr int kTile = 128;            // rows of a row tile, keys of a step
constexpr int kPair = 2 * kTile;      // rows of a pair
constexpr int kBlock = 16384;         // bytes of 128 rows x 64 channels of 16 bits
constexpr float kLead = 8.f;
constexpr uint64_t kWaitNs = 2000000000ull;   // a wait that is never over is given up then
constexpr int kTmemCols = 512;        // S_0, S_1 (128 each), O_0, O_1 (d each)
constexpr int kParts = 2;             // P is handed over in halves of a key tile

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
// Products and commits are issued by one thread, but by a warp that stays together, so that the compiler knows descriptors and
// addresses to be the same in all its threads: with one thread in a branch of its own each product took 70 cycles to
// issue, and the 16 products of a key tile and stream were what bounded the kernel.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool acc) {
    asm volatile("{\n\t.reg .pred p, one;\n\telect.sync _|one, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@one tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(desc), "r"(acc ? 1u : 0u));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool acc) {
    asm volatile("{\n\t.reg .pred p, one;\n\telect.sync _|one, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(desc), "r"(acc ? 1u : 0u));
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t"
                 "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
                 : "memory");
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
__device__ __forceinline__ void tm_st1(uint32_t t, float v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(t), "f"(v) : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
    int narrow;       // one row tile, whose keys the streams take in turn
};
static_assert(sizeof(Work) == 48, "three 16-byte loads");

struct Plan {
    int *count;          // [0] works, [1] records of a head, [2] pairs that are cut
    Work *work;
    int *cut;            // [records / 2] their first pieces
    float *rec;          // [records] per row the power of 2 that its p are taken against and l, then [d][256] sums of p v
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

constexpr int kPlanThreads = 256;   // (1,024 took 1.3 us longer, for their barriers)
constexpr int kLeastPiece = 4;      // key tiles of a piece (8: 100 tokens of 8 heads to a key head over 3,000 keys 26.7 us instead of 21.8)
constexpr int kUncut = 8;           // up to as many nothing is cut, and no room for records is needed

// Lists the works of `pairs` pairs of row tiles for kv heads: those of many key tiles first, cut along the keys so that no
// piece is longer than an SM's share of all, or where that makes more pieces than SMs, somewhat longer.  find(i, w): pair i's key tiles, and in w all of its work but the piece.  One
// CTA of kPlanThreads; places within a size differ from run to run, what a work is does not.
template <typename Find>
__device__ void plan_list(int pairs, int kv, int sms, const Plan &plan, Find find) {
    constexpr int BINS = 256;
    __shared__ int scan[32], hist[BINS], rounds[kPlanThreads / 32], longest, recs, placed, cuts;
    __shared__ unsigned long long units;
    const int tid = threadIdx.x;
    if (tid == 0) {
        longest = recs = placed = cuts = 0;
        units = 0;
    }
    if (tid < BINS) hist[tid] = 0;
    __syncthreads();
    unsigned long long sum = 0;
    int most = 0;
    Work w;
    for (int i = tid; i < pairs; i += kPlanThreads) {
        const int tiles = find(i, w);
        sum += tiles;
        most = max(most, tiles);
    }
    most = __reduce_max_sync(kFull, most);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if ((tid & 31) == 0 && sum) {
        atomicMax(&longest, most);
        atomicAdd(&units, sum);
    }
    __syncthreads();
    // with a pair's pieces fewer than twice its tiles / chunk, all pieces of cut pairs are fewer than 2 SMs' number
    int chunk = (int)min((unsigned long long)INT_MAX, max((unsigned long long)kLeastPiece, (units * kv + sms - 1) / sms));
    auto pieces_of = [&](int tiles) { return tiles > chunk && plan.recs > 0 ? (tiles + chunk - 1) / chunk : 1; };
    if (pairs * kv <= sms && plan.recs > 0) {
        // A piece more than there are SMs waits for a second round.  Each warp tries another length from here to twice that;
        // taken is the one whose rounds are soonest over.  (40 heads' 32 tokens over 2,048 slots: 4 pieces a head are 160.)
        const int c = chunk, warp = tid >> 5;
        chunk += (int)((long long)c * warp / (kPlanThreads / 32));
        int n = 0, top = 0, half = 0, most = 0;   // pieces, the longest, and how many are longer than half and 3/4 of that
        for (int i = tid & 31; i < pairs; i += 32) {
            const int tiles = find(i, w), pieces = pieces_of(tiles);
            n += pieces;
            top = max(top, (tiles + pieces - 1) / pieces);
        }
        n = __reduce_add_sync(kFull, n) * kv;
        top = __reduce_max_sync(kFull, top);
        if (n > sms) {
            for (int i = tid & 31; i < pairs; i += 32) {
                const int tiles = find(i, w), pieces = pieces_of(tiles), size = (tiles + pieces - 1) / pieces;
                if (2 * size > top) half += pieces;
                if (4 * size > 3 * top) most += pieces;
            }
            half = __reduce_add_sync(kFull, half) * kv;
            most = __reduce_add_sync(kFull, most) * kv;
        }
        // in quarters of a tile; beside its tiles a piece costs some 3 more.  The shortest pieces are a CTA's second.
        if ((tid & 31) == 0)
            rounds[warp] = n <= sms ? 4 * top + 12 : n > 2 * sms ? 12 * top + 36 : (half <= sms ? 4 : most <= sms ? 6 : 8) * top + 24;
        __syncthreads();
        int best = 0;
        for (int i = 1; i < kPlanThreads / 32; ++i)
            if (rounds[i] < rounds[best]) best = i;
        chunk = c + (int)((long long)c * best / (kPlanThreads / 32));
    }
    const int big = min(longest, chunk);
    auto bin_of = [&](int tiles, int pieces) {
        return BINS - 1 - min((tiles + pieces - 1) / pieces, big) * (BINS - 1) / max(big, 1);   // tiles are at most 2^17 and one
    };
    for (int i = tid; i < pairs; i += kPlanThreads) {
        const int tiles = find(i, w), pieces = pieces_of(tiles);
        atomicAdd(&hist[bin_of(tiles, pieces)], pieces);
        if (pieces > 1) {
            atomicAdd(&recs, pieces);
            atomicAdd(&cuts, 1);
        }
    }
    __syncthreads();
    const int mine = tid < BINS ? hist[tid] : 0;
    int all;
    const int place = block_excl_scan(mine, scan, &all);
    if (tid < BINS) hist[tid] = place;
    if (tid == 0) {
        plan.count[0] = all;
        plan.count[1] = recs;
        plan.count[2] = cuts;
        cuts = 0;
    }
    __syncthreads();
    const int lane = tid & 31;
    for (int i0 = tid - lane; i0 < pairs; i0 += kPlanThreads) {
        int tiles = 0, pieces = 0, to = 0;
        if (i0 + lane < pairs) {
            tiles = find(i0 + lane, w);
            pieces = pieces_of(tiles);
            to = atomicAdd(&hist[bin_of(tiles, pieces)], pieces);
            w.pieces = pieces;
            w.rec = w.p = w.j0 = 0;
            w.j1 = tiles;
            if (pieces > 1) {
                w.rec = atomicAdd(&placed, pieces);
                plan.cut[atomicAdd(&cuts, 1)] = to;
            } else {
                plan.work[to] = w;
            }
        }
        // a pair's pieces are written by the warp
        for (uint32_t cut = __ballot_sync(kFull, pieces > 1); cut; cut &= cut - 1) {
            const int from = __ffs(cut) - 1, n = __shfl_sync(kFull, pieces, from), at = __shfl_sync(kFull, to, from);
            Work x;
#pragma unroll
            for (int e = 0; e < (int)(sizeof(Work) / 4); ++e)
                reinterpret_cast<int *>(&x)[e] = __shfl_sync(kFull, reinterpret_cast<const int *>(&w)[e], from);
            const uint32_t all = x.j1;
            for (int p = lane; p < n; p += 32) {
                x.p = p;
                x.j0 = all * p / n;
                x.j1 = all * (p + 1) / n;
                plan.work[at + p] = x;
            }
        }
    }
}

// A list's place: its works' number and how many records there are; returns the bytes.
inline size_t plan_scratch(size_t works, int recs, int d, char *at, Plan *plan) {
    const size_t list = align256((works + recs) * sizeof(Work)), cut = align256((size_t)recs / 2 * sizeof(int));
    if (plan) {
        plan->count = reinterpret_cast<int *>(at);
        plan->work = reinterpret_cast<Work *>(at + 256);
        plan->cut = reinterpret_cast<int *>(at + 256 + list);
        plan->rec = reinterpret_cast<float *>(at + 256 + list + cut);
        plan->recs = recs;
    }
    return 256 + list + cut + (size_t)recs * rec_floats(d) * sizeof(float);
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
    uint64_t s_full[2], p_full[2][kParts], o_full[2];
    uint64_t ready, taken;                  // narrow work: stream 1 is done; it has been added to stream 0
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
        for (int i = 0; i < kParts; ++i) mbar_init(&b.p_full[t][i], kTile);
        mbar_init(&b.o_full[t], 1);
    }
    mbar_init(&b.ready, kTile);
    mbar_init(&b.taken, kTile);
    mbar_init(&b.drain, 1);
    mbar_fence_init();
}

// Waits that are not over at the first look; kept out of the loops, whose code the streams' warps fetch side by side.
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, uint32_t *err) {
    if (mbar_wait(bar, parity, kWaitNs)) return true;
    atomicOr(err, CS_DEVERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint32_t *err) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, err);
}
// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, uint32_t *err) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    return __all_sync(kFull, wait_long(bar, parity, err));
}

// Two waits in one: half of the warp's threads look at one barrier, half at the other.
__device__ __forceinline__ bool wait_both(uint64_t *a, uint32_t parity_a, uint64_t *b, uint32_t parity_b, uint32_t *err) {
    uint64_t *bar = threadIdx.x & 1 ? b : a;
    const uint32_t parity = threadIdx.x & 1 ? parity_b : parity_a;
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    return __all_sync(kFull, wait_long(bar, parity, err));
}

// A work's streams: stream t has key tiles first[t], first[t] + step, ... below end[t]; last: the end of both.
struct Streams {
    int first[2], end[2], step, last;
};
// ends: where row tile t's keys end (at most j1)
__device__ __forceinline__ Streams streams_of(const Work &w, int end0, int end1) {
    Streams s;
    s.first[0] = w.j0;
    s.first[1] = w.narrow ? w.j0 + 1 : w.j0;
    s.end[0] = end0;
    s.end[1] = w.narrow ? end0 : end1;
    s.step = w.narrow ? 2 : 1;
    s.last = max(s.end[0], s.end[1]);
    return s;
}

// The same value in all of a warp's threads, as the compiler can see.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(kFull, x, 0); }

// The order in which a work's key and value tiles are used: every key tile, and after it the value tile `ahead` key tiles
// back, so that a stream's next scores come right behind its product with V.
template <typename F>
__device__ __forceinline__ bool tiles_in_order(const Streams &s, F tile) {
    int key = s.first[0], val = key;   // one place for both, so that the tile's code is there once
    while (val < s.last) {
        const bool value = key - val >= s.step || key == s.last;
        if (!tile(value, value ? val++ : key++)) return false;
    }
    return true;
}

// ------------------------------------------------------------- the products' warp

// What is not finite in a tile in shared memory becomes 0; a whole warp, whose products read it next.
template <bool BF16>
__device__ __noinline__ void clean_tile(uint32_t at, int bytes) {
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    for (uint32_t x = at + (threadIdx.x & 31) * 16; x < at + bytes; x += 512) {
        uint32_t v[4], bad = 0;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(x) : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t out = ((v[i] & kExp) == kExp ? 0xffffu : 0u) | ((v[i] >> 16 & kExp) == kExp ? 0xffff0000u : 0u);
            v[i] &= ~out;
            bad |= out;
        }
        if (bad)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(x), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
    }
    fence_async();
    __syncwarp();
}

// Issues a work's products; a whole warp, whose arguments are the same in all threads.  (With a warp for each stream both
// streams' products share the tensor cores, and each stream waits twice as long for its own: 8,192 tokens of 16 heads 541 us
// instead of 412.)
struct MmaState {
    uint32_t stage = 0, parity = 0, n_q = 0, n_p[2] = {0, 0};   // the ring's next tile; works and P tiles so far
};
// SPLIT: key tiles below `split` come as two, fp16 values and behind them what their rounding left.
// CLEAN: of value tiles from `clean` on, values that are not finite count as 0.
template <int D, bool BF16, int STAGES, bool SPLIT = false, bool CLEAN = false>
__device__ __forceinline__ bool issue_work(const Streams &w, Bars<STAGES> &b, uint32_t tmem, uint32_t q_at, uint32_t ring, MmaState &st,
                                           uint32_t *err, int split = 0, int clean = 0) {
    constexpr uint32_t kS = mma_desc(BF16, false, kTile), kO = mma_desc(BF16, true, D);
    constexpr int DB = D / 64, STEPS = kTile / 16 / kParts;
    const int first = w.first[0];
    const bool narrow = w.step == 2;
    if (w.last <= first) return true;
    uint32_t stage = 0;
    auto next = [&]() {
        stage = st.stage;
        const uint32_t parity = st.parity;
        if (++st.stage == STAGES) {
            st.stage = 0;
            st.parity ^= 1;
        }
        return wait_warp(&b.full[stage], parity, err);
    };
    auto scores = [&](int t, uint32_t stage, bool more, uint32_t rest) {
        const uint64_t q = mat_desc(q_at + (narrow ? 0 : t) * DB * kBlock, 16, 1024);
        auto product = [&](uint32_t of, bool add) {
            const uint64_t k = mat_desc(ring + of * DB * kBlock, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t in = ((kk >> 2) * kBlock + (kk & 3) * 32) >> 4;
                mma_ss(tmem + t * kTile, q + in, k + in, kS, add || kk > 0);
            }
        };
        product(stage, false);
        if (SPLIT && more) product(rest, true);
        mma_commit(&b.s_full[t]);
    };
    auto values = [&](int t, uint32_t stage, bool fresh, bool done) {
        const uint64_t v = mat_desc(ring + stage * DB * kBlock, kBlock, 1024);
        const uint32_t n = t ? st.n_p[1]++ : st.n_p[0]++;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if (!wait_warp(&b.p_full[t][i], n & 1, err)) return false;
            tc_after();
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                const int kk = i * STEPS + k;
                mma_ts(tmem + 2 * kTile + t * D, tmem + t * kTile + kk * 8, v + (kk * 2048 >> 4), kO, !fresh || kk > 0);
            }
        }
        if (done) mma_commit(&b.o_full[t]);
        return true;
    };
    if (!wait_warp(&b.q_full, st.n_q & 1, err)) return false;
    ++st.n_q;
    // The streams in turn, t known at compile time: the product with the value tile that lies a step back, then scores of
    // key tile j.
    uint32_t vs = 0, ks = 0, kr = 0;
    auto turn = [&](auto stream, int j) {
        constexpr int t = decltype(stream)::value;
        const int jv = j - w.step, end = w.end[t];
        if (narrow || t == 0) {
            if (jv >= first && jv < w.last) {
                if (!next()) return false;
                vs = stage;
                if (CLEAN && jv >= clean) clean_tile<BF16>(ring + vs * DB * kBlock, DB * kBlock);
            }
            if (j < w.last) {
                if (!next()) return false;
                ks = stage;
                if (SPLIT && j < split) {
                    if (!next()) return false;
                    kr = stage;
                }
            }
        }
        if (jv >= first && jv < end) {
            if (!values(t, vs, jv == w.first[t], jv + w.step >= end)) return false;
        } else {
            tc_after();
        }
        if (j < end) scores(t, ks, SPLIT && j < split, kr);
        if (narrow || t == 1) {
            if (jv >= first && jv < w.last) mma_commit(&b.empty[vs]);
            if (j < w.last) mma_commit(&b.empty[ks]);
            if (SPLIT && j < w.last && j < split) mma_commit(&b.empty[kr]);
            if (j == w.last - 1) mma_commit(&b.q_empty);
        }
        return true;
    };
#pragma unroll 1
    for (int j = first; j < w.last + w.step; j += w.step)
        if (!turn(std::integral_constant<int, 0>(), j) || !turn(std::integral_constant<int, 1>(), narrow ? j + 1 : j)) return false;
    return true;
}

// -------------------------------------------------------------- a row's softmax

struct RowState {
    float m, l;   // the maximum that p is taken against (-inf: none yet), the sum of p
    uint32_t n_s = 0, n_o = 0, n_join = 0;   // waits so far
};

// fp16's p are taken 2^7 larger, so that those of 2^-31 of the largest are still there: with m following
// the maximum by 2^8 they stay below 2^16.  bf16 has fp32's range: taken 2^32 smaller, 2^24 of them times any v stay in it (and v
// have all their weight down to 2^-106: outputs of such values 1.77e-3 off in the norm instead of 1.71e-3, of 2^-110 7.7e-3).
template <bool BF16>
constexpr float kShift = BF16 ? -32.f : 7.f;

// What the rows of a warp see of a key tile: all of it, all the same keys, or each row keys of its own.
enum Sight { SEE_ALL, SEE_SAME, SEE_OWN };

// What is done to some tiles' scores in tensor memory stands out of the loop over tiles, whose code the warps of two streams
// and of the other roles fetch side by side.
//
// Keys that nobody sees are columns, most often few: written over one by one (128 selections in the loop and their way back
// to tensor memory took 1,400 cycles of a tile's 5,300).  w: the keys that are seen.
__device__ __noinline__ void hide_columns(uint32_t s_at, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const uint32_t out = ~(i == 0 ? w0 : i == 1 ? w1 : i == 2 ? w2 : w3);
        if (out == kFull) {
            float none[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) none[e] = -INFINITY;
            tm_st32(s_at + 32 * i, none);
        } else {
            for (uint32_t b = out; b; b &= b - 1) tm_st1(s_at + 32 * i + __ffs(b) - 1, -INFINITY);
        }
    }
    tm_wait_st();
}
// What this row does not see becomes -inf; for a negative scale, all scores are negated.
__device__ __noinline__ void hide_scores(uint32_t s_at, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, bool all, bool neg) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const uint32_t mine = all ? kFull : i == 0 ? w0 : i == 1 ? w1 : i == 2 ? w2 : w3;
        if (!neg && __all_sync(kFull, mine == kFull)) continue;
        float x[32];
        tm_ld32(s_at + 32 * i, x);
        tm_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = mine >> e & 1u ? (neg ? -x[e] : x[e]) : -INFINITY;
        tm_st32(s_at + 32 * i, x);
    }
    tm_wait_st();
}

// Stream t's key tiles first, first + step, ... below end: its rows' statistics in r, their sums of p v in tensor memory.
// mask(j, w): what the warp's rows see of tile j, and unless it is all the bits of those keys.
template <int D, bool BF16, int STAGES, typename Mask>
__device__ __forceinline__ bool softmax_rows(RowState &r, int first, int end, int step, int t, Bars<STAGES> &b, uint32_t tmem, float c,
                                             bool neg, uint32_t *err, Mask mask) {
    const uint32_t lane = ((threadIdx.x & 127) & ~31u) << 16;
    const uint32_t s_at = tmem + lane + t * kTile, o_at = tmem + lane + 2 * kTile + t * D;
    r.m = -INFINITY;
    r.l = 0.f;
    float base = 0.f, lead = -INFINITY;   // m, or 0 where that is -inf; a score beyond `lead` moves m
    for (int j = first; j < end; j += step) {
        uint32_t w[4];
        const Sight sight = mask(j, w);
        if (!wait_warp(&b.s_full[t], r.n_s & 1, err)) return false;
        ++r.n_s;
        tc_after();
        if (sight == SEE_SAME && !neg) hide_columns(s_at, w[0], w[1], w[2], w[3]);
        else if (sight != SEE_ALL || neg) hide_scores(s_at, w[0], w[1], w[2], w[3], sight == SEE_ALL, neg);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kTile; i += 64) {
            float x[64];
            tm_ld32(s_at + i, x);
            tm_ld32(s_at + i + 32, x + 32);
            tm_wait_ld();
#pragma unroll
            for (int e = 0; e < 64; e += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], x[e + q], x[e + 4 + q]);
        }
        constexpr int CK = 32, N = kTile / CK;   // scores read at a time
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        if (__any_sync(kFull, top > lead)) {
            const float m = top > lead ? top : r.m;
            const float keep = r.m == -INFINITY ? 0.f : ex2((r.m - m) * c);
            r.m = m;
            base = m == -INFINITY ? 0.f : m;
            lead = m == -INFINITY ? -INFINITY : m + kLead / c;
            r.l *= keep;
            if (j > first) {
#pragma unroll 1
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
        float s[2][CK];
        tm_ld32(s_at, s[0]);
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float (&v)[CK] = s[i & 1];
            if (i < N - 1) tm_ld32(s_at + CK * (i + 1), s[(i + 1) & 1]);
            uint32_t p[CK / 2];
#pragma unroll
            for (int e = 0; e < CK / 2; ++e) {
                float &x = v[2 * e], &y = v[2 * e + 1];
                fma2(x, y, c, add);
                x = ex2(x);
                y = ex2(y);
                p[e] = pack2<BF16>(x, y);
                add2(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], x, y);
            }
            // P's columns are half as many: they are of scores that have been read
            if (i < N - 1) tm_wait_ld();
            tm_st16(s_at + CK / 2 * i, p);
            if ((i + 1) % (N / kParts) == 0) {
                tm_wait_st();
                tc_before();
                mbar_arrive(&b.p_full[t][(i + 1) / (N / kParts) - 1]);
            }
        }
        r.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
    if (first < end) {
        if (!wait_warp(&b.o_full[t], r.n_o & 1, err)) return false;
        ++r.n_o;
        tc_after();
    }
    return true;
}

// What a warpgroup has to do with a work's sums when its stream is done.
struct Sums {
    float f0, f1;        // factors of this row's sums of stream t, and of stream 1 for narrow work
    bool some, other;    // whether there are such sums
};

// Narrow work: warpgroup 0 takes stream 1's statistics over into r, and gets the streams' factors.
template <int STAGES>
__device__ __forceinline__ bool join_streams(RowState &r, const Streams &w, int t, Bars<STAGES> &b, float2 *stat, float c, Sums &s, uint32_t *err) {
    const int row = threadIdx.x & 127;
    s.some = w.first[t] < w.end[t];
    s.f0 = s.f1 = 1.f;
    s.other = false;
    if (w.step == 1) return true;
    if (t == 1) {
        stat[row] = make_float2(r.m, r.l);
        tc_before();
        mbar_arrive(&b.ready);
        return true;
    }
    if (!wait_warp(&b.ready, r.n_join & 1, err)) return false;
    tc_after();
    const float2 o = stat[row];
    s.other = w.first[1] < w.end[1];
    if (!s.other) return true;
    const float m = fmaxf(r.m, o.x), base = m == -INFINITY ? 0.f : m;
    s.f0 = ex2((r.m - base) * c);
    s.f1 = ex2((o.x - base) * c);
    r.l = fmaf(s.f0, r.l, s.f1 * o.y);
    r.m = m;
    return true;
}
// The end of narrow work: stream 1's tensor memory is free again.
template <int STAGES>
__device__ __forceinline__ bool leave_streams(RowState &r, const Streams &w, int t, Bars<STAGES> &b, uint32_t *err) {
    if (w.step == 1) return true;
    const uint32_t parity = r.n_join++ & 1;
    if (t == 0) {
        tc_before();
        mbar_arrive(&b.taken);
        return true;
    }
    if (!wait_warp(&b.taken, parity, err)) return false;
    tc_after();
    return true;
}

// 32 columns of a row's sums, of both streams.
template <int D>
__device__ __forceinline__ void load_sums(uint32_t o_at, int i, const Sums &s, float (&o)[32]) {
    if (s.some) {
        tm_ld32(o_at + 32 * i, o);
        tm_wait_ld();
        if (s.other) {
            float x[32];
            tm_ld32(o_at + D + 32 * i, x);
            tm_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(s.f1, x[e], s.f0 * o[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
    }
}

// A row's statistics in its record.  What p are taken against is left as softmax_rows rounds it, so that pieces fit together.
template <bool BF16>
__device__ __forceinline__ void put_stat(float *rec, const RowState &r, float c) {
    __stcg(rec, r.m == -INFINITY ? -INFINITY : -fmaf(-r.m, c, kShift<BF16>));
    __stcg(rec + kPair, r.l);
}

// What join_records has to know of a row: where its outputs are, whether it has any, whether they are not just zeros.
struct RowPlace {
    char *at;
    bool there, valid;
};

// The outputs of the work that was cut, a warp for 8 channels of 32 rows: place(w, h, rt, row) tells of a row of row tile rt,
// put(at, i, o) takes channels 8 i .. of it.  Four pieces' loads are under way together.
template <int D, typename Place, typename Put>
__device__ __forceinline__ void join_records(const Plan &plan, int kv, Place place, Put put) {
    constexpr int G = D / 8, STEP = 4;
    const int lane = threadIdx.x & 31, warps = gridDim.x * (blockDim.x >> 5);
    const int total = ld_dep(plan.count + 2) * kv * (kPair / 32) * G, recs = ld_dep(plan.count + 1);
    for (int x = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); x < total; x += warps) {
        const int i = x % G, rows = x / G % (kPair / 32), h = x / (G * kPair / 32) % kv;
        const Work w = load_work(plan.work + ld_dep(plan.cut + x / (G * kPair / 32) / kv));
        const RowPlace row = place(w, h, rows / 4, rows % 4 * 32 + lane);
        if (!__any_sync(kFull, row.there)) continue;
        const float *rec = plan.rec + (int64_t)(h * recs + w.rec) * rec_floats(D) + rows * 32 + lane;
        float m = -INFINITY, l = 0.f, o[8] = {};
        for (int p0 = 0; p0 < w.pieces; p0 += STEP) {
            float pm[STEP], pl[STEP], v[STEP][8];
#pragma unroll
            for (int p = 0; p < STEP; ++p) {
                const bool some = row.valid && p0 + p < w.pieces;
                const float *r = rec + (p0 + p) * rec_floats(D);
                pm[p] = some ? __ldcg(r) : -INFINITY;
                pl[p] = some ? __ldcg(r + kPair) : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[p][e] = some ? __ldcg(r + (2 + 8 * i + e) * kPair) : 0.f;
            }
#pragma unroll
            for (int p = 0; p < STEP; ++p) {
                if (pm[p] == -INFINITY && pl[p] == 0.f) continue;   // saw nothing, may have written nothing
                const float up = fmaxf(m, pm[p]), base = up == -INFINITY ? 0.f : up;
                const float keep = m == -INFINITY ? 0.f : ex2(m - base), f = ex2(pm[p] - base);
                m = up;
                l = fmaf(f, pl[p], l * keep);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fmaf(f, v[p][e], o[e] * keep);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= inv;
        if (row.there) put(row.at, i, o);
    }
}
constexpr int kJoinThreads = 256;

// 8 or 32 values of a row as 16 bits, their place on a 16-byte boundary.
template <bool BF16>
__device__ __forceinline__ void store8(char *at, const float *v) {
    *reinterpret_cast<uint4 *>(at) = make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
}
template <bool BF16>
__device__ __forceinline__ void store32(char *at, const float *v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) store8<BF16>(at + 16 * i, v + 8 * i);
}

// Rows of 16-bit outputs, a thread's row in 32 channels at a time.  Written by the warp in lines: 64 channels of its 32 rows
// go through 4 KB of shared memory (threads that store rows of 128 channels themselves take a line for every 16 bytes: 5,000
// cycles a work, and as many until the loads behind them come through).  Few rows, or rows of 64 channels (LINES false; 8,192
// tokens of 16 heads 156 us, 165 in lines), are stored as they are.
template <bool BF16, bool LINES>
struct RowWriter {
    uint32_t at;       // the warp's shared memory
    char *row;         // where this thread's row goes
    uint32_t valid;    // the warp's rows that are written

    __device__ __forceinline__ RowWriter(uint32_t at, char *row, bool valid) : at(at), row(row), valid(__ballot_sync(kFull, valid)) {}

    // Channels 32 i .. of all rows; the whole warp.
    __device__ __forceinline__ void put(int i, const float *v) const {
        if constexpr (LINES) {
            if (__popc(valid) > 8) {
                put_lines(i, v);
                return;
            }
        }
        if (valid >> (threadIdx.x & 31) & 1u) store32<BF16>(row + 64 * i, v);
    }

private:
    __device__ __forceinline__ void put_lines(int i, const float *v) const {
        const int lane = threadIdx.x & 31, c0 = (i & 1) * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + lane * 128 + (((c0 + c) ^ (lane & 7)) << 4)),
                         "r"(pack2<BF16>(v[8 * c], v[8 * c + 1])), "r"(pack2<BF16>(v[8 * c + 2], v[8 * c + 3])),
                         "r"(pack2<BF16>(v[8 * c + 4], v[8 * c + 5])), "r"(pack2<BF16>(v[8 * c + 6], v[8 * c + 7]))
                         : "memory");
        if (!(i & 1)) return;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + lane / 8, c = lane & 7;
            char *to = reinterpret_cast<char *>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(row), r));
            uint4 x;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "r"(at + r * 128 + ((c ^ (r & 7)) << 4)) : "memory");
            if (valid >> r & 1u) *reinterpret_cast<uint4 *>(to + 64 * (i - 1) + 16 * c) = x;
        }
        __syncwarp();
    }
};

}  // namespace

}  // namespace cs
