// Attention for a tree of drafted tokens over the 4-bit KV cache.
//
// The streams of cs_attn_tc.cuh over tiles that six warps make from the codes: a
// tile's 128 slots become fp16 values, offset + scale * code with one rounding,
// in the layout that the products take.  Another warp copies codes, scales
// and positions into a ring ahead of them.  The tile behind the last slot
// holds the drafted tokens themselves, and there a row sees its own ancestors.
// Codes come as 8 nibbles to a word, of which an AND and an OR make two fp16
// numbers 1024 + n with n four channels apart: within 8 channels, the products
// run in the order 0 4 1 5 2 6 3 7.  q is written in that order too, and the
// outputs are put back when they are written.
//
// q's rows are scaled by powers of two to [2^14, 2^15), which fp16 holds with all
// bits of fp16 and bf16 inputs down to 2^-29 of a row's largest.
//
// Bound (32 ragged sequences of up to 8,192 slots, trees of 64 tokens, 64 over 8 heads
// of 128, bf16: 325 us, 845 TFLOP/s): a key tile for a pair of row tiles takes 4,600 cycles.  Issue slots are half
// used: P is 2 x 600 instructions a warp, a tile's 32,768 values 2,600 (three and a quarter per pair of codes), beside
// which the products' bandwidth in shared memory makes every store and barrier slow.  Narrow work (16 tokens: 133 us) waits for
// its tiles: 2,600 cycles for one.  Tried: 10, 8 or 14 makers instead of 6 370, 335 and 454 us instead of 363, narrow work 150 instead of 152;
// makers in three groups with a tile each 445 and 229; codes by each thread's own loads, three tiles ahead, 506 and 282.
#include <cstddef>

#include "cs_attn_tc.cuh"

namespace cs {

namespace {

constexpr int kMaxTree = 128;         // drafted tokens of a sequence: one key tile
constexpr int kTreeThreads = 512;     // two warpgroups of rows, kMakers warps that make tiles, one that loads codes, one for the products
constexpr int kMakers = 6, kLoader = 14, kIssuer = 15;
constexpr int kTreeStages = 4;
constexpr int kRaw = 3;               // tiles of codes under way
constexpr int kSeenRing = 8;          // tiles by which the makers can be ahead of the rows, and more
constexpr int kParentRing = 4;        // works likewise

struct TreeK {
    QCacheK c;
    QRowsK q, k, v, out;
    int heads, group, n, per, kv;
    const int32_t *length, *parent, *n_new;
    float scale;
    uint32_t *err;
    int sms;
};

// Drafted rows as the cache would take them: within fp16's range, NaN as 0.
__device__ __forceinline__ float as_drafted(float x) { return x != x ? 0.f : fminf(fmaxf(x, -65504.f), 65504.f); }

__device__ __forceinline__ float half_drafted(float x) { return __half2float(__float2half_rn(as_drafted(x))); }

__device__ __forceinline__ int tree_count(const TreeK &a, int b) {
    if (!a.n_new) return a.n;
    const int n = ld_dep(a.n_new + b);
    if (n < 0 || n > a.n) atomicOr(a.err, CS_DEVERR_COUNT);
    return min(max(n, 0), a.n);
}

// Work: tok0 is a token of the tree, toks how many of the pair's the sequence has (the others' rows are zeros), n_k its slots,
// k0 how many drafted tokens it has.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(TreeK a, Plan plan) {
    pdl_wait();
    pdl_launch_dependents();
    const int pair = 2 * a.per, each = (a.n + pair - 1) / pair;
    plan_list(a.c.batch * each, a.kv, a.sms, plan, [&](int i, Work &w) {
        const int b = i / each, t = (i - b * each) * pair;
        w.n_k = q_length(a.length, b, a.c.cap, a.err);
        w.tok0 = t;
        w.k0 = tree_count(a, b);
        w.toks = min(pair, w.k0 - t);
        w.seq = b;
        w.lim0 = 0;
        w.narrow = w.toks <= a.per;
        return w.toks > 0 ? (w.n_k + kTile - 1) / kTile + 1 : 0;
    });
}

template <int D>
struct TreeCfg {
    static constexpr int DB = D / 64;
    static constexpr int CH = D / 32;                 // 16-byte chunks of a slot's codes
    static constexpr int ROWS = 2 * 32 / CH;          // slots of a unit: a warp's chunks, two to a thread
    static constexpr int UNITS = kTile / ROWS;        // of a tile
    static constexpr int CODES = kTile * D / 2, SCALES = kTile * 4 * DB, RAW = CODES + SCALES + 4 * kTile;
    static constexpr size_t smem = (size_t)(2 + kTreeStages) * DB * kBlock + kRaw * RAW + 1024;
};

struct TreeShared {
    Bars<kTreeStages> bars;
    uint64_t seen_full[kSeenRing], raw_full[kRaw], raw_empty[kRaw];
    alignas(16) uint32_t seen[kSeenRing][4];    // of a tile of slots, those that are there
    uint8_t parents[kParentRing][kMaxTree];     // parent + 1 of every drafted token of a work's sequence
    float2 stat[kTile];
    uint32_t tmem;
};

static_assert(offsetof(TreeShared, seen) % 16 == 0, "read by 16 bytes");

// 16-byte chunk c of row r of a 128-byte swizzled tile of 64 channels
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
__device__ __forceinline__ void sts16(uint32_t at, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) { return pack2<false>(lo, hi); }

// 8 codes as fp16 values, in the products' order.
__device__ __forceinline__ void decode8(uint32_t w, __half2 s, __half2 z, uint32_t (&v)[4]) {
    const __half2 k1024 = __float2half2_rn(1024.f), k16th = __float2half2_rn(0.0625f), k64 = __float2half2_rn(-64.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = w >> 8 * i;
        const __half2 a = __hsub2(u2h((x & 0x000f000fu) | 0x64006400u), k1024);        // n, exact
        const __half2 b = __hfma2(u2h((x & 0x00f000f0u) | 0x64006400u), k16th, k64);   // (1024 + 16 n) / 16 - 64
        v[2 * i] = h2u(__hfma2(a, s, z));
        v[2 * i + 1] = h2u(__hfma2(b, s, z));
    }
}

// 8 channels of a row of any of the call's types, in order.
__device__ __forceinline__ void load8(const QRowsK &r, int64_t i, float (&x)[8]) {
    if (r.vec) {
        const uint4 v = ld_dep(reinterpret_cast<const uint4 *>(r.p + 2 * i));
        if (r.dt == CS_F16) unpack<__half>(v, x);
        else unpack<__nv_bfloat16>(v, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = q_load1(r, i + e);
    }
}

// fp16 inputs over caches of up to so many slots: keys count with all their bits, as a tile of fp16 values and one of what their
// rounding left (SPLIT).  Where a row has few keys nothing averages their roundings out: 24 tokens over 54 slots 3.2e-4 to 3.7e-4 of
// the output in the norm, of which the output's own rounding is 2.1e-4, and 2.7e-4 so; over 250 2.7e-4 to 3.6e-4, and 2.3e-4 to 2.5e-4.
// The host knows a cache's capacity, not the lengths: few slots of a larger cache are rounded.  (64 tokens over 1,000 slots 67 us
// instead of 44; decided work by work, by lengths, in one kernel: trees without them 2 to 25% slower.)
constexpr int kSplitSlots = 256;

// What the rounding of a tile's values to fp16 left, by the same units as the values, into the tile at `to`.
template <int D>
__device__ __noinline__ void make_rest(uint32_t codes, uint32_t to, int unit, int chunk, int in_unit) {
    using C = TreeCfg<D>;
    for (; unit < C::UNITS; unit += kMakers)
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const int r = unit * C::ROWS + in_unit + (i >> 2) * (C::ROWS / 2), k = i & 3;
            uint32_t sz, word, v[4];
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sz) : "r"(codes + C::CODES + (r * C::DB + chunk / 2) * 4));
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(word) : "r"(codes + r * (D / 2) + chunk * 16 + 4 * k));
            const __half2 hz = u2h(sz);
            float s, z;
            half2x(sz, s, z);
            decode8(word, __low2half2(hz), __high2half2(hz), v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo, hi;
                half2x(h2u(__hmin2(u2h(v[e]), __float2half2_rn(65504.f))), lo, hi);
                lo = fminf(fmaf((float)(word >> 4 * e & 15u), s, z), 65504.f) - lo;
                hi = fminf(fmaf((float)(word >> (4 * e + 16) & 15u), s, z), 65504.f) - hi;
                v[e] = half2_of(lo, hi);
            }
            sts16(to + chunk_at(r, (chunk & 1) * 4 + k), v);
        }
}

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(TreeK a, Plan plan) {
    using C = TreeCfg<D>;
    constexpr int CH = C::CH;
    extern __shared__ uint8_t dsm[];
    __shared__ TreeShared sh;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const uint32_t q_at = (smem_addr(dsm) + 1023u) & ~1023u, ring = q_at + 2 * C::DB * kBlock;
    const uint32_t raw = ring + kTreeStages * C::DB * kBlock;
    if (warp == kIssuer) tm_alloc(&sh.tmem);
    if (tid == 32 * kLoader) {
        init_bars(sh.bars, kPair, kMakers);
        for (int i = 0; i < kSeenRing; ++i) mbar_init(&sh.seen_full[i], kMakers);
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&sh.raw_full[i], 33);
            mbar_init(&sh.raw_empty[i], kMakers);
        }
        mbar_fence_init();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = uniform(sh.tmem);
    pdl_wait();
    pdl_launch_dependents();
    const int total = uniform(ld_dep(plan.count) * a.kv), recs = ld_dep(plan.count + 1);
    auto streams = [&](const Work &w) { return streams_of(w, w.toks > 0 ? w.j1 : w.j0, w.toks > a.per ? w.j1 : w.j0); };

    if (warp < 8) {
        const int t = warp >> 2, row = tid & 127, tok = row / a.group, g = row - tok * a.group;
        const bool neg = a.scale < 0.f;
        RowState r;
        uint32_t tiles = 0, works = 0;   // of this CTA, before this work
        for (int i = 0;; ++i) {
            const int x = nth_work(i);
            if (x >= total) break;
            const Work w = load_work(plan.work + x / a.kv);
            const int h = x % a.kv, rt = w.narrow ? 0 : t, at = rt * a.per + tok;
            const Streams st = streams(w);
            const bool valid = tok < a.per && at < w.toks, there = tok < a.per && w.tok0 + at < a.n;
            const int token = w.tok0 + at, head = h * a.group + g;
            float c = fabsf(a.scale) * 1.44269504088896341f;
            if (st.last > w.j0) {
                // the row's q, twice: for its power of two, and scaled
                const int64_t src = w.seq * a.q.ldb + token * a.q.ldt + (int64_t)head * a.q.ldh;
                float big = 0.f;
                if (valid) {
#pragma unroll 4
                    for (int e = 0; e < D; e += 8) {
                        float v[8];
                        load8(a.q, src + e, v);
#pragma unroll
                        for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(v[k]));
                    }
                }
                const int eb = (int)(__float_as_uint(big) >> 23);
                const int up = big > 0.f && eb < 255 ? min(141 - eb, 127) : 0;
                const float f1 = __uint_as_float((uint32_t)(127 + up / 2) << 23), f2 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
                // kept where c stays in fp32's range (beyond, one slot takes all as well)
                c = fminf(fmaxf(c * exp2f((float)-up), 1.2e-38f), 1.2e30f);
                if (rt == t) {
#pragma unroll 2
                    for (int e = 0; e < D; e += 8) {
                        float v[8] = {};
                        if (valid) load8(a.q, src + e, v);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = v[k] * f1 * f2;
                        const uint32_t p[4] = {half2_of(v[0], v[4]), half2_of(v[1], v[5]), half2_of(v[2], v[6]), half2_of(v[3], v[7])};
                        sts16(q_at + (t * C::DB + e / 64) * kBlock + chunk_at(row, e / 8 % 8), p);
                    }
                    fence_async();
                }
                mbar_arrive(&sh.bars.q_full);
            }
            const int drafted = (w.n_k + kTile - 1) / kTile;   // the tile of the drafted tokens
            if (!softmax_rows<D, false>(r, st.first[t], st.end[t], st.step, t, sh.bars, tmem, c, neg, a.err, [&](int j, uint32_t (&m)[4]) {
                    const uint32_t n = tiles + (j - w.j0), s = n % kSeenRing;
                    wait_warp(&sh.seen_full[s], n / kSeenRing & 1, a.err);
                    if (j < drafted) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(sh.seen[s]);
                        m[0] = uniform(v.x);
                        m[1] = uniform(v.y);
                        m[2] = uniform(v.z);
                        m[3] = uniform(v.w);
                        return (m[0] & m[1] & m[2] & m[3]) != kFull ? SEE_SAME : SEE_ALL;
                    }
                    m[0] = m[1] = m[2] = m[3] = 0;
                    if (valid) {
                        const uint8_t *parent = sh.parents[works % kParentRing];
                        if (!a.parent) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int n = token + 1 - 32 * e;
                                m[e] = n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1u;
                            }
                        } else {
                            for (int u = token; u >= 0; u = (int)parent[u] - 1) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (u >> 5 == e) m[e] |= 1u << (u & 31);
                            }
                        }
                    }
                    return SEE_OWN;
                }))
                break;
            if (st.last > w.j0) {
                tiles += st.last - w.j0;
                ++works;
            }
            Sums sums;
            if (!join_streams(r, st, t, sh.bars, sh.stat, c, sums, a.err)) break;
            const bool mine = !(w.narrow && t == 1);   // whose rows these are
            // a row tile's q has been read when its outputs are there: its memory takes them on their way
            const int64_t to = w.seq * a.out.ldb + token * a.out.ldt + (int64_t)head * a.out.ldh;
            RowWriter<BF16, D == 128> writer(q_at + rt * C::DB * kBlock + (warp & 3) * 4096, a.out.p + 2 * to, there);
            auto put = [&](int b, const float *o) {
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = o[(e & ~7) + (e & 3) * 2 + (e >> 2 & 1)];
                if (a.out.vec) {
                    writer.put(b, v);
                } else if (there) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) q_store1(a.out, to + 32 * b + e, v[e]);
                }
            };
            float *rec = w.pieces > 1 ? plan.rec + (int64_t)(h * recs + w.rec) * rec_floats(D) : nullptr;
            if (mine) {
                const uint32_t o_at = tmem + (((uint32_t)row & ~31u) << 16) + 2 * kTile + t * D;
                float *my = rec ? rec + w.p * rec_floats(D) + rt * kTile + row : nullptr;
                const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
                if (my) put_stat<false>(my, r, c);
#pragma unroll 1
                for (int b = 0; b < D / 32; ++b) {
                    float o[32];
                    load_sums<D>(o_at, b, sums, o);
                    if (my) {
                        if (sums.some && valid) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) __stcg(my + (2 + 32 * b + e) * kPair, o[e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = valid ? o[e] * inv : 0.f;
                        put(b, o);
                    }
                }
            } else if (w.p == 0 && tok < a.per && w.tok0 + a.per + tok < a.n) {
                // the pair's second row tile has no tokens: zeros
                const int64_t to = w.seq * a.out.ldb + (token + a.per) * a.out.ldt + (int64_t)head * a.out.ldh;
                for (int e = 0; e < D; ++e) q_store1(a.out, to + e, 0.f);
            }
            if (!leave_streams(r, st, t, sh.bars, a.err)) break;
        }
    } else if (warp < 8 + kMakers) {
        // a thread's chunk and slot: 8 threads side by side, which store together, have chunks of the same 64 channels in 4 slots,
        // so that their 16 bytes lie in different banks
        const int chunk = CH == 2 ? lane & 1 : (lane & 1) | (lane >> 2 & 2), in_unit = CH == 2 ? lane >> 1 : (lane >> 1 & 3) | (lane >> 2 & 4);
        const int c0 = (chunk & 1) * 4;
        uint32_t it = 0, cached = 0, tiles = 0, works = 0, units = warp - 8;   // units: until this warp's next one
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const int x = nth_work(i);
            if (x >= total) break;
            const Work w = load_work(plan.work + x / a.kv);
            const int h = x % a.kv, drafted = (w.n_k + kTile - 1) / kTile;
            const Streams st = streams(w);
            if (st.last <= w.j0) continue;
            ok = tiles_in_order(st, [&](bool value, int j) {
                const uint32_t stage = it % kTreeStages, tile = tiles + (j - w.j0), slot = tile % kSeenRing;
                // the stage is free, and the codes are there (a parity of 1 is that of the phase before the first)
                const uint32_t free = (it / kTreeStages & 1) ^ 1, from = cached % kRaw, codes = raw + from * C::RAW;
                if (!(j == drafted ? wait_warp(&sh.bars.empty[stage], free, a.err)
                                   : wait_both(&sh.bars.empty[stage], free, &sh.raw_full[from], cached / kRaw & 1, a.err)))
                    return false;
                ++it;
                const uint32_t to = ring + (stage * C::DB + chunk / 2) * kBlock;
                if (j == drafted) {
                    const QRowsK &rows = value ? a.v : a.k;
                    const int64_t src = w.seq * rows.ldb + h * rows.ldh + chunk * 32;
                    for (; units < C::UNITS; units += kMakers) {
                        if (!value && units == 0 && a.parent) {
                            for (int t = lane; t < w.k0; t += 32) {
                                int p = ld_dep(a.parent + (int64_t)w.seq * a.n + t);
                                if (p < -1 || p >= t) {
                                    atomicOr(a.err, CS_DEVERR_INDEX);
                                    p = -1;
                                }
                                sh.parents[works % kParentRing][t] = (uint8_t)(p + 1);
                            }
                        }
#pragma unroll 1
                        for (int ik = 0; ik < 8; ++ik) {
                            const int r = units * C::ROWS + in_unit + (ik >> 2) * (C::ROWS / 2), k = ik & 3;
                            float v[8] = {};
                            if (r < w.k0) load8(rows, src + r * rows.ldt + k * 8, v);
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = as_drafted(v[e]);
                            const uint32_t p[4] = {half2_of(v[0], v[4]), half2_of(v[1], v[5]), half2_of(v[2], v[6]), half2_of(v[3], v[7])};
                            sts16(to + chunk_at(r, c0 + k), p);
                        }
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (!value) mbar_arrive(&sh.seen_full[slot]);
                        mbar_arrive(&sh.bars.full[stage]);
                    }
                } else {
                    ++cached;
                    const int left = w.n_k - j * kTile;
                    const uint32_t first = units;
#pragma unroll 1
                    for (; units < C::UNITS; units += kMakers) {
                        const int r0 = units * C::ROWS + in_unit, mine = units * C::ROWS + (lane & (C::ROWS - 1));
                        uint4 cw[2];
                        uint32_t sz[2];
                        int pos = 0;
                        if (a.c.pos) asm volatile("ld.shared.s32 %0, [%1];" : "=r"(pos) : "r"(codes + C::CODES + C::SCALES + mine * 4));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = r0 + i * (C::ROWS / 2);
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sz[i]) : "r"(codes + C::CODES + (r * C::DB + chunk / 2) * 4));
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(cw[i].x), "=r"(cw[i].y), "=r"(cw[i].z), "=r"(cw[i].w)
                                         : "r"(codes + r * (D / 2) + chunk * 16));
                        }
                        const uint32_t bits = __ballot_sync(kFull, pos >= 0 && mine < left);
                        if (!value && lane == 0) {
                            if (C::ROWS == 16) reinterpret_cast<uint16_t *>(sh.seen[slot])[units] = (uint16_t)bits;
                            else sh.seen[slot][units & 3] = bits;
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = r0 + i * (C::ROWS / 2);
                            // a slot that is not there may hold anything: its value counts with 0 (and its key's scores are not looked at)
                            if (value && !(bits >> (in_unit + i * (C::ROWS / 2)) & 1u)) sz[i] = 0;
                            const __half2 hz = u2h(sz[i]), s = __low2half2(hz), z = __high2half2(hz);
                            const uint32_t word[4] = {cw[i].x, cw[i].y, cw[i].z, cw[i].w}, at = to + chunk_at(r, c0);
                            uint32_t v[4][4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) decode8(word[k], s, z, v[k]);
                            float sf, zf;
                            half2x(sz[i], sf, zf);
                            if (fmaf(15.f, sf, zf) > 65504.f) {   // a group that spans nearly all of fp16's range
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) v[k][e] = h2u(__hmin2(u2h(v[k][e]), __float2half2_rn(65504.f)));
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) sts16(at ^ (k << 4), v[k]);   // chunk c0 + k, as c0 is 0 or 4
                        }
                    }
                    const uint32_t rest = it % kTreeStages;
                    const bool more = SPLIT && !value;
                    if (more) {
                        if (!wait_warp(&sh.bars.empty[rest], (it / kTreeStages & 1) ^ 1, a.err)) return false;
                        ++it;
                        make_rest<D>(codes, ring + (rest * C::DB + chunk / 2) * kBlock, first, chunk, in_unit);
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (!value) mbar_arrive(&sh.seen_full[slot]);
                        mbar_arrive(&sh.raw_empty[from]);
                        mbar_arrive(&sh.bars.full[stage]);
                        if (more) mbar_arrive(&sh.bars.full[rest]);
                    }
                }
                units -= C::UNITS;
                return true;
            });
            tiles += st.last - w.j0;
            ++works;
        }
    } else if (warp == kLoader) {
        uint32_t it = 0;
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const int x = nth_work(i);
            if (x >= total) break;
            const Work w = load_work(plan.work + x / a.kv);
            const int h = x % a.kv, drafted = (w.n_k + kTile - 1) / kTile;
            const Streams st = streams(w);
            if (st.last <= w.j0) continue;
            ok = tiles_in_order(st, [&](bool value, int j) {
                if (j == drafted) return true;
                const uint32_t to = it % kRaw, codes = raw + to * C::RAW, bytes = min(kTile, w.n_k - j * kTile) * (D / 2);
                if (it >= kRaw && !wait_warp(&sh.raw_empty[to], (it / kRaw - 1) & 1, a.err)) return false;
                ++it;
                const int64_t slot0 = a.c.slot0(w.seq, h) + (int64_t)j * kTile;
                const int left = w.n_k - j * kTile;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.raw_full[to], bytes);
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(codes),
                                 "l"((value ? a.c.v : a.c.k) + slot0 * (D / 2)), "r"(bytes), "r"(smem_addr(&sh.raw_full[to]))
                                 : "memory");
                }
                const uint32_t *scales = (value ? a.c.vs : a.c.ks) + slot0 * C::DB;
#pragma unroll
                for (int e = 0; e < kTile; e += 32) {
                    const int r = e + lane;
                    if (r >= left) break;
                    copy_async<4 * C::DB>(codes + C::CODES + r * 4 * C::DB, scales + r * C::DB);
                    if (a.c.pos) copy_async<4>(codes + C::CODES + C::SCALES + r * 4, a.c.pos + slot0 + r);
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sh.raw_full[to])) : "memory");
                return true;
            });
        }
        if (!ok) {
            // what is under way lands before the memory is given back
            cp_async_commit();
            cp_async_wait<0>();
            for (uint32_t n = it > kRaw ? it - kRaw : 0; n < it; ++n) mbar_wait(&sh.raw_full[n % kRaw], n / kRaw & 1, kWaitNs);
        }
    } else {
        MmaState ms;
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const int x = nth_work(i);
            if (x >= total) break;
            Work w = load_work(plan.work + x / a.kv);
            w.toks = uniform(w.toks);
            w.j0 = uniform(w.j0);
            w.j1 = uniform(w.j1);
            w.narrow = uniform(w.narrow);
            ok = issue_work<D, false, kTreeStages, SPLIT>(streams(w), sh.bars, tmem, q_at, ring, ms, a.err,
                                                          SPLIT ? (uniform(w.n_k) + kTile - 1) / kTile : 0);
        }
        if (!ok) {
            mma_commit(&sh.bars.drain);
            mbar_wait(&sh.bars.drain, 0, kWaitNs);
        }
    }
    tc_before();
    __syncthreads();
    if (warp == kIssuer) tm_free(tmem);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(TreeK a, Plan plan) {
    pdl_wait();
    pdl_launch_dependents();
    join_records<D>(
        plan, a.kv,
        [&](const Work &w, int h, int rt, int row) {
            const int tok = row / a.group, at = rt * a.per + tok, token = w.tok0 + at;
            const int64_t to = w.seq * a.out.ldb + token * a.out.ldt + (int64_t)(h * a.group + row - tok * a.group) * a.out.ldh;
            const bool mine = tok < a.per && !(w.narrow && rt == 1);
            return RowPlace{a.out.p + 2 * to, mine && token < a.n, mine && at < w.toks};
        },
        [&](char *at, int i, const float *o) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = o[(e & 3) * 2 + (e >> 2)];
            if (a.out.vec) {
                store8<BF16>(at + 16 * i, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) q_store1(a.out, (at - a.out.p) / 2 + 8 * i + e, v[e]);
            }
        });
}

// -------------------------------------------------------------------- few rows
//
// The products above work on 128 rows however few there are.  Up to kFewRows rows
// of a cache head, which are one pass of the kernels of cs_qcache_attention, these
// go over the slots instead, and leave outputs in 32 bits with each row's
// statistics; a warp to a row then adds the drafted tokens on its path.  With 16 rows
// 131,001 slots of 8 heads take 75 us so and 110 with the products above, 32 ragged sequences of up to
// 8,192 105 and 125, 40 heads of 2,048 28 and 31; with 32 rows, two passes, 148 and 108, 207 and 126, 52 and 31.

constexpr int kFewRows = 16;

template <int D>
__global__ void __launch_bounds__(256) tree_path_kernel(TreeK a, const float *cached, const float2 *stat) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;   // [batch, n, heads]
    if (row >= (int64_t)a.c.batch * a.n * a.heads) return;
    const int lane = threadIdx.x & 31, head = (int)(row % a.heads), t = (int)(row / a.heads % a.n);
    const int b = (int)(row / a.heads / a.n), h = head / a.group, n = tree_count(a, b);
    float o[D / 32] = {};
    if (t < n) {
        const float c = a.scale * 1.44269504088896341f;
        const float2 st = ld_dep(stat + row);
        float m = st.x, l = st.y, x[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x[i] = c * q_load1(a.q, b * a.q.ldb + t * a.q.ldt + (int64_t)head * a.q.ldh + lane + 32 * i);
            o[i] = l * ld_dep(cached + row * D + lane + 32 * i);
        }
        for (int u = t; u >= 0;) {
            float s = 0.f, v[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int ch = lane + 32 * i;
                s = fmaf(x[i], half_drafted(q_load1(a.k, b * a.k.ldb + u * a.k.ldt + h * a.k.ldh + ch)), s);
                v[i] = half_drafted(q_load1(a.v, b * a.v.ldb + u * a.v.ldt + h * a.v.ldh + ch));
            }
            int next = u - 1;
            if (a.parent) {
                next = ld_dep(a.parent + (int64_t)b * a.n + u);
                if (next < -1 || next >= u) next = -1;   // flagged below
            }
            s = warp_sum(s);
            const float up = fmaxf(m, s), base = up == -INFINITY ? 0.f : up;
            const float keep = m == -INFINITY ? 0.f : exp2f(m - base), p = exp2f(s - base);
            m = up;
            l = fmaf(l, keep, p);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], keep, p * v[i]);
            u = next;
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = l == 0.f ? 0.f : o[i] / l;
        if (a.parent && head == 0 && lane == 0) {
            const int p = ld_dep(a.parent + (int64_t)b * a.n + t);
            if (p < -1 || p >= t) atomicOr(a.err, CS_DEVERR_INDEX);
        }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        q_store1(a.out, b * a.out.ldb + t * a.out.ldt + (int64_t)head * a.out.ldh + lane + 32 * i, o[i]);
}

// ------------------------------------------------------------------- host side

bool tree_sizes(int batch, int kv_heads, int capacity, int d_head, int n_heads, int n) {
    return batch >= 1 && batch <= kQMaxBatch && kv_heads >= 1 && kv_heads <= kMaxHeads && capacity >= 1 && capacity <= kMaxCapacity &&
           (d_head == 64 || d_head == 128) && n_heads >= kv_heads && n_heads % kv_heads == 0 && n >= 1 && n <= kMaxTree &&
           n_heads / kv_heads <= kTile && (int64_t)n_heads / kv_heads * n <= kQMaxRows;
}

// For few rows, `rows` of them in all and `each` of a cache head: the slots' outputs, the rows' statistics, and the other kernels' own.
struct FewScratch {
    size_t out, stat, attn;
    size_t all() const { return out + stat + attn; }
};
FewScratch few_scratch(int batch, int cap, int d, size_t rows, int each, int sms) {
    return FewScratch{align256(rows * d * sizeof(float)), align256(rows * sizeof(float2)),
                      qattn_scratch(batch, 1, cap, d, each, 1, false, sms)};
}
// For more: the list's place behind the control words, with `pairs` pairs of row tiles; returns the bytes.
size_t many_scratch(size_t pairs, int cap, int d, int sms, char *at, Plan *plan) {
    return plan_scratch(pairs, cap > (kUncut - 1) * kTile ? 2 * sms : 0, d, at, plan);
}
int tree_pairs(int group, int n) { return (n + 2 * (kTile / group) - 1) / (2 * (kTile / group)); }

// What calls of up to these sizes need: of fewer heads, tokens, or cache heads, and so of larger groups.
size_t tree_scratch(int batch, int kv_heads, int cap, int d, int n_heads, int n, int sms) {
    const int most = n_heads < kTile ? n_heads : kTile;
    int pairs = 0;
    for (int group = 1; group <= most; ++group) {
        const int p = tree_pairs(group, n < kQMaxRows / group ? n : kQMaxRows / group);
        pairs = p > pairs ? p : pairs;
    }
    const int rows = n_heads * n < kFewRows * kv_heads ? n_heads * n : kFewRows * kv_heads, each = most * n < kFewRows ? most * n : kFewRows;
    const size_t many = many_scratch((size_t)batch * pairs, cap, d, sms, nullptr, nullptr);
    const size_t few = few_scratch(batch, cap, d, (size_t)batch * rows, each, sms).all();
    return many > few ? many : few;
}

cudaError_t run_few(const TreeK &a, const FewScratch &need, char *scratch, cudaStream_t s) {
    float *out = reinterpret_cast<float *>(scratch);
    float2 *stat = reinterpret_cast<float2 *>(scratch + need.out);
    QAttnArgs q{};
    q.c = a.c;
    q.q = a.q;
    q.out = QRowsK{scratch, (int64_t)a.n * a.heads * a.c.d, (int64_t)a.heads * a.c.d, a.c.d, CS_F32, 1};
    q.heads = a.heads;
    q.n_q = a.n;
    q.length = a.length;
    q.scale = a.scale;
    q.taken = a.c.pos != nullptr;
    q.stat = stat;
    q.err = a.err;
    q.scratch = scratch + need.out + need.stat;
    q.sms = a.sms;
    cudaError_t e = launch_qattn(q, s);
    const dim3 grid((unsigned)(((int64_t)a.c.batch * a.n * a.heads + 7) / 8));
    if (e == cudaSuccess)
        e = a.c.d == 64 ? launch(tree_path_kernel<64>, grid, dim3(256), 0, s, pdl_enabled(), a, (const float *)out, (const float2 *)stat)
                        : launch(tree_path_kernel<128>, grid, dim3(256), 0, s, pdl_enabled(), a, (const float *)out, (const float2 *)stat);
    return e;
}

template <int D, bool BF16, bool SPLIT>
cudaError_t run_tree(const TreeK &a, const Plan &plan, cudaStream_t s) {
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(&tree_kernel<D, BF16, SPLIT>));
    if (e == cudaSuccess) e = launch(tree_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, pdl_enabled(), a, plan);
    if (e != cudaSuccess) return e;
    const int64_t most = ((int64_t)a.c.batch * ((a.n + 2 * a.per - 1) / (2 * a.per)) + plan.recs) * a.kv;
    e = launch(tree_kernel<D, BF16, SPLIT>, dim3((unsigned)(most < a.sms ? most : a.sms)), dim3(kTreeThreads), TreeCfg<D>::smem, s,
               pdl_enabled(), a, plan);
    if (e == cudaSuccess && plan.recs > 0)
        e = launch(tree_join_kernel<D, BF16>, dim3(4 * a.sms), dim3(kJoinThreads), 0, s, pdl_enabled(), a, plan);
    return e;
}

}  // namespace

}  // namespace cs

using namespace cs;

extern "C" {

size_t cs_qcache_tree_workspace_size(int batch, int kv_heads, int capacity, int d_head, int n_heads, int n) {
    if (!tree_sizes(batch, kv_heads, capacity, d_head, n_heads, n)) return 0;
    return kControlBytes + tree_scratch(batch, kv_heads, capacity, d_head, n_heads, n, device_sm_count());
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
    if (!tree_sizes(cache->batch, cache->n_heads, cache->capacity, cache->d_head, n_heads, n)) {
        set_error("%s: n=%d above %d, n_heads / the cache's above %d (%d), or %lld query rows per cache head above %d", who, n, kMaxTree,
                  kTile, n_heads / cache->n_heads, (long long)n_heads / cache->n_heads * n, kQMaxRows);
        return CS_ERR_UNSUPPORTED;
    }
    CS_CHECK(length && aligned(length, 4), "%s: length is null or misaligned", who);
    CS_CHECK(aligned(parent, 4) && aligned(n_new, 4), "%s: parent and n_new must be 4-byte aligned", who);
    CS_CHECK(scale == scale && scale - scale == 0.f, "%s: scale must be finite", who);
    a.heads = n_heads;
    a.group = n_heads / cache->n_heads;
    a.sms = device_sm_count();
    char *scratch = static_cast<char *>(ws) + kControlBytes;
    const bool few = a.group * n <= kFewRows;
    Plan plan;
    const FewScratch parts = few_scratch(a.c.batch, a.c.cap, a.c.d, (size_t)a.c.batch * n * n_heads, few ? a.group * n : 1, a.sms);
    const size_t need = few ? parts.all() : many_scratch((size_t)a.c.batch * tree_pairs(a.group, n), a.c.cap, a.c.d, a.sms, scratch, &plan);
    st = check_qws(ws, ws_bytes, kControlBytes + need, who);
    if (st != CS_OK) return st;
    a.n = n;
    a.per = kTile / a.group;
    a.kv = a.c.heads;
    a.length = length;
    a.parent = parent;
    a.n_new = n_new;
    a.scale = scale != 0.f ? scale : 1.f / sqrtf((float)cache->d_head);
    a.err = static_cast<uint32_t *>(ws);
    if (few) {
        if ((int64_t)cache->batch * cache->n_heads * ((cache->capacity + 15) / 16 + 32) >= INT32_MAX) {
            set_error("%s: batch x n_heads x capacity is too large", who);
            return CS_ERR_UNSUPPORTED;
        }
        const cudaError_t e = run_few(a, parts, scratch, (cudaStream_t)stream);
        return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
    }
    auto go = [&](auto run) { return run(a, plan, (cudaStream_t)stream); };
    auto by_type = [&](auto d) {
        if (q->dtype == CS_BF16) return go(run_tree<d(), true, false>);
        return a.c.cap <= kSplitSlots ? go(run_tree<d(), false, true>) : go(run_tree<d(), false, false>);
    };
    const cudaError_t e = a.c.d == 64 ? by_type(std::integral_constant<int, 64>()) : by_type(std::integral_constant<int, 128>());
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
