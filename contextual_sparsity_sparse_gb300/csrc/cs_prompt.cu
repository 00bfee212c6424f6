// Attention of whole prompts, packed one behind the other: causal or not, with
// grouped heads.
//
// Three kernels.  The first lists the work: for every sequence, pairs of row tiles
// (cs_attn_tc.cuh) with the key tiles that they see, longest first, cut along
// the keys where few rows see many.  In the second a CTA per SM goes through
// the list for all key/value heads: one thread loads tiles by TMA, one issues
// the products, two warpgroups have the rows.  The third adds up what was cut.  A few works that need not be cut
// are listed by each CTA for itself, and there is only the second kernel.
//
// The rows of a tile are whole tokens of one group of heads: 128 / group tokens.
// A tile's box of q is [tokens][group][64 channels], so that it lands row by
// row as the products want it, whatever q's strides.
//
// A product with V adds p v for all 128 keys of a tile, and p = 0 does not undo a
// NaN or infinity in a v that a row does not see.  Such rows end up not finite,
// which is looked for when they are written.  When a CTA is through its list, it
// does the works with such rows once more: in value tiles that not all of a
// work's rows see (three at the most), what is not finite counts as 0, and a row
// adds what it does see of it.  So this takes about as long as those works did,
// however long the sequences are (4,090 tokens of 64 over 8 heads, not causal,
// with a NaN behind them: 366 us, and 829; 16,384 of 8 heads 370, with all values
// NaN 940).
#include "cs_attn_tc.cuh"

namespace cs {

namespace {

constexpr int kMaxGroup = 128;         // query heads of one key/value head
// Listed by every CTA itself are up to 32 pairs (a warp's lanes) of up to 31 sequences with up to kOwnTiles key tiles, which then
// are not cut.  Without the first and third kernels, and with them: 9 tokens of 8 heads 6.4 and 10.7 us, 10 prompts of 200 of 32 heads
// 24 and 29, 2,048 tokens of 40 heads 45 and 50; but where few works see many keys, cutting them is worth more: 100 tokens of 8 heads to
// a key head over 2,000 keys 30 and 22, one token over 2,048 18 and 17.  The tiles are those of all sequences together, which is all
// that the host knows.  With room for 32 of them 16 prompts of 200 tokens of 8 heads 12 us instead of 18, one of 2,304 of 40 heads 55
// instead of 61, but 100 tokens over 2,500 keys 35 instead of 23, over 4,096 52 instead of 24.
constexpr int kOwnPairs = 32, kOwnTiles = 16;
constexpr int kPromptThreads = 320;    // two warpgroups of rows, the products' warp, the loads' warp

struct PromptK {
    QRowsK q, k, v, out;
    int kv, group, batch, q_total, k_total, causal;
    const int32_t *q_start, *k_start;
    int one;             // both starts are the same, cut to the same total
    float scale;
    uint32_t *err;
    int per;             // tokens of a row tile
    int sms;
    int own;             // every CTA lists the works itself
};

// ------------------------------------------------------------------- the list

// Block-wide exclusive running maximum.
__device__ __forceinline__ int block_excl_max(int v, int *wmax) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc = max(inc, n);
    }
    if (lane == 31) wmax[warp] = inc;
    __syncthreads();
    int before = __shfl_up_sync(kFull, inc, 1);
    if (lane == 0) before = 0;
    for (int w = 0; w < warp; ++w) before = max(before, wmax[w]);
    __syncthreads();
    return before;
}

// start[0 .. batch], cut to [0, total] and made not to fall, into at.
__device__ void plan_starts(const int32_t *start, int batch, int total, int *at, int *wmax, uint32_t *err) {
    const int each = (batch + kPlanThreads) / kPlanThreads;
    const int b0 = min(batch + 1, (int)threadIdx.x * each), b1 = min(batch + 1, b0 + each);
    int top = 0;
    for (int b = b0; b < b1; ++b) {
        const int x = ld_dep(start + b);
        top = max(top, min(max(x, 0), total));
        at[b] = x;
    }
    int run = block_excl_max(top, wmax);
    for (int b = b0; b < b1; ++b) {
        const int x = at[b];
        run = max(run, min(max(x, 0), total));
        if (x != run) atomicOr(err, CS_DEVERR_COUNT);
        at[b] = run;
    }
}

// Pair i of sequence b, whose tokens and keys are these rows: its key tiles, and in w all of its work but the piece.
__device__ __forceinline__ int prompt_work(const PromptK &a, int b, int i, int q0, int q1, int k0, int k1, Work &w) {
    const int pair = 2 * a.per, t = i * pair, n_q = q1 - q0, n_k = k1 - k0;
    const int lim = a.causal ? min(max(n_k - n_q + min(t + pair, n_q), 0), n_k) : n_k;
    w.tok0 = q0 + t;
    w.toks = min(pair, n_q - t);
    w.seq = b;
    w.lim0 = a.causal ? n_k - n_q + t + 1 : n_k;
    w.n_k = n_k;
    w.k0 = k0;
    w.narrow = w.toks <= a.per;
    return (lim + kTile - 1) / kTile;
}

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(PromptK a, Plan plan) {
    extern __shared__ int starts[];
    __shared__ int scan[32];
    int *qs = starts, *ks = qs + a.batch + 1, *first = ks + a.batch + 1;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    plan_starts(a.q_start, a.batch, a.q_total, qs, scan, a.err);
    if (a.one) ks = qs;
    else plan_starts(a.k_start, a.batch, a.k_total, ks, scan, a.err);
    __syncthreads();
    const int pair = 2 * a.per;
    // the first pair of every sequence
    const int each = (a.batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(a.batch, tid * each), b1 = min(a.batch, b0 + each);
    int n = 0, total;
    for (int b = b0; b < b1; ++b) n += (qs[b + 1] - qs[b] + pair - 1) / pair;
    int at = block_excl_scan(n, scan, &total);
    for (int b = b0; b < b1; ++b) {
        first[b] = at;
        at += (qs[b + 1] - qs[b] + pair - 1) / pair;
    }
    __syncthreads();
    plan_list(total, a.kv, a.sms, plan, [&](int i, Work &w) {
        int lo = 0, hi = a.batch;   // the last sequence whose first pair is not behind i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i) lo = mid;
            else hi = mid;
        }
        return prompt_work(a, lo, i - first[lo], qs[lo], qs[lo + 1], ks[lo], ks[lo + 1], w);
    });
}

// The list of a few works that are not cut, by a warp: each CTA writes its own; returns their number.
__device__ __forceinline__ int own_list(const PromptK &a, Work *list) {
    const int lane = threadIdx.x & 31, pair = 2 * a.per;
    // lane b: sequence b's starts
    auto starts = [&](const int32_t *start, int total) {
        const int x = lane <= a.batch ? ld_dep(start + lane) : INT_MIN;
        int run = min(max(x, 0), total);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(kFull, run, o);
            if (lane >= o) run = max(run, n);
        }
        if (lane <= a.batch && x != run) atomicOr(a.err, CS_DEVERR_COUNT);
        return run;
    };
    const int q0 = starts(a.q_start, a.q_total), k0 = a.one ? q0 : starts(a.k_start, a.k_total);
    const int q1 = __shfl_down_sync(kFull, q0, 1), k1 = __shfl_down_sync(kFull, k0, 1);
    const int n = lane < a.batch ? (q1 - q0 + pair - 1) / pair : 0;
    int behind = n;   // the pairs of sequences up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, behind, o);
        if (lane >= o) behind += x;
    }
    const int total = __shfl_sync(kFull, behind, 31);
    // lane i: pair i, of the first sequence that has more behind it
    int b = 0;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (__shfl_sync(kFull, behind, b + o - 1) <= lane) b += o;
    b = min(b, a.batch - 1);
    Work w;
    const int at = lane - __shfl_sync(kFull, behind - n, b), qb = __shfl_sync(kFull, q0, b), qe = __shfl_sync(kFull, q1, b);
    const int kb = __shfl_sync(kFull, k0, b), ke = __shfl_sync(kFull, k1, b);
    w.j1 = prompt_work(a, b, at, qb, qe, kb, ke, w);
    w.j0 = w.p = w.rec = 0;
    w.pieces = 1;
    int place = 0;   // behind those of more tiles
    for (int i = 0; i < total; ++i) {
        const int x = __shfl_sync(kFull, w.j1, i);
        place += x > w.j1 || (x == w.j1 && i < lane);
    }
    if (lane < total) list[place] = w;
    return total;
}

// -------------------------------------------------------------- the attention

template <int D>
struct PromptCfg {
    static constexpr int DB = D / 64;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int OUT = D == 128 ? 4096 : 0;   // of each row warp, for its outputs
    static constexpr size_t smem = (size_t)(2 + STAGES) * DB * kBlock + 8 * OUT + 1024;
};

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *m, int c, int h, int row, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(m), "r"(c), "r"(h), "r"(row), "r"(smem_addr(bar))
                 : "memory");
}

// The first key tile of a sequence that not every row of the work sees.
__device__ __forceinline__ int first_masked(const Work &w) { return min(max(w.lim0, 0), w.n_k) / kTile; }

// What a warp's rows see of values that are not finite, in a work done without them, whose key `from` is the first of a tile
// that they may have been taken out of.  A thread has a row and its place: `to`, behind the last key that it sees (not falling
// from row to row; 0: not to be looked at), add, what p = 2^(c s + add) is taken against, and inv, the factor of its sums, or rec, where
// they are.  Per row and channel one such value is added, the last, or NaN where there are infinities of both signs, or a NaN.
// Lane l has channels N l ..; a key's values are read once for all rows, and a row's scores with those last keys alone worked out.
template <typename T, int D>
__device__ __noinline__ void add_seen(const PromptK &a, int64_t k0, int h, int from, int token, int head, int to, float c, float add,
                                      float inv, float *rec) {
    constexpr int N = D / 32, STEP = 8;
    struct alignas(2 * N) Vec {
        T x[N];
    };
    const int ch = N * (threadIdx.x & 31);
    const T *k = reinterpret_cast<const T *>(a.k.p) + k0 * a.k.ldt + h * a.k.ldh + ch;
    const T *v = reinterpret_cast<const T *>(a.v.p) + k0 * a.v.ldt + h * a.v.ldh + ch;
    int last[N], done = from;   // the last key before `done` with such a value, or -1
    bool up[N], down[N];        // whether there was one above 0 (or NaN), below 0 (or NaN)
#pragma unroll
    for (int i = 0; i < N; ++i) {
        last[i] = -1;
        up[i] = down[i] = false;
    }
    for (uint32_t rows = __ballot_sync(kFull, to > from); rows; rows &= rows - 1) {
        const int row = __ffs(rows) - 1, end = __shfl_sync(kFull, to, row);
        for (int j = done; j < end; j += STEP) {
            Vec y[STEP];
#pragma unroll
            for (int e = 0; e < STEP; ++e) y[e] = *reinterpret_cast<const Vec *>(v + min(j + e, end - 1) * a.v.ldt);
#pragma unroll
            for (int e = 0; e < STEP; ++e)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float x = (float)y[e].x[i];
                    if (isfinite(x)) continue;
                    last[i] = min(j + e, end - 1);
                    up[i] |= !(x < 0.f);
                    down[i] |= !(x > 0.f);
                }
        }
        done = max(done, end);
        int left[N], key = -1;
#pragma unroll
        for (int i = 0; i < N; ++i) key = max(key, left[i] = last[i]);
        key = __reduce_max_sync(kFull, key);
        if (key < 0) continue;
        const int tok = __shfl_sync(kFull, token, row), hq = __shfl_sync(kFull, head, row);
        const float plus = __shfl_sync(kFull, add, row), f = __shfl_sync(kFull, inv, row);
        const Vec q = *reinterpret_cast<const Vec *>(reinterpret_cast<const T *>(a.q.p) + tok * a.q.ldt + hq * a.q.ldh + ch);
        T *to_out = reinterpret_cast<T *>(a.out.p) + tok * a.out.ldt + hq * a.out.ldh + ch;
        float *to_rec = reinterpret_cast<float *>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(rec), row));
        while (key >= 0) {
            const Vec kk = *reinterpret_cast<const Vec *>(k + key * a.k.ldt), vv = *reinterpret_cast<const Vec *>(v + key * a.v.ldt);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) s = fmaf(a.scale < 0.f ? -(float)q.x[i] : (float)q.x[i], (float)kk.x[i], s);
            const float p = exp2f(fmaf(warp_sum(s), c, plus));
            int next = -1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (left[i] == key) {
                    left[i] = -1;
                    const float o = up[i] && down[i] ? NAN : p * (float)vv.x[i];
                    if (to_rec) __stcg(to_rec + (2 + ch + i) * kPair, __ldcg(to_rec + (2 + ch + i) * kPair) + o);
                    else to_out[i] = (T)((float)to_out[i] + o * f);
                }
                next = max(next, left[i]);
            }
            key = __reduce_max_sync(kFull, next);
        }
    }
}

// What the roles of a CTA share beside their barriers; state: whether a work was spoilt, whether a role has given up.
constexpr int SPOILT = 1, GAVE_UP = 2;
struct PromptShared {
    float2 stat[kTile];
    uint32_t spoilt[32];   // a bit for each of the CTA's works, and for every 1,024th behind it
    uint32_t tmem;
    int listed, state;

    __device__ __forceinline__ bool is_spoilt(int i) const { return spoilt[i >> 5 & 31] >> (i & 31) & 1u; }
};

// A CTA's works of `total`; AGAIN: those alone that were spoilt, without the values that can have spoilt them.
template <int D, bool BF16, bool AGAIN>
__device__ __forceinline__ void prompt_works(const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mv, const PromptK &a,
                                             const Plan &plan, const Work *works, int total, int recs, uint32_t q_at, uint32_t ring,
                                             uint32_t tmem, Bars<PromptCfg<D>::STAGES> &bars, PromptShared &s) {
    using C = PromptCfg<D>;
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, step = a.causal;
    // where a row tile's keys end in a work
    auto end_of = [&](const Work &w, int t) {
        const int toks = min(a.per, w.toks - t * a.per);
        const int lim = toks > 0 ? min(max(w.lim0 + step * (t * a.per + toks - 1), 0), w.n_k) : 0;
        return min(w.j1, (lim + kTile - 1) / kTile);
    };

    if (warp < 8) {
        const int t = warp >> 2, row = tid & 127, tok = row / a.group, g = row - tok * a.group;
        const bool neg = a.scale < 0.f;
        const float c = fabsf(a.scale) * 1.44269504088896341f;
        RowState r;
        for (int i = 0;; ++i) {
            const int x = nth_work(i);
            if (x >= total) break;
            if (AGAIN && !s.is_spoilt(i)) continue;
            const Work w = load_work(works + x / a.kv);
            const int h = x % a.kv, rt = w.narrow ? 0 : t, at = rt * a.per + tok;
            const Streams st = streams_of(w, end_of(w, 0), end_of(w, 1));
            const bool valid = tok < a.per && at < w.toks;
            const int token = w.tok0 + at;
            const int lim = valid ? min(max(w.lim0 + step * at, 0), w.n_k) : 0;
            const int all = __reduce_min_sync(kFull, valid ? lim : INT_MAX);   // keys that all of the warp's rows see
            if (!softmax_rows<D, BF16>(r, st.first[t], st.end[t], st.step, t, bars, tmem, c, neg, a.err, [&](int j, uint32_t (&m)[4]) {
                    if (all >= (j + 1) * kTile) return SEE_ALL;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int n = lim - j * kTile - 32 * e;
                        m[e] = n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1u;
                    }
                    return SEE_OWN;
                })) {
                atomicOr(&s.state, GAVE_UP);
                break;
            }
            Sums sums;
            if (!join_streams(r, st, t, bars, s.stat, c, sums, a.err)) {
                atomicOr(&s.state, GAVE_UP);
                break;
            }
            const bool mine = !(w.narrow && t == 1);   // whose rows these are
            T *out = reinterpret_cast<T *>(a.out.p) + token * a.out.ldt + (int64_t)(h * a.group + g) * a.out.ldh;
            float *rec = w.pieces > 1 ? plan.rec + (int64_t)(h * recs + w.rec) * rec_floats(D) : nullptr;
            if (mine) {
                const uint32_t o_at = tmem + (((uint32_t)row & ~31u) << 16) + 2 * kTile + t * D;
                float *my = rec ? rec + w.p * rec_floats(D) + rt * kTile + row : nullptr;
                const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
                if (my) put_stat<BF16>(my, r, c);
                RowWriter<BF16, D == 128> writer(ring + C::STAGES * C::DB * kBlock + warp * C::OUT, reinterpret_cast<char *>(out), valid);
                float odd = 0.f;   // NaN, if anything is not finite
#pragma unroll 1
                for (int b = 0; b < D / 32; ++b) {
                    float o[32];
                    load_sums<D>(o_at, b, sums, o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) odd = fmaf(o[e], 0.f, odd);
                    if (my) {
                        if (sums.some && valid) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) __stcg(my + (2 + 32 * b + e) * kPair, o[e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= inv;
                        writer.put(b, o);
                    }
                }
                const int from = first_masked(w) * kTile;
                if (AGAIN) {
                    __syncwarp();   // what is there has been written
                    add_seen<T, D>(a, w.k0, h, max(from, w.j0 * kTile), token, h * a.group + g,
                                   valid && isfinite(r.l) ? min(lim, w.j1 * kTile) : 0, c,
                                   fmaf(-(r.m == -INFINITY ? 0.f : r.m), c, kShift<BF16>), inv, my);
                } else if (__any_sync(kFull, valid && sums.some && !(odd == 0.f) && isfinite(r.l))) {
                    // (with a sum of p that is not finite all of the row is NaN, as it should be)
                    if (lane == 0) {
                        atomicOr(&s.spoilt[i >> 5 & 31], 1u << (i & 31));
                        atomicOr(&s.state, SPOILT);
                    }
                }
            }
            if (!leave_streams(r, st, t, bars, a.err)) {
                atomicOr(&s.state, GAVE_UP);
                break;
            }
        }
    } else if (warp == 8) {
        MmaState ms;
        bool ok = true;
        for (int i = 0; ok; ++i) {
            const int x = nth_work(i);
            if (x >= total) break;
            if (AGAIN && !s.is_spoilt(i)) continue;
            Work w = load_work(works + x / a.kv);
            const int end0 = uniform(end_of(w, 0)), end1 = uniform(end_of(w, 1));
            w.j0 = uniform(w.j0);
            w.narrow = uniform(w.narrow);
            ok = issue_work<D, BF16, C::STAGES, false, AGAIN>(streams_of(w, end0, end1), bars, tmem, q_at, ring, ms, a.err, 0,
                                                              AGAIN ? uniform(first_masked(w)) : 0);
        }
        if (!ok) {
            atomicOr(&s.state, GAVE_UP);
            mma_commit(&bars.drain);
            mbar_wait(&bars.drain, 0, kWaitNs);
        }
    } else {
        if (lane == 0) {
            uint32_t it = 0, n_q = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const int x = nth_work(i);
                if (x >= total) break;
                if (AGAIN && !s.is_spoilt(i)) continue;
                const Work w = load_work(works + x / a.kv);
                const int h = x % a.kv;
                const Streams st = streams_of(w, end_of(w, 0), end_of(w, 1));
                if (st.last <= w.j0) continue;
                if (n_q > 0 && !wait(&bars.q_empty, (n_q - 1) & 1, a.err)) {
                    ok = false;
                    break;
                }
                ++n_q;
                const int q0 = w.j0 < end_of(w, 0), q1 = !w.narrow && w.j0 < st.end[1];
                mbar_arrive_expect_tx(&bars.q_full, C::DB * a.per * a.group * 128 * (q0 + q1));
                for (int t = 0; t < 2; ++t)
                    if (t == 0 ? q0 : q1)
                        for (int b = 0; b < C::DB; ++b)
                            load_box(q_at + (t * C::DB + b) * kBlock, mq, 64 * b, h * a.group, w.tok0 + t * a.per, &bars.q_full);
                ok = tiles_in_order(st, [&](bool value, int j) {
                    const uint32_t at = it % C::STAGES;
                    if (it >= C::STAGES && !wait(&bars.empty[at], (it / C::STAGES - 1) & 1, a.err)) return false;
                    mbar_arrive_expect_tx(&bars.full[at], C::DB * kBlock);
#pragma unroll
                    for (int b = 0; b < C::DB; ++b)
                        load_box(ring + (at * C::DB + b) * kBlock, value ? mv : mk, 64 * b, h, w.k0 + j * kTile, &bars.full[at]);
                    ++it;
                    return true;
                });
            }
            if (!ok) {
                atomicOr(&s.state, GAVE_UP);
                // what is under way lands before the memory is given back
                for (uint32_t n = it > C::STAGES ? it - C::STAGES : 0; n < it; ++n)
                    mbar_wait(&bars.full[n % C::STAGES], n / C::STAGES & 1, kWaitNs);
                if (n_q > 0) mbar_wait(&bars.q_full, (n_q - 1) & 1, kWaitNs);
            }
        }
        __syncwarp();
    }
}

// The second time, out of line and with nothing held in registers for it, so that it costs next to nothing where there is nothing to
// mend: 8,192 tokens of 64 over 8 heads 680 us, of 16 heads of 64 channels 158 (with both times in one loop 732 and 178, with its
// arguments at hand 690 and 167, without it 678 and 156).
template <int D, bool BF16>
__device__ __noinline__ void prompt_again(const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mv, const PromptK &a,
                                          const Plan &plan, Bars<PromptCfg<D>::STAGES> &bars, PromptShared &s) {
    extern __shared__ uint8_t dsm[];
    const uint32_t q_at = (smem_addr(dsm) + 1023u) & ~1023u, ring = q_at + 2 * PromptCfg<D>::DB * kBlock, tmem = uniform(s.tmem);
    const Work *works = a.own ? plan.work + blockIdx.x * kOwnPairs : plan.work;
    const int total = uniform((a.own ? s.listed : ld_dep(plan.count)) * a.kv), recs = a.own ? 0 : ld_dep(plan.count + 1);
    prompt_works<D, BF16, true>(mq, mk, mv, a, plan, works, total, recs, q_at, ring, tmem, bars, s);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPromptThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
              const __grid_constant__ PromptK a, const __grid_constant__ Plan plan) {
    using C = PromptCfg<D>;
    extern __shared__ uint8_t dsm[];
    __shared__ Bars<C::STAGES> bars, more;   // of the works, and of those done once more
    __shared__ PromptShared s;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const uint32_t q_at = (smem_addr(dsm) + 1023u) & ~1023u, ring = q_at + 2 * C::DB * kBlock;
    if (warp == 8) tm_alloc(&s.tmem);
    if (tid == 288) {
        init_bars(bars, 1, 1);
        s.state = 0;
    }
    if (tid < 32) s.spoilt[tid] = 0;
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = uniform(s.tmem);
    pdl_wait();
    pdl_launch_dependents();
    const Work *works = plan.work;
    if (a.own) {
        Work *list = plan.work + blockIdx.x * kOwnPairs;
        if (warp == 0) {
            const int n = own_list(a, list);
            if (lane == 0) s.listed = n;
        }
        works = list;
        __syncthreads();
    }
    const int total = uniform((a.own ? s.listed : ld_dep(plan.count)) * a.kv), recs = a.own ? 0 : ld_dep(plan.count + 1);
    prompt_works<D, BF16, false>(&mq, &mk, &mv, a, plan, works, total, recs, q_at, ring, tmem, bars, s);
    tc_before();
    __syncthreads();
    if (s.state == SPOILT) {
        if (tid == 288) init_bars(more, 1, 1);
        __syncthreads();
        tc_after();
        prompt_again<D, BF16>(&mq, &mk, &mv, a, plan, more, s);
        tc_before();
        __syncthreads();
    }
    if (warp == 8) tm_free(tmem);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(PromptK a, Plan plan) {
    pdl_wait();
    pdl_launch_dependents();
    join_records<D>(
        plan, a.kv,
        [&](const Work &w, int h, int rt, int row) {
            const int tok = row / a.group, at = rt * a.per + tok;
            const bool valid = tok < a.per && at < w.toks;
            const int64_t to = (w.tok0 + at) * a.out.ldt + (int64_t)(h * a.group + row - tok * a.group) * a.out.ldh;
            return RowPlace{a.out.p + 2 * to, valid, valid};
        },
        [](char *at, int i, const float *o) { store8<BF16>(at + 16 * i, o); });
}

// ------------------------------------------------------------------- host side

bool prompt_sizes(int batch, int n_heads, int kv_heads, int d_head, int q_total, int k_total) {
    return batch >= 1 && batch <= kQMaxBatch && kv_heads >= 1 && n_heads >= kv_heads && n_heads <= kMaxHeads &&
           n_heads % kv_heads == 0 && n_heads / kv_heads <= kMaxGroup && (d_head == 64 || d_head == 128) && q_total >= 0 &&
           q_total <= kMaxTokens && k_total >= 0 && k_total <= kMaxTokens;
}

// The list's place behind the control words, with groups of `group` heads; returns the bytes.
size_t prompt_scratch(int batch, int group, int d, int q_total, int k_total, int sms, char *at, Plan *plan) {
    const int per = kTile / group;
    const int recs = k_total > kUncut * kTile ? 2 * sms : 0;
    const size_t works = (size_t)q_total / (2 * per) + batch, own = (size_t)kOwnPairs * sms;   // (calls of smaller sizes may list their own)
    return plan_scratch(works > own ? works : own, recs, d, at, plan);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);
EncodeFn encoder() {
    static const EncodeFn f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return f;
}

// [tokens, heads, d] rows in boxes of box_t tokens x box_h heads x 64 channels, swizzled by 128 bytes; zeros past the end.
bool head_map(CUtensorMap *m, const QRowsK &r, int d, int heads, int tokens, int box_h, int box_t) {
    const cuuint64_t row = (cuuint64_t)d * 2;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t ld[2] = {heads > 1 ? (cuuint64_t)r.ldh * 2 : row, tokens > 1 ? (cuuint64_t)r.ldt * 2 : row};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_h, (cuuint32_t)box_t}, step[3] = {1, 1, 1};
    return encoder()(m, r.dt == CS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, ld, box, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16>
cudaError_t run_prompt(const PromptK &a, const Plan &plan, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                       cudaStream_t s) {
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(&prompt_kernel<D, BF16>));
    if (e == cudaSuccess && !a.own) {
        e = allow_smem(reinterpret_cast<const void *>(&prompt_plan_kernel));
        if (e == cudaSuccess)
            e = launch(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 3 * ((size_t)a.batch + 1) * sizeof(int), s, pdl_enabled(), a, plan);
    }
    if (e != cudaSuccess) return e;
    // no more CTAs than there can be works
    const int64_t most = ((int64_t)a.q_total / (2 * a.per) + a.batch + plan.recs) * a.kv;
    e = launch(prompt_kernel<D, BF16>, dim3((unsigned)(most < a.sms ? most : a.sms)), dim3(kPromptThreads), PromptCfg<D>::smem, s,
               pdl_enabled(), mq, mk, mv, a, plan);
    if (e == cudaSuccess && plan.recs > 0 && !a.own)
        e = launch(prompt_join_kernel<D, BF16>, dim3(4 * a.sms), dim3(kJoinThreads), 0, s, pdl_enabled(), a, plan);
    return e;
}

}  // namespace

}  // namespace cs

using namespace cs;

extern "C" {

size_t cs_prompt_workspace_size(int batch, int n_heads, int kv_heads, int d_head, int q_total, int k_total) {
    if (!prompt_sizes(batch, n_heads, kv_heads, d_head, q_total, k_total)) return 0;
    // calls of fewer key/value heads have larger groups, and so more works
    const int group = n_heads < kMaxGroup ? n_heads : kMaxGroup;
    return kControlBytes + prompt_scratch(batch, group, d_head, q_total, k_total, device_sm_count(), nullptr, nullptr);
}

cs_status cs_prompt_attention(const cs_head_rows *q, const cs_head_rows *k, const cs_head_rows *v, int n_heads,
                              int kv_heads, int d_head, int batch, const int32_t *q_start, int q_total,
                              const int32_t *k_start, int k_total, int causal, float scale,
                              const cs_head_rows *out, void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_prompt_attention";
    PromptK a;
    CS_CHECK(q_total >= 0 && k_total >= 0, "%s: q_total and k_total must be >= 0 (%d, %d)", who, q_total, k_total);
    cs_status st = check_packed(q, q_total, n_heads, q_total == 0, "q", who, &a.q);
    if (st == CS_OK) st = check_packed(k, k_total, kv_heads, k_total == 0, "k", who, &a.k);
    if (st == CS_OK) st = check_packed(v, k_total, kv_heads, k_total == 0, "v", who, &a.v);
    if (st == CS_OK) st = check_packed(out, q_total, n_heads, q_total == 0, "out", who, &a.out);
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
    a.sms = device_sm_count();
    Plan plan;
    const size_t need = kControlBytes + prompt_scratch(batch, n_heads / kv_heads, d_head, q_total, k_total, a.sms,
                                                       static_cast<char *>(ws) + kControlBytes, &plan);
    st = check_qws(ws, ws_bytes, need, who);
    if (st != CS_OK) return st;
    if (q_total == 0) return CS_OK;
    a.kv = kv_heads;
    a.group = n_heads / kv_heads;
    a.batch = batch;
    a.q_total = q_total;
    a.k_total = k_total;
    a.causal = causal != 0;
    a.q_start = q_start;
    a.k_start = k_start ? k_start : q_start;
    a.one = a.k_start == q_start && q_total == k_total;
    a.scale = scale != 0.f ? scale : 1.f / sqrtf((float)d_head);
    a.err = static_cast<uint32_t *>(ws);
    a.per = kTile / a.group;
    a.own = batch < 32 && q_total / (2 * a.per) + batch <= kOwnPairs && k_total <= kOwnTiles * kTile;
    if (!encoder()) {
        set_error("%s: the driver has no tensor maps", who);
        return CS_ERR_CUDA;
    }
    CUtensorMap mq, mk, mv;
    bool ok = head_map(&mq, a.q, d_head, n_heads, q_total, a.group, a.per);
    if (k_total > 0)
        ok = ok && head_map(&mk, a.k, d_head, kv_heads, k_total, 1, kTile) && head_map(&mv, a.v, d_head, kv_heads, k_total, 1, kTile);
    else
        mk = mv = mq;   // there is no key to load
    if (!ok) {
        set_error("%s: the strides of q, k or v cannot be described as a tensor map", who);
        return CS_ERR_UNSUPPORTED;
    }
    const bool h = q->dtype == CS_F16;
    auto go = [&](auto run) { return run(a, plan, mq, mk, mv, (cudaStream_t)stream); };
    const cudaError_t e = d_head == 64 ? (h ? go(run_prompt<64, false>) : go(run_prompt<64, true>))
                                       : (h ? go(run_prompt<128, false>) : go(run_prompt<128, true>));
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
