// The KV cache held in 4 bits: writing rows, reading them back, choosing the
// slots to give up, and cutting a cache down.  (Attention: cs_qattn.cu.)
//
// Contextual sparsity keeps what a token needs and leaves the rest; a serving
// process does the same with its cache: the slots that gathered the least
// attention are given up, and the rows that stay are held in 4 bits.
#include "cs_qcache.cuh"

namespace cs {

namespace {

// ---------------------------------------------------------------- append, read

struct QRowsCall {
    QCacheK c;
    QRowsK k, v;
    int n;
    const int32_t *start, *slots, *n_new, *pos;
    uint32_t *err;
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

// One thread quantises 8 channels; the 8 threads of a group find its bounds
// together.  Consecutive groups of threads take consecutive channels, then
// tokens, of one head, so that the codes are written in long runs.  The code is
// the nearest of (x - offset) / scale in exact arithmetic: an fp32 quotient is
// off by less than 1e-5 where it matters (below 16), so only one within 1e-4
// of a half is divided again in 64 bits.
__global__ void __launch_bounds__(256) qappend_kernel(QRowsCall a) {
    pdl_wait();
    pdl_launch_dependents();
    const int per = a.c.d / 8, h = blockIdx.y, b = blockIdx.z;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = item / per;            // (token, k or v)
    const int c8 = (int)(item % per) * 8;
    const int t = (int)(row >> 1), isv = (int)(row & 1);
    int n = a.n;
    if (a.n_new) {
        const int m = ld_dep(a.n_new + b);
        if (m < 0 || m > n) atomicOr(a.err, CS_DEVERR_COUNT);
        n = m < 0 ? 0 : m < n ? m : n;
    }
    const bool on = t < n;
    const int slot = on ? slot_of(a, b, h, t) : -1;
    const QRowsK &r = isv ? a.v : a.k;
    float x[8];
    float lo = INFINITY, hi = -INFINITY;
    if (on) {
        load8(r, b * r.ldb + t * r.ldt + h * r.ldh + c8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = x[e] != x[e] ? 0.f : fminf(fmaxf(x[e], -65504.f), 65504.f);
            lo = fminf(lo, x[e]);
            hi = fmaxf(hi, x[e]);
        }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    }
    if (slot < 0) return;
    const __half sh = __float2half_rn((hi - lo) * (1.f / 15.f)), zh = __float2half_rn(lo);
    const float s = __half2float(sh), z = __half2float(zh), inv = 1.f / s;
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float n = 0.f;
        if (s > 0.f) {
            const float q = (x[e] - z) * inv;
            n = rintf(q);
            if (fabsf(fabsf(q - n) - 0.5f) < 1e-4f) n = (float)rint(((double)x[e] - (double)z) / (double)s);
            n = fminf(fmaxf(n, 0.f), 15.f);
        }
        codes |= (uint32_t)n << (4 * e);
    }
    const int64_t at = a.c.slot0(b, h) + slot;
    reinterpret_cast<uint32_t *>(isv ? a.c.v : a.c.k)[at * per + c8 / 8] = codes;
    if (c8 % kQGroup == 0)
        (isv ? a.c.vs : a.c.ks)[at * (a.c.d / kQGroup) + c8 / kQGroup] =
            (uint32_t)__half_as_ushort(sh) | (uint32_t)__half_as_ushort(zh) << 16;
    if (c8 == 0 && isv) {
        if (a.c.weight) a.c.weight[at] = 0.f;
        if (a.c.pos) a.c.pos[at] = ld_dep(a.pos + b) + t;
    }
}

// The same division of the work the other way round: one thread, 8 channels.
__global__ void __launch_bounds__(256) qread_kernel(QRowsCall a) {
    pdl_wait();
    pdl_launch_dependents();
    const int per = a.c.d / 8, h = blockIdx.y, b = blockIdx.z;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = item / per;
    const int c8 = (int)(item % per) * 8;
    const int t = (int)(row >> 1), isv = (int)(row & 1);
    if (t >= a.n) return;
    const int slot = slot_of(a, b, h, t);
    float x[8] = {};
    if (slot >= 0) {
        const int64_t at = a.c.slot0(b, h) + slot;
        const uint32_t codes = ld_dep(reinterpret_cast<const uint32_t *>(isv ? a.c.v : a.c.k) + at * per + c8 / 8);
        float s, z;
        half2x(ld_dep((isv ? a.c.vs : a.c.ks) + at * (a.c.d / kQGroup) + c8 / kQGroup), s, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(s, (float)(codes >> (4 * e) & 15u), z);
    }
    const QRowsK &r = isv ? a.v : a.k;
    store8(r, b * r.ldb + t * r.ldt + h * r.ldh + c8, x);
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

constexpr int kEvictThreads = 512;

// A total order on weights as unsigned integers: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0;
    if (u == 0x80000000u) u = 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One CTA per (sequence, head).  The slots to give up are the first e of the
// order (class, weight, slot), class 0 empty, 1 plain, 2 protected: the class
// and then the weight's four bytes are found one histogram at a time, and a
// last pass in slot order writes the chosen slots (or, for a trim, the others).
__global__ void __launch_bounds__(kEvictThreads) qevict_kernel(QEvictCall a) {
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
    const int32_t *pos = a.c.pos ? a.c.pos + slot0 : nullptr;
    const int64_t from = a.recent > 0 ? (int64_t)ld_dep(a.next_pos + b) - a.recent : INT64_MAX;
    auto cls = [&](int i) {
        if (!pos) return 1;
        const int p = ld_dep(pos + i);
        return p < 0 ? 0 : p < a.sinks || p >= from ? 2 : 1;
    };
    int want = e;            // still to take at or above the prefix found so far
    int c = -1;
    uint32_t key = 0;
    if (e > 0) {
        for (int i = tid; i < 4; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < used; i += kEvictThreads) atomicAdd(&hist[cls(i)], 1);
        __syncthreads();
        for (c = 0; c < 2 && want > hist[c]; ++c) want -= hist[c];
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < used; i += kEvictThreads) {
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
    for (int i0 = 0; i0 < used; i0 += kEvictThreads) {
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
        for (int i = e + tid; i < a.n; i += kEvictThreads) out[i] = used + i - e;
}

// One thread copies 4 bytes of a slot: words 0 .. d / 4 - 1 are its codes, the
// next 2 d / 64 its scales, then its weight and position.
__global__ void __launch_bounds__(256) qtrim_kernel(QEvictCall a, QCacheK dst) {
    pdl_wait();
    pdl_launch_dependents();
    const int h = blockIdx.y, b = blockIdx.z;
    const int cw = a.c.d / 8, sw = a.c.d / kQGroup, words = 2 * (cw + sw) + 2;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int t = (int)(item / words);
    int w = (int)(item % words);
    if (t >= min(a.keep, q_length(a.length, b, a.c.cap, nullptr))) return;
    const int slot = ld_dep(a.out + ((int64_t)b * a.c.heads + h) * a.keep + t);
    if (slot < 0 || slot >= a.c.cap) return;
    const int64_t from = a.c.slot0(b, h) + slot;
    const int64_t to = dst.slot0(b, h) + t;
    auto word = [](void *p, int64_t slot, int per, int i) { return reinterpret_cast<uint32_t *>(p) + slot * per + i; };
    if (w < cw) { *word(dst.k, to, cw, w) = ld_dep(word(a.c.k, from, cw, w)); return; }
    if ((w -= cw) < cw) { *word(dst.v, to, cw, w) = ld_dep(word(a.c.v, from, cw, w)); return; }
    if ((w -= cw) < sw) { *word(dst.ks, to, sw, w) = ld_dep(word(a.c.ks, from, sw, w)); return; }
    if ((w -= sw) < sw) { *word(dst.vs, to, sw, w) = ld_dep(word(a.c.vs, from, sw, w)); return; }
    if ((w -= sw) == 0) dst.weight[to] = ld_dep(a.c.weight + from);
    else if (dst.pos) dst.pos[to] = a.c.pos ? ld_dep(a.c.pos + from) : -1;
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

// append and read: 256 threads take 8 channels each of the key and value rows of one head
dim3 rows_grid(const QCacheK &c, int n) {
    return dim3((unsigned)(((int64_t)n * 2 * (c.d / 8) + 255) / 256), c.heads, c.batch);
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
    const cudaError_t e = launch(qappend_kernel, rows_grid(a.c, n), dim3(256), 0, (cudaStream_t)stream, pdl_enabled(), a);
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

cs_status cs_qcache_read(const cs_qcache *cache, const cs_head_rows *k, const cs_head_rows *v, int n,
                         const int32_t *start, const int32_t *slots, void *ws, size_t ws_bytes, cs_stream_t stream) {
    const char *who = "cs_qcache_read";
    QRowsCall a;
    const cs_status st = rows_call(cache, k, v, n, start, slots, ws, ws_bytes, who, &a);
    if (st != CS_OK) return st;
    if (n == 0) return CS_OK;
    const cudaError_t e = launch(qread_kernel, rows_grid(a.c, n), dim3(256), 0, (cudaStream_t)stream, pdl_enabled(), a);
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
    const cudaError_t e = launch(qevict_kernel, dim3(a.c.heads, a.c.batch), dim3(kEvictThreads), 0, (cudaStream_t)stream,
                                 pdl_enabled(), a);
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
    cudaError_t e = launch(qevict_kernel, dim3(a.c.heads, a.c.batch), dim3(kEvictThreads), 0, (cudaStream_t)stream, pdl_enabled(), a);
    const int words = 2 * (a.c.d / 8 + a.c.d / kQGroup) + 2;
    if (e == cudaSuccess)
        e = launch(qtrim_kernel, dim3((unsigned)(((int64_t)a.keep * words + 255) / 256), a.c.heads, a.c.batch), dim3(256), 0,
                   (cudaStream_t)stream, pdl_enabled(), a, to);
    return e == cudaSuccess ? CS_OK : cuda_fail(e, who);
}

}  // extern "C"
