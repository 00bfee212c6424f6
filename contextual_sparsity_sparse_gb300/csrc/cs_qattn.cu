// Host side of the attention over the 4-bit KV cache: scratch sizes, and the
// passes over a call's query rows.  The kernels are in cs_qattn.cuh.
#include "cs_qattn.cuh"

namespace cs {

extern template cudaError_t run_qattn<64>(QAttnK, int, int64_t, cudaStream_t);
extern template cudaError_t run_qattn<128>(QAttnK, int, int64_t, cudaStream_t);
extern template cudaError_t run_qattn<192>(QAttnK, int, int64_t, cudaStream_t);
extern template cudaError_t run_qattn<256>(QAttnK, int, int64_t, cudaStream_t);

namespace {

constexpr int kPass = 16;   // query rows of a pass

int mode_of(int rows) { return rows <= 4 ? PACK4 : rows <= 8 ? ONE8 : TWO8; }
int cols_of(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }
int unit_of(int d) { return d <= 128 ? 32 : 16; }
int64_t units_of(int cap, int d) { return (cap + unit_of(d) - 1) / unit_of(d); }
// The longest that a call's split axis can be.
int64_t cost_of(int batch, int kv_heads, int cap, int d) { return (int64_t)batch * kv_heads * (units_of(cap, d) + kHeadCost); }

int ctas_of(int sms) { return kMaxPerSm * (sms > 0 ? sms : 1); }
size_t left_bytes(int sms) { return align256((size_t)ctas_of(sms) * 4 * sizeof(int4)); }
size_t part_bytes(int d, int rows, int sms) { return align256((size_t)ctas_of(sms) * 2 * cols_of(rows) * (d + 3) * sizeof(float)); }
// For every number of CTAs per SM, which goes by the batch and by the rows of a pass.
size_t logit_bytes(int64_t cost, int cap, int d, int rows, int sms) {
    int64_t units = 0;
    for (int n = 1; n <= kMaxPerSm; ++n) {
        const int grid = qattn_grid(cost, ctas_of(sms) / kMaxPerSm * n);
        const int64_t u = grid * qattn_area(cost, grid, units_of(cap, d));
        units = u > units ? u : units;
    }
    return align256((size_t)units * unit_of(d) * cols_of(rows) * sizeof(float));
}

}  // namespace

size_t qattn_scratch(int batch, int kv_heads, int cap, int d, int heads, int n_q, bool weights, int sms) {
    const int rows = heads / kv_heads * n_q;
    return left_bytes(sms) + part_bytes(d, rows, sms) +
           (weights ? logit_bytes(cost_of(batch, kv_heads, cap, d), cap, d, rows, sms) : 0);
}

cudaError_t launch_qattn(const QAttnArgs &a, cudaStream_t s) {
    QAttnK k{a, a.heads / a.c.heads, 0, 0, 0, 0, nullptr, nullptr, nullptr, 0, (a.scale < 0 ? -a.scale : a.scale) * 1.44269504088896341f,
             a.scale < 0 ? -1.f : 1.f};
    const int rows = k.group * a.n_q, d = a.c.d;
    k.left = reinterpret_cast<int4 *>(a.scratch);
    k.part = reinterpret_cast<float *>(a.scratch + left_bytes(a.sms));
    if (a.weight) k.logit = reinterpret_cast<float *>(a.scratch + left_bytes(a.sms) + part_bytes(d, rows, a.sms));
    const int64_t cost = cost_of(a.c.batch, a.c.heads, a.c.cap, d);
    // a later pass adds its weights to an earlier one's
    for (k.row0 = 0; k.row0 < rows; k.row0 += kPass) {
        k.rows = rows - k.row0 < kPass ? rows - k.row0 : kPass;
        if (k.row0 > 0 && a.weight) {
            k.a.decay = 1.f;
            k.a.c.weight = a.weight;
        }
        const int mode = mode_of(k.rows);
        const cudaError_t e = d == 64    ? run_qattn<64>(k, mode, cost, s)
                              : d == 128 ? run_qattn<128>(k, mode, cost, s)
                              : d == 192 ? run_qattn<192>(k, mode, cost, s)
                                         : run_qattn<256>(k, mode, cost, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace cs
