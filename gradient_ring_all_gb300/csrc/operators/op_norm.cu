// op_norm.cu -- the join behind a block and the norm before the next one:
// ra_norm_block.
#include "op_norm.cuh"

namespace ra {
namespace op {
namespace {

struct NormParams {
    const void *x, *f, *gate;
    void *x_out, *h;
    float *kept;
    int64_t ld_x, ld_f, ld_gate, ld_x_out, ld_h, rows, d;
    Side post, pre;
    int gate_kind;
    bool gate_f32, gate_wide;
    float alpha, beta, per_d;  // per_d: 1 / d
};

template <class TX, class TF, int W, int N, int WARPS, bool JOIN, bool CLUSTER>
__global__ void __launch_bounds__(WARPS * 32 < kNormThreads ? kNormThreads : WARPS * 32) norm_kernel(const NormParams p) {
    constexpr int kGroups = WARPS * 32 < kNormThreads ? kNormThreads / (WARPS * 32) : 1;  // rows at a time
    using Sums = RowSums<2, WARPS, CLUSTER>;
    __shared__ Sums sums[kGroups];
    pdl_enter();
    if constexpr (CLUSTER) cluster_meet();  // every block is there before another writes to it
    const int id = threadIdx.x / (WARPS * 32);
    const Columns<W, N, WARPS, CLUSTER> col;
    int turn = 0;
    const int64_t blocks = CLUSTER ? gridDim.x / cluster_blocks() : gridDim.x, block = CLUSTER ? blockIdx.x / cluster_blocks() : blockIdx.x;

    // m and rstd of a row.  The sums of the values and of their squares are made at
    // once; where the mean is so large that their difference loses more than 4
    // bits, the squares of the differences from it are summed after it.
    auto moments = [&](const float (&v)[N][W], const Side &side, float *m, float *rstd) {
        float s[2] = {0.0f, 0.0f}, var;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) {  // columns past the row's end hold 0
                s[0] += v[i][j];
                s[1] = fmaf(v[i][j], v[i][j], s[1]);
            }
        row_sum(s, sums[id], id, turn);
        *m = 0.0f;
        var = s[1] * p.per_d;
        if (side.kind == RA_NORM_LAYER) {
            *m = s[0] * p.per_d;
            const float left = fmaf(-*m, *m, var);
            if (!(left * 16.0f >= var) && var > 0.0f) {  // the same for the whole row
                s[0] = s[1] = 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (col[i] < p.d) {
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            const float c = v[i][j] - *m;
                            s[0] = fmaf(c, c, s[0]);
                        }
                    }
                row_sum(s, sums[id], id, turn);
                var = s[0] * p.per_d;
            } else {
                var = left;
            }
        }
        *rstd = rsqrtf(var + side.eps);
    };
    auto apply = [&](float (&v)[W], const Side &side, float m, float rstd, int64_t c) {
        float g[W], b[W];
        load_param<W>(side.gain, side.f32, side.gain_wide, c, 1.0f, g);
        load_param<W>(side.bias, side.f32, side.bias_wide, c, 0.0f, b);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = fmaf((v[j] - m) * rstd, g[j], b[j]);
    };

    for (int64_t r = block * kGroups + id; r < p.rows; r += blocks * kGroups) {
        Raw<TX, W> rx[N];
        Raw<TF, W> rf[JOIN ? N : 1], rg[JOIN ? N : 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (col[i] < p.d) {
                rx[i].load(static_cast<const TX *>(p.x) + r * p.ld_x + col[i]);
                if constexpr (JOIN) {
                    rf[i].load(static_cast<const TF *>(p.f) + r * p.ld_f + col[i]);
                    if (p.gate_kind == RA_GATE_MATRIX) rg[i].load(static_cast<const TF *>(p.gate) + r * p.ld_gate + col[i]);
                }
            } else {
                rx[i].zero();
                if constexpr (JOIN) rf[i].zero();
            }
        }
        float v[N][W], m_f = 0.0f, rstd_f = 0.0f, m_x = 0.0f, rstd_x = 0.0f;
        if constexpr (JOIN) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = rf[i][j];
            if (p.post.kind != RA_NORM_NONE) moments(v, p.post, &m_f, &rstd_f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (col[i] >= p.d) continue;
                if (p.post.kind != RA_NORM_NONE) apply(v[i], p.post, m_f, rstd_f, col[i]);
                if (p.gate_kind == RA_GATE_MATRIX) {
#pragma unroll
                    for (int j = 0; j < W; ++j) v[i][j] *= rg[i][j];
                } else if (p.gate_kind == RA_GATE_VECTOR) {
                    float g[W];
                    load_param<W>(p.gate, p.gate_f32, p.gate_wide, col[i], 1.0f, g);
#pragma unroll
                    for (int j = 0; j < W; ++j) v[i][j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = fmaf(p.alpha, rx[i][j], p.beta * v[i][j]);
                store_w<TX, W>(static_cast<TX *>(p.x_out) + r * p.ld_x_out + col[i], v[i]);
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = to_f32<TX>(from_f32<TX>(v[i][j]));  // the norm is that of the row as stored
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = rx[i][j];
        }
        if (p.pre.kind != RA_NORM_NONE) {
            moments(v, p.pre, &m_x, &rstd_x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (col[i] >= p.d) continue;
                apply(v[i], p.pre, m_x, rstd_x, col[i]);
                store_w<TF, W>(static_cast<TF *>(p.h) + r * p.ld_h + col[i], v[i]);
            }
        }
        if (p.kept != nullptr && col.first == 0) reinterpret_cast<float4 *>(p.kept)[r] = make_float4(m_f, rstd_f, m_x, rstd_x);
    }
}

template <class TX, class TF, bool JOIN>
cudaError_t launch_norm(const NormParams &p, bool wide, cudaStream_t s) {
    auto go = [&](auto kernel, int warps, int cluster) {
        const Shape sh{warps, cluster};
        const int64_t most = 152 * 16;
        const int64_t blocks = ceil_div<int64_t>(p.rows, sh.groups());
        return launch_clusters(kernel, (blocks < most ? blocks : most) * cluster, cluster, sh.threads(), 0, s, p);
    };
    const int64_t d = p.d;
    if (wide) {
        if (d <= 256) return go(norm_kernel<TX, TF, 8, 1, 1, JOIN, false>, 1, 1);
        if (d <= 512) return go(norm_kernel<TX, TF, 8, 2, 1, JOIN, false>, 1, 1);
        if (d <= 1024) return go(norm_kernel<TX, TF, 8, 2, 2, JOIN, false>, 2, 1);
        if (d <= 2048) return go(norm_kernel<TX, TF, 8, 2, 4, JOIN, false>, 4, 1);
        if (d <= 4096) return go(norm_kernel<TX, TF, 8, 2, 8, JOIN, false>, 8, 1);
        if (d <= 8192) return go(norm_kernel<TX, TF, 8, 2, 16, JOIN, false>, 16, 1);
        return go(norm_kernel<TX, TF, 8, 2, 16, JOIN, true>, 16, d <= 16384 ? 2 : 4);
    }
    if (d <= 256) return go(norm_kernel<TX, TF, 1, 8, 1, JOIN, false>, 1, 1);
    if (d <= 512) return go(norm_kernel<TX, TF, 1, 16, 1, JOIN, false>, 1, 1);
    if (d <= 1024) return go(norm_kernel<TX, TF, 1, 16, 2, JOIN, false>, 2, 1);
    if (d <= 2048) return go(norm_kernel<TX, TF, 1, 16, 4, JOIN, false>, 4, 1);
    if (d <= 4096) return go(norm_kernel<TX, TF, 1, 16, 8, JOIN, false>, 8, 1);
    if (d <= 8192) return go(norm_kernel<TX, TF, 1, 16, 16, JOIN, false>, 16, 1);
    return go(norm_kernel<TX, TF, 1, 16, 16, JOIN, true>, 16, d <= 16384 ? 2 : 4);
}

template <bool JOIN>
cudaError_t launch_norm(const NormParams &p, int x_dtype, int f_dtype, bool wide, cudaStream_t s) {
    if (x_dtype == RA_BF16) return launch_norm<uint16_t, uint16_t, JOIN>(p, wide, s);
    return f_dtype == RA_F32 ? launch_norm<float, float, JOIN>(p, wide, s) : launch_norm<float, uint16_t, JOIN>(p, wide, s);
}

}  // namespace
}  // namespace op
}  // namespace ra

extern "C" ra_status ra_norm_block(const ra_norm_block_args *args, void *stream) {
    using namespace ra;
    using namespace ra::op;
    if (args == nullptr) return RA_ERR_INVALID_ARG;
    const ra_norm_block_args &a = *args;
    const bool join = a.f != nullptr, pre = a.pre.kind != RA_NORM_NONE;
    if (!sizes_ok(a.rows, a.d) || !types_ok(a.x_dtype, a.f_dtype) || !side_ok(a.pre)) return RA_ERR_INVALID_ARG;
    if (a.rows == 0 || a.d == 0) return RA_OK;
    if (!join && !pre) return RA_ERR_INVALID_ARG;
    const int gate = join ? a.gate_kind : RA_GATE_NONE, ex = esize(a.x_dtype), ef = esize(a.f_dtype);
    if (join && (!side_ok(a.post) || gate < RA_GATE_NONE || gate > RA_GATE_MATRIX)) return RA_ERR_INVALID_ARG;
    if (gate != RA_GATE_NONE && (a.gate == nullptr || (gate == RA_GATE_VECTOR && esize(a.gate_dtype) == 0))) return RA_ERR_INVALID_ARG;
    const int eg = gate == RA_GATE_VECTOR ? esize(a.gate_dtype) : ef;
    const Mat x{a.x, a.rows, a.d, a.ld_x, ex}, f{a.f, join ? a.rows : 0, a.d, a.ld_f, ef}, x_out{a.x_out, join ? a.rows : 0, a.d, a.ld_x_out, ex};
    const Mat h{a.h, pre ? a.rows : 0, a.d, a.ld_h, ef}, kept{a.kept, a.kept ? a.rows : 0, 4, 4, 4};
    const Mat gm{a.gate, gate == RA_GATE_MATRIX ? a.rows : gate == RA_GATE_VECTOR ? 1 : 0, a.d, a.ld_gate, eg};
    if (!mat_ok(x) || !mat_ok(f) || !mat_ok(x_out) || !mat_ok(h) || !mat_ok(gm) || !wide_at(a.kept)) return RA_ERR_INVALID_ARG;
    if (a.d > RA_NORM_MAX_D) return RA_ERR_UNSUPPORTED;
    const Side post = join ? side_of(a.post) : Side{}, ahead = side_of(a.pre);
    const Mat in[] = {x, f, gm, vector_of(post.gain, a.d, post.f32 ? 4 : 2), vector_of(post.bias, a.d, post.f32 ? 4 : 2),
                      vector_of(ahead.gain, a.d, ahead.f32 ? 4 : 2), vector_of(ahead.bias, a.d, ahead.f32 ? 4 : 2)};
    const Mat out[] = {x_out, h, kept};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 7; ++i)
            if (mats_overlap(out[o], in[i]) && !(o == 0 && i == 0 && same_mat(x, x_out))) return RA_ERR_OVERLAP;
        for (int q = 0; q < o; ++q)
            if (mats_overlap(out[o], out[q])) return RA_ERR_OVERLAP;
    }
    const Mat rows[] = {x, f, x_out, h, gate == RA_GATE_MATRIX ? gm : Mat{nullptr, 0, 0, 0, 4}};
    const NormParams p{a.x,  a.f,  a.gate, a.x_out, a.h,     a.kept, a.ld_x, a.ld_f,                  a.ld_gate,       a.ld_x_out, a.ld_h, a.rows,
                       a.d,  post, ahead,  gate,    gate == RA_GATE_VECTOR && a.gate_dtype == RA_F32, wide_at(a.gate), a.alpha,    a.beta, 1.0f / (float)a.d};
    const bool wide = all_wide(rows, a.d);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(join ? launch_norm<true>(p, a.x_dtype, a.f_dtype, wide, s) : launch_norm<false>(p, a.x_dtype, a.f_dtype, wide, s));
}
