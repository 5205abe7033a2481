// op_norm_grad.cu -- the gradients of the join behind a block and of the norm
// before the next one: ra_norm_block_grad.
#include "op_norm.cuh"

namespace ra {
namespace op {
namespace {

enum { kPreGain, kPreBias, kPostGain, kPostBias, kGate, kVectors };

struct NormGradParams {
    const void *dh, *dx_new, *x, *f, *gate;
    const float *kept;
    void *dx, *df, *dgate;  // dgate: a matrix's
    float *parts;           // blocks x (kVectors or 2) x d, or null
    int64_t ld_dh, ld_dx_new, ld_x, ld_f, ld_gate, ld_dx, ld_df, ld_dgate, rows, d;
    Side post, pre;
    int gate_kind;
    bool gate_f32, gate_wide;
    float alpha, beta, per_d;
};

template <class TX, class TF, int W, int N, int WARPS, bool JOIN, bool CLUSTER>
__global__ void __launch_bounds__(WARPS * 32 < kNormThreads ? kNormThreads : WARPS * 32) norm_grad_kernel(const NormGradParams p) {
    constexpr int kGroups = WARPS * 32 < kNormThreads ? kNormThreads / (WARPS * 32) : 1, kSums = JOIN ? kVectors : 2;
    using Sums = RowSums<2, WARPS, CLUSTER>;
    using Cols = Columns<W, N, WARPS, CLUSTER>;
    __shared__ Sums sums[kGroups];
    __shared__ float joined[kGroups > 1 ? Cols::kMost : 1];
    pdl_enter();
    if constexpr (CLUSTER) cluster_meet();
    const int id = threadIdx.x / (WARPS * 32);
    const Cols col;
    int turn = 0;
    const int64_t blocks = CLUSTER ? gridDim.x / cluster_blocks() : gridDim.x, block = CLUSTER ? blockIdx.x / cluster_blocks() : blockIdx.x;
    float acc[kSums][N][W];
#pragma unroll
    for (int a = 0; a < kSums; ++a)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) acc[a][i][j] = 0.0f;

    for (int64_t r = block * kGroups + id; r < p.rows; r += blocks * kGroups) {
        Raw<TX, W> rx[N], rd[N];
        Raw<TF, W> rh[N], rf[JOIN ? N : 1], rg[JOIN ? N : 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            rx[i].zero();
            rd[i].zero();
            rh[i].zero();
            if constexpr (JOIN) rf[i].zero();
            if constexpr (JOIN) rg[i].zero();
            if (col[i] < p.d) {
                if (p.dh != nullptr) {
                    rh[i].load(static_cast<const TF *>(p.dh) + r * p.ld_dh + col[i]);
                    rx[i].load(static_cast<const TX *>(p.x) + r * p.ld_x + col[i]);
                }
                if (p.dx_new != nullptr) rd[i].load(static_cast<const TX *>(p.dx_new) + r * p.ld_dx_new + col[i]);
                if constexpr (JOIN) {
                    rf[i].load(static_cast<const TF *>(p.f) + r * p.ld_f + col[i]);
                    if (p.gate_kind == RA_GATE_MATRIX) rg[i].load(static_cast<const TF *>(p.gate) + r * p.ld_gate + col[i]);
                }
            }
        }
        const float4 kept = p.kept != nullptr ? reinterpret_cast<const float4 *>(p.kept)[r] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float full[N][W];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) full[i][j] = rd[i][j];
        if (p.dh != nullptr) {
            float s[2] = {0.0f, 0.0f}, v[N][W];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (col[i] >= p.d) continue;
                load_param<W>(p.pre.gain, p.pre.f32, p.pre.gain_wide, col[i], 1.0f, v[i]);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float unit = (rx[i][j] - kept.z) * kept.w;
                    v[i][j] *= rh[i][j];
                    s[0] = fmaf(v[i][j], unit, s[0]);
                    s[1] += v[i][j];
                    acc[kPreGain][i][j] = fmaf(rh[i][j], unit, acc[kPreGain][i][j]);
                    acc[kPreBias][i][j] += rh[i][j];
                }
            }
            row_sum(s, sums[id], id, turn);
            const float by_unit = s[0] * p.per_d, plain = p.pre.kind == RA_NORM_LAYER ? s[1] * p.per_d : 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (col[i] >= p.d) continue;
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float unit = (rx[i][j] - kept.z) * kept.w;
                    full[i][j] = fmaf(kept.w, v[i][j] - plain - unit * by_unit, full[i][j]);
                }
            }
        }
        if (p.dx != nullptr) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (col[i] >= p.d) continue;
                float y[W];
#pragma unroll
                for (int j = 0; j < W; ++j) y[j] = JOIN ? p.alpha * full[i][j] : full[i][j];
                store_w<TX, W>(static_cast<TX *>(p.dx) + r * p.ld_dx + col[i], y);
            }
        }
        if constexpr (JOIN) {
            float s[2] = {0.0f, 0.0f};
            const bool normed = p.post.kind != RA_NORM_NONE;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (col[i] >= p.d) continue;
                float gain[W], bias[W], gate[W];
                load_param<W>(normed ? p.post.gain : nullptr, p.post.f32, p.post.gain_wide, col[i], 1.0f, gain);
                load_param<W>(normed ? p.post.bias : nullptr, p.post.f32, p.post.bias_wide, col[i], 0.0f, bias);
                load_param<W>(p.gate_kind == RA_GATE_VECTOR ? p.gate : nullptr, p.gate_f32, p.gate_wide, col[i], 1.0f, gate);
                float dg[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float unit = normed ? (rf[i][j] - kept.x) * kept.y : rf[i][j];
                    const float u = p.beta * full[i][j];
                    dg[j] = u * fmaf(unit, gain[j], bias[j]);
                    acc[kGate][i][j] += dg[j];
                    const float v = u * (p.gate_kind == RA_GATE_MATRIX ? rg[i][j] : gate[j]);
                    acc[kPostGain][i][j] = fmaf(v, unit, acc[kPostGain][i][j]);
                    acc[kPostBias][i][j] += v;
                    full[i][j] = v * gain[j];
                    s[0] = fmaf(full[i][j], unit, s[0]);
                    s[1] += full[i][j];
                }
                if (p.dgate != nullptr) store_w<TF, W>(static_cast<TF *>(p.dgate) + r * p.ld_dgate + col[i], dg);
            }
            if (normed) {
                row_sum(s, sums[id], id, turn);
                const float by_unit = s[0] * p.per_d, plain = p.post.kind == RA_NORM_LAYER ? s[1] * p.per_d : 0.0f;
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        const float unit = (rf[i][j] - kept.x) * kept.y;
                        full[i][j] = kept.y * (full[i][j] - plain - unit * by_unit);
                    }
            }
            if (p.df != nullptr) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (col[i] < p.d) store_w<TF, W>(static_cast<TF *>(p.df) + r * p.ld_df + col[i], full[i]);
            }
        }
    }

    if (p.parts == nullptr) return;
#pragma unroll
    for (int a = 0; a < kSums; ++a) {
        if constexpr (kGroups > 1) {  // the groups' sums in their order
            for (int g = 0; g < kGroups; ++g) {
                __syncthreads();
                if (id != g) continue;
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        float &at = joined[col[i] + j];
                        at = g == 0 ? acc[a][i][j] : at + acc[a][i][j];
                    }
            }
            __syncthreads();
            for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) p.parts[(block * kSums + a) * p.d + c] = joined[c];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (col[i] < p.d) p.parts[(block * kSums + a) * p.d + col[i] + j] = acc[a][i][j];
        }
    }
}

// The blocks' sums, added in their order: a block takes 32 columns of one
// vector, warp w the parts w, w + 8, ...
struct PartsParams {
    const float *parts;
    float *out[kVectors];
    int64_t count, d;  // parts
    int vectors, accumulate;
};
__global__ void __launch_bounds__(256) parts_kernel(const PartsParams p) {
    __shared__ float sum[8][32];
    pdl_enter();
    const int64_t strips = ceil_div<int64_t>(p.d, 32);
    const int a = (int)(blockIdx.x / strips), lane = threadIdx.x & 31, w = threadIdx.x / 32;
    const int64_t c = blockIdx.x % strips * 32 + lane;
    float *out = p.out[0];
#pragma unroll
    for (int k = 1; k < kVectors; ++k)
        if (a == k) out = p.out[k];
    if (out == nullptr) return;
    float s = 0.0f;
    if (c < p.d)
        for (int64_t b = w; b < p.count; b += 8) s += p.parts[(b * p.vectors + a) * p.d + c];
    sum[w][lane] = s;
    __syncthreads();
    if (w != 0 || c >= p.d) return;
    for (int k = 1; k < 8; ++k) s += sum[k][lane];
    out[c] = p.accumulate ? out[c] + s : s;
}

// ---------------------------------------------------------------------------
// host

// 8 values a thread, as their sums over the rows are held beside them
Shape grad_shape(int64_t d) {
    if (d <= 256) return {1, 1};
    if (d <= 512) return {2, 1};
    if (d <= 1024) return {4, 1};
    if (d <= 2048) return {8, 1};
    if (d <= 4096) return {16, 1};
    return {16, d <= 8192 ? 2 : d <= 16384 ? 4 : 8};
}
// blocks (or clusters) that share the rows, each with a part of the sums
int64_t grad_parts(int64_t rows, int64_t d) {
    const Shape sh = grad_shape(d);
    const int64_t most = 152 * (sh.warps == 16 ? 1 : 2) / sh.cluster, blocks = ceil_div<int64_t>(rows, sh.groups());
    return blocks < most ? blocks : most;
}

template <class TX, class TF, bool JOIN>
cudaError_t launch_grad(const NormGradParams &p, bool wide, cudaStream_t s) {
    const Shape sh = grad_shape(p.d);
    auto go = [&](auto kernel, auto scalar) {
        return launch_clusters(wide ? kernel : scalar, grad_parts(p.rows, p.d) * sh.cluster, sh.cluster, sh.threads(), 0, s, p);
    };
    switch (sh.warps) {
        case 1: return go(norm_grad_kernel<TX, TF, 8, 1, 1, JOIN, false>, norm_grad_kernel<TX, TF, 1, 8, 1, JOIN, false>);
        case 2: return go(norm_grad_kernel<TX, TF, 8, 1, 2, JOIN, false>, norm_grad_kernel<TX, TF, 1, 8, 2, JOIN, false>);
        case 4: return go(norm_grad_kernel<TX, TF, 8, 1, 4, JOIN, false>, norm_grad_kernel<TX, TF, 1, 8, 4, JOIN, false>);
        case 8: return go(norm_grad_kernel<TX, TF, 8, 1, 8, JOIN, false>, norm_grad_kernel<TX, TF, 1, 8, 8, JOIN, false>);
        default: break;
    }
    if (sh.cluster == 1) return go(norm_grad_kernel<TX, TF, 8, 1, 16, JOIN, false>, norm_grad_kernel<TX, TF, 1, 8, 16, JOIN, false>);
    return go(norm_grad_kernel<TX, TF, 8, 1, 16, JOIN, true>, norm_grad_kernel<TX, TF, 1, 8, 16, JOIN, true>);
}

template <bool JOIN>
cudaError_t launch_grad(const NormGradParams &p, int x_dtype, int f_dtype, bool wide, cudaStream_t s) {
    if (x_dtype == RA_BF16) return launch_grad<uint16_t, uint16_t, JOIN>(p, wide, s);
    return f_dtype == RA_F32 ? launch_grad<float, float, JOIN>(p, wide, s) : launch_grad<float, uint16_t, JOIN>(p, wide, s);
}

}  // namespace
}  // namespace op
}  // namespace ra

extern "C" {

size_t ra_norm_block_grad_workspace_bytes(int64_t rows, int64_t d) {
    using namespace ra::op;
    if (!sizes_ok(rows, d) || rows == 0 || d == 0 || d > RA_NORM_MAX_D) return 0;
    return (size_t)(grad_parts(rows, d) * kVectors * d * 4);
}

ra_status ra_norm_block_grad(const ra_norm_block_grad_args *args, void *stream) {
    using namespace ra;
    using namespace ra::op;
    if (args == nullptr) return RA_ERR_INVALID_ARG;
    const ra_norm_block_grad_args &a = *args;
    if (!sizes_ok(a.rows, a.d) || !types_ok(a.x_dtype, a.f_dtype) || !side_ok(a.pre) || a.reserved != 0) return RA_ERR_INVALID_ARG;
    if (a.d == 0) return RA_OK;
    // an empty array has no address: without rows every part counts as there
    const bool none = a.rows == 0, join = a.f != nullptr || none, pre = a.pre.kind != RA_NORM_NONE;
    const int gate = join ? a.gate_kind : RA_GATE_NONE, ex = esize(a.x_dtype), ef = esize(a.f_dtype);
    if (join && (!side_ok(a.post) || gate < RA_GATE_NONE || gate > RA_GATE_MATRIX)) return RA_ERR_INVALID_ARG;
    const bool post = join && a.post.kind != RA_NORM_NONE, by_vector = gate == RA_GATE_VECTOR, by_matrix = gate == RA_GATE_MATRIX;
    if (by_vector && esize(a.gate_dtype) == 0) return RA_ERR_INVALID_ARG;
    if (!none && (pre != (a.dh != nullptr) || (!pre && a.dx_new == nullptr))) return RA_ERR_INVALID_ARG;
    // outputs of parts that the call does not have
    if ((!pre && (a.dpre_gain || a.dpre_bias)) || (!post && (a.dpost_gain || a.dpost_bias)) || (!join && a.df) || (gate == RA_GATE_NONE && a.dgate))
        return RA_ERR_INVALID_ARG;
    const int eg = by_vector ? esize(a.gate_dtype) : ef;
    const Mat dh{a.dh, pre ? a.rows : 0, a.d, a.ld_dh, ef}, dx_new{a.dx_new, a.dx_new ? a.rows : 0, a.d, a.ld_dx_new, ex}, x{a.x, pre ? a.rows : 0, a.d, a.ld_x, ex};
    const Mat f{a.f, join ? a.rows : 0, a.d, a.ld_f, ef}, gm{a.gate, by_matrix ? a.rows : by_vector ? 1 : 0, a.d, a.ld_gate, eg};
    const Mat kept{a.kept, pre || post ? a.rows : 0, 4, 4, 4};
    const Mat dx{a.dx, a.dx ? a.rows : 0, a.d, a.ld_dx, ex}, df{a.df, a.df ? a.rows : 0, a.d, a.ld_df, ef};
    const Mat dgate{a.dgate, a.dgate ? (by_matrix ? a.rows : 1) : 0, a.d, a.ld_dgate, by_matrix ? ef : 4};
    float *const vectors[kVectors] = {a.dpre_gain, a.dpre_bias, a.dpost_gain, a.dpost_bias, by_vector ? static_cast<float *>(a.dgate) : nullptr};
    const Mat all[] = {dh, dx_new, x, f, gm, kept, dx, df, dgate, vector_of(a.dpre_gain, a.d, 4), vector_of(a.dpre_bias, a.d, 4), vector_of(a.dpost_gain, a.d, 4),
                       vector_of(a.dpost_bias, a.d, 4)};
    for (const Mat &m : all)
        if (!mat_ok(m)) return RA_ERR_INVALID_ARG;
    if (!wide_at(a.kept)) return RA_ERR_INVALID_ARG;
    if (a.d > RA_NORM_MAX_D) return RA_ERR_UNSUPPORTED;
    bool sums = false;
    for (const float *v : vectors) sums = sums || v != nullptr;
    const size_t need = sums ? ra_norm_block_grad_workspace_bytes(a.rows, a.d) : 0;
    if (need > 0 && (a.ws == nullptr || !wide_at(a.ws) || a.ws_bytes < need)) return RA_ERR_INVALID_ARG;
    const Side behind = join ? side_of(a.post) : Side{}, ahead = side_of(a.pre);
    const Mat in[] = {dx_new, dh, x, f, gm, kept, vector_of(behind.gain, a.d, behind.f32 ? 4 : 2), vector_of(behind.bias, a.d, behind.f32 ? 4 : 2),
                      vector_of(ahead.gain, a.d, ahead.f32 ? 4 : 2), vector_of(ahead.bias, a.d, ahead.f32 ? 4 : 2)};
    const Mat out[] = {dx, df, dgate, all[9], all[10], all[11], all[12], Mat{a.ws, need ? 1 : 0, (int64_t)need, (int64_t)need, 1}};
    for (int o = 0; o < 8; ++o) {
        for (int i = 0; i < 10; ++i)
            if (mats_overlap(out[o], in[i]) && !(o == 0 && i == 0 && same_mat(dx, dx_new))) return RA_ERR_OVERLAP;
        for (int q = 0; q < o; ++q)
            if (mats_overlap(out[o], out[q])) return RA_ERR_OVERLAP;
    }
    const Mat rows[] = {dh, dx_new, x, f, dx, df, by_matrix ? gm : Mat{nullptr, 0, 0, 0, 4}, by_matrix ? dgate : Mat{nullptr, 0, 0, 0, 4}};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!none) {
        const NormGradParams p{a.dh, a.dx_new, a.x, a.f, a.gate, pre || post ? a.kept : nullptr, a.dx, a.df, by_matrix ? a.dgate : nullptr,
                               sums ? static_cast<float *>(a.ws) : nullptr, a.ld_dh, a.ld_dx_new, a.ld_x, a.ld_f, a.ld_gate, a.ld_dx, a.ld_df, a.ld_dgate, a.rows, a.d,
                               behind, ahead, gate, by_vector && a.gate_dtype == RA_F32, wide_at(a.gate), a.alpha, a.beta, 1.0f / (float)a.d};
        const bool wide = all_wide(rows, a.d);
        const cudaError_t e = join ? launch_grad<true>(p, a.x_dtype, a.f_dtype, wide, s) : launch_grad<false>(p, a.x_dtype, a.f_dtype, wide, s);
        if (e != cudaSuccess) return cuda_status(e);
    }
    if (!sums) return RA_OK;
    PartsParams q{static_cast<const float *>(a.ws), {}, none ? 0 : grad_parts(a.rows, a.d), a.d, join ? kVectors : 2, a.accumulate};
    for (int k = 0; k < kVectors; ++k) q.out[k] = vectors[k];
    return cuda_status(launch_pdl(parts_kernel, ceil_div<int64_t>(a.d, 32) * q.vectors, 256, 0, s, q));
}

}  // extern "C"
