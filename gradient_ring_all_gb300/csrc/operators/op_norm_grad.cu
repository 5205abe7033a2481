// op_norm_grad.cu -- the gradients of the join behind a block and of the norm
// before the next one: ra_norm_block_grad.
#include "op_norm.cuh"

namespace ra {
namespace op {
namespace {

enum { kPreGain, kPreBias, kPostGain, kPostBias, kGate, kVectors };

// A thread's values of a vector of parameters, read anew for each row (from L1): in
// registers they would leave no room for the sums.
template <bool WIDE, class C>
__device__ __forceinline__ void load_vector(const void *v, bool f32, const C &col, int count, float none, float (&out)[kOwn]) {
    if (v != nullptr && count > 0 && WIDE && reinterpret_cast<uintptr_t>(v) % 16 == 0) {
        if (f32)
            load_w<float, kOwn>(static_cast<const float *>(v) + col.first, out);
        else
            load_w<uint16_t, kOwn>(static_cast<const uint16_t *>(v) + col.first, out);
    } else {
        load_param(v, f32, col, count, none, out);
    }
}
template <bool WIDE, int WARPS, bool CLUSTER>
__device__ __forceinline__ void load_gain(const Side &side, const Columns<WIDE, WARPS, CLUSTER> &col, int count, float (&out)[kOwn]) {
    load_vector<WIDE>(side.gain, side.f32, col, count, 1.0f, out);
}

struct NormGradParams {
    const void *dh, *dx_new, *x, *f, *gate;
    const float *kept;
    void *dx, *df, *dgate;  // dgate: a matrix's
    float *parts;           // shares x (kVectors or 2) x d, or null
    int64_t ld_dh, ld_dx_new, ld_x, ld_f, ld_gate, ld_dx, ld_df, ld_dgate, rows;
    int d, gate_kind;
    Side post, pre;
    bool gate_f32;
    float alpha, beta, per_d;
};

// rows under way a group
template <class TX, class TF>
constexpr int grad_stages() {
    return sizeof(TF) == 4 ? 2 : 3;
}
// 16-byte places a thread needs for a row: dh, x, dx_new, f, the gate, kept
template <class TX, class TF, bool JOIN>
__host__ __device__ constexpr int grad_places(bool gate_matrix) {
    return 1 + places<TF>() * ((JOIN ? 2 : 1) + (gate_matrix ? 1 : 0)) + 2 * places<TX>();
}

template <class TX, class TF, bool WIDE, int WARPS, bool JOIN, bool CLUSTER>
__global__ void __launch_bounds__(WARPS == 16 ? 512 : kNormThreads, WARPS == 16 ? 1 : 2) norm_grad_kernel(const NormGradParams p) {
    constexpr int kThreads = WARPS == 16 ? 512 : kNormThreads, kGroups = kThreads / (WARPS * 32), kSums = JOIN ? kVectors : 2;
    constexpr int kPitch = kThreads * 16, kAhead = grad_stages<TX, TF>() - 1;
    __shared__ RowSums<2, WARPS, CLUSTER> sums[kGroups];
    __shared__ float joined[kGroups > 1 ? WARPS * 32 * kOwn : 1];
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_enter();
    if constexpr (CLUSTER) cluster_meet();
    const int id = threadIdx.x / (WARPS * 32);
    const Columns<WIDE, WARPS, CLUSTER> col;
    const int count = col.count(p.d);
    int turn = 0;
    const bool by_matrix = JOIN && p.gate_kind == RA_GATE_MATRIX, has_pre = p.dh != nullptr, has_new = p.dx_new != nullptr;
    const bool normed = p.post.kind != RA_NORM_NONE;

    float acc[kSums][kOwn];
#pragma unroll
    for (int a = 0; a < kSums; ++a)
#pragma unroll
        for (int j = 0; j < kOwn; ++j) acc[a][j] = 0.0f;

    const int blocks = CLUSTER ? gridDim.x / cluster_blocks() : gridDim.x, block = CLUSTER ? blockIdx.x / cluster_blocks() : blockIdx.x;
    const int64_t first = (int64_t)block * kGroups + id, step = (int64_t)blocks * kGroups;
    const int stage_bytes = grad_places<TX, TF, JOIN>(by_matrix) * kPitch;
    const uint32_t mine = smem_addr(ring) + threadIdx.x * 16;
    auto fetch = [&](int64_t r, int stage) {
        if (r < p.rows && count > 0) {
            uint32_t to = mine + stage * stage_bytes;
            if (p.kept != nullptr) copy_own(to, kPitch, reinterpret_cast<const uint16_t *>(p.kept + r * 4));
            to += kPitch;
            if (has_pre) {
                copy_own(to, kPitch, static_cast<const TF *>(p.dh) + r * p.ld_dh + col.first);
                copy_own(to + places<TF>() * kPitch, kPitch, static_cast<const TX *>(p.x) + r * p.ld_x + col.first);
            }
            to += (places<TF>() + places<TX>()) * kPitch;
            if (has_new) copy_own(to, kPitch, static_cast<const TX *>(p.dx_new) + r * p.ld_dx_new + col.first);
            to += places<TX>() * kPitch;
            if constexpr (JOIN) {
                to = copy_own(to, kPitch, static_cast<const TF *>(p.f) + r * p.ld_f + col.first);
                if (by_matrix) copy_own(to, kPitch, static_cast<const TF *>(p.gate) + r * p.ld_gate + col.first);
            }
        }
        copies_done();
    };
    int stage = 0;
    if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(first + k * step, k);
    }
    for (int64_t r = first; r < p.rows; r += step) {
        Own<TX, WIDE> x, d;
        Own<TF, WIDE> h, f, g;
        float4 kept = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        uint32_t at = mine + stage * stage_bytes + kPitch;
        if constexpr (WIDE) {
            fetch(r + kAhead * step, stage == 0 ? kAhead : stage - 1);
            await_copies<kAhead>();
            h.zero();
            x.zero();
            if (count > 0) {
                if (p.kept != nullptr)
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(kept.x), "=f"(kept.y), "=f"(kept.z), "=f"(kept.w) : "r"(at - kPitch) : "memory");
                if (has_pre) {
                    h.take(at, kPitch);
                    x.take(at + places<TF>() * kPitch, kPitch);
                }
            }
            at += (places<TF>() + places<TX>()) * kPitch;
            stage = stage == kAhead ? 0 : stage + 1;
        } else {
            if (p.kept != nullptr) kept = reinterpret_cast<const float4 *>(p.kept)[r];
            h.zero();
            x.zero();
            if (has_pre) {
                h.load(static_cast<const TF *>(p.dh) + r * p.ld_dh, col, count);
                x.load(static_cast<const TX *>(p.x) + r * p.ld_x, col, count);
            }
            d.zero();
            if (has_new) d.load(static_cast<const TX *>(p.dx_new) + r * p.ld_dx_new, col, count);
            if constexpr (JOIN) {
                f.load(static_cast<const TF *>(p.f) + r * p.ld_f, col, count);
                if (by_matrix) g.load(static_cast<const TF *>(p.gate) + r * p.ld_gate, col, count);
            }
        }
        float full[kOwn], by_unit = 0.0f, plain = 0.0f;
        if (has_pre) {
            float s[2] = {0.0f, 0.0f}, gain[kOwn];
            load_gain(p.pre, col, count, gain);
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {  // columns past the row's end: h and x are 0, and so is what they add
                const float unit = (x[j] - kept.z) * kept.w;
                full[j] = h[j] * gain[j];
                s[0] = fmaf(full[j], unit, s[0]);
                s[1] += full[j];
                acc[kPreGain][j] = fmaf(h[j], unit, acc[kPreGain][j]);
                acc[kPreBias][j] += h[j];
            }
            row_sum(s, sums[id], id, turn);
            by_unit = s[0] * p.per_d;
            plain = p.pre.kind == RA_NORM_LAYER ? s[1] * p.per_d : 0.0f;
        }
        if constexpr (WIDE) {
            d.zero();
            if (count > 0) {
                if (has_new) d.take(at, kPitch);
                if constexpr (JOIN) {
                    f.take(at + places<TX>() * kPitch, kPitch);
                    if (by_matrix) g.take(at + (places<TX>() + places<TF>()) * kPitch, kPitch);
                }
            } else if constexpr (JOIN) {
                f.zero();
            }
        }
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            full[j] = has_pre ? fmaf(kept.w, full[j] - plain - (x[j] - kept.z) * kept.w * by_unit, d[j]) : d[j];
        if (p.dx != nullptr) {
            float y[kOwn];
#pragma unroll
            for (int j = 0; j < kOwn; ++j) y[j] = JOIN ? p.alpha * full[j] : full[j];
            store_own<TX, WIDE>(static_cast<TX *>(p.dx) + r * p.ld_dx, col, count, y);
        }
        if constexpr (JOIN) {
            float s[2] = {0.0f, 0.0f}, gain[kOwn], bias[kOwn], gate[kOwn], dg[kOwn];
            if (normed) {
                load_gain(p.post, col, count, gain);
            } else {
                kept.x = 0.0f;
                kept.y = 1.0f;
#pragma unroll
                for (int j = 0; j < kOwn; ++j) gain[j] = 1.0f;
            }
            load_vector<WIDE>(normed ? p.post.bias : nullptr, p.post.f32, col, count, 0.0f, bias);
            load_vector<WIDE>(p.gate_kind == RA_GATE_VECTOR ? p.gate : nullptr, p.gate_f32, col, count, 1.0f, gate);
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                if (!WIDE && j >= count) full[j] = 0.0f;
                const float unit = (f[j] - kept.x) * kept.y, u = p.beta * full[j];
                dg[j] = u * fmaf(unit, gain[j], bias[j]);
                acc[kGate][j] += dg[j];
                const float v = u * (by_matrix ? g[j] : gate[j]);
                acc[kPostGain][j] = fmaf(v, unit, acc[kPostGain][j]);
                acc[kPostBias][j] += v;
                full[j] = v * gain[j];
                s[0] = fmaf(full[j], unit, s[0]);
                s[1] += full[j];
            }
            if (p.dgate != nullptr) store_own<TF, WIDE>(static_cast<TF *>(p.dgate) + r * p.ld_dgate, col, count, dg);
            if (normed) {
                if (WIDE && count == 0) s[0] = s[1] = 0.0f;
                row_sum(s, sums[id], id, turn);
                by_unit = s[0] * p.per_d;
                plain = p.post.kind == RA_NORM_LAYER ? s[1] * p.per_d : 0.0f;
#pragma unroll
                for (int j = 0; j < kOwn; ++j) full[j] = kept.y * (full[j] - plain - (f[j] - kept.x) * kept.y * by_unit);
            }
            if (p.df != nullptr) store_own<TF, WIDE>(static_cast<TF *>(p.df) + r * p.ld_df, col, count, full);
        }
    }

    if (p.parts == nullptr) return;
    float *const part = p.parts + (int64_t)block * kSums * p.d;
#pragma unroll
    for (int a = 0; a < kSums; ++a) {
        if constexpr (kGroups > 1) {  // the groups' sums in their order
            for (int k = 0; k < kGroups; ++k) {
                __syncthreads();
                if (id != k) continue;
#pragma unroll
                for (int j = 0; j < kOwn; ++j) {
                    float &to = joined[col[j]];
                    to = k == 0 ? acc[a][j] : to + acc[a][j];
                }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.d; c += kThreads) part[(int64_t)a * p.d + c] = joined[c];
        } else if constexpr (WIDE) {
            if (count > 0) store_w<float, kOwn>(part + (int64_t)a * p.d + col.first, acc[a]);
        } else {
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
                if (j < count) part[(int64_t)a * p.d + col[j]] = acc[a][j];
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

// blocks (or clusters) that share the rows, each with a part of the sums
int64_t grad_parts(int64_t rows, int64_t d) { return Shape(d).shares(rows, 2); }

template <class TX, class TF, bool JOIN>
cudaError_t launch_grad(const NormGradParams &p, bool wide, cudaStream_t s) {
    const Shape sh(p.d);
    return with_shape(sh, [&](auto warps, auto cluster) {
        constexpr int kWarps = decltype(warps)::value;
        constexpr bool kCluster = decltype(cluster)::value != 0;
        const int64_t grid = grad_parts(p.rows, p.d) * sh.cluster;
        if (!wide) return launch_clusters(norm_grad_kernel<TX, TF, false, kWarps, JOIN, kCluster>, grid, sh.cluster, sh.threads(), 0, s, p);
        const int place = grad_stages<TX, TF>() * 16 * sh.threads();
        const cudaError_t e = opt_in_smem<norm_grad_kernel<TX, TF, true, kWarps, JOIN, kCluster>>(place * grad_places<TX, TF, JOIN>(JOIN));
        if (e != cudaSuccess) return e;
        return launch_clusters(norm_grad_kernel<TX, TF, true, kWarps, JOIN, kCluster>, grid, sh.cluster, sh.threads(),
                               place * grad_places<TX, TF, JOIN>(p.gate_kind == RA_GATE_MATRIX), s, p);
    });
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
                               sums ? static_cast<float *>(a.ws) : nullptr, a.ld_dh, a.ld_dx_new, a.ld_x, a.ld_f, a.ld_gate, a.ld_dx, a.ld_df, a.ld_dgate, a.rows, (int)a.d,
                               gate, behind, ahead, by_vector && a.gate_dtype == RA_F32, a.alpha, a.beta, 1.0f / (float)a.d};
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
