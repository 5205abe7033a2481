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
    int64_t ld_x, ld_f, ld_gate, ld_x_out, ld_h, rows;
    int d, gate_kind;
    Side post, pre;
    bool gate_f32;
    float alpha, beta, per_d;  // per_d: 1 / d
};

// A row's threads keep their columns from row to row, 16 each, so that gains, biases
// and gate stay in their registers, and every value is read once: a row is held
// there from its first moment to its last product.  The next rows are on their way
// meanwhile (op_norm.cuh).  Memory bounds rows of 16-byte boundaries: 8192 x 2048 bf16
// with a join take 27 us (5.0 TB/s), 2048 x 8192 binary32 to bf16 without one 18 (5.7);
// what is left of the way to 20 and 15 is the sums over a row, one or two in turn, in
// 16 warps an SM.  Rows of odd lengths take 39 us (2047): one value an access.
constexpr int kOwn = 16;  // columns a thread has, in every row

// rows under way a group: as many as shared memory has room for in the widest blocks
template <class TX, class TF, bool JOIN>
constexpr int norm_stages() {
    return JOIN && sizeof(TF) == 4 ? 2 : 3;
}
// bytes a thread needs for a row
template <class TX, class TF, bool JOIN>
__host__ __device__ constexpr int norm_bytes(bool gate_matrix) {
    return kOwn * (int)(sizeof(TX) + (JOIN ? sizeof(TF) * (gate_matrix ? 2 : 1) : 0));
}

template <class TX, class TF, bool WIDE, int WARPS, bool JOIN, bool CLUSTER>
__global__ void __launch_bounds__(WARPS == 16 ? 512 : kNormThreads, WARPS == 16 ? 1 : 2) norm_kernel(const NormParams p) {
    constexpr int kThreads = WARPS == 16 ? 512 : kNormThreads, kGroups = kThreads / (WARPS * 32);  // kGroups: rows at a time
    constexpr int kAhead = norm_stages<TX, TF, JOIN>() - 1, kPairs = kOwn / 2;
    constexpr int kEach = each_of<TX, TF, WIDE>();
    constexpr bool kRing = WIDE && !CLUSTER;
    using C = Columns<kOwn, kEach, WARPS, CLUSTER>;
    __shared__ RowSums<WARPS, CLUSTER> sums[kGroups];
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_enter();
    if constexpr (CLUSTER) cluster_meet();  // every block is there before another writes to it
    const int id = threadIdx.x / (WARPS * 32);
    const C col(p.d);
    const int count = col.count();
    int turn = 0;
    const bool by_matrix = JOIN && p.gate_kind == RA_GATE_MATRIX;

    const int blocks = CLUSTER ? gridDim.x / cluster_blocks() : gridDim.x, block = CLUSTER ? blockIdx.x / cluster_blocks() : blockIdx.x;
    // (below 2^31 rows: no sum of these wraps)
    const uint32_t first = block * kGroups + id, step = blocks * kGroups, last = (uint32_t)p.rows;
    // a stage: f, the gate, x; the threads' pieces of each side by side
    constexpr int kRowF = kOwn * (int)sizeof(TF) * kThreads, kRowX = kOwn * (int)sizeof(TX) * kThreads;
    const int stage_bytes = norm_bytes<TX, TF, JOIN>(by_matrix) * kThreads;
    const uint32_t base = smem_addr(ring), mine_f = base + threadIdx.x * kEach * (int)sizeof(TF), mine_x = base + stage_bytes - kRowX + threadIdx.x * kEach * (int)sizeof(TX);
    auto fetch = [&](uint32_t r, int stage) {
        if (r < last) {
            const int to = stage * stage_bytes;
            if constexpr (JOIN) {
                copy_own(mine_f + to, kThreads, row_of_matrix<WIDE>(static_cast<const TF *>(p.f), p.ld_f, r), col, count);
                if (by_matrix) copy_own(mine_f + to + kRowF, kThreads, row_of_matrix<WIDE>(static_cast<const TF *>(p.gate), p.ld_gate, r), col, count);
            }
            copy_own(mine_x + to, kThreads, row_of_matrix<WIDE>(static_cast<const TX *>(p.x), p.ld_x, r), col, count);
        }
        copies_done();
    };
    auto cache = [&](uint32_t r) {
        if (WARPS == 1 || r >= last) return;
        cache_own(row_of_matrix<WIDE>(static_cast<const TX *>(p.x), p.ld_x, r), col);
        if constexpr (JOIN) {
            cache_own(row_of_matrix<WIDE>(static_cast<const TF *>(p.f), p.ld_f, r), col);
            if (by_matrix) cache_own(row_of_matrix<WIDE>(static_cast<const TF *>(p.gate), p.ld_gate, r), col);
        }
    };
    int stage = 0;
    if constexpr (kRing) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(first + k * step, k);
    } else {
        cache(first + step);
    }

    // post as (v - m) rstd a + b with the gate and beta in a and b, unless the gate
    // has a value of its own for each v
    Pair a_post[JOIN ? kPairs : 1], b_post[JOIN ? kPairs : 1], a_pre[kPairs], b_pre[kPairs];
    {
        float a[kOwn], b[kOwn];
        if constexpr (JOIN) {
            float g[kOwn];
            load_param(p.post.gain, p.post.f32, col, count, 1.0f, a);
            load_param(p.post.bias, p.post.f32, col, count, 0.0f, b);
            load_param(p.gate_kind == RA_GATE_VECTOR ? p.gate : nullptr, p.gate_f32, col, count, 1.0f, g);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                a_post[j] = pair(a[2 * j] * (p.beta * g[2 * j]), a[2 * j + 1] * (p.beta * g[2 * j + 1]));
                b_post[j] = pair(b[2 * j] * (p.beta * g[2 * j]), b[2 * j + 1] * (p.beta * g[2 * j + 1]));
            }
        }
        load_param(p.pre.gain, p.pre.f32, col, count, 1.0f, a);
        load_param(p.pre.bias, p.pre.f32, col, count, 0.0f, b);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            a_pre[j] = pair(a[2 * j], a[2 * j + 1]);
            b_pre[j] = pair(b[2 * j], b[2 * j + 1]);
        }
    }

    // m and rstd of a row.  The sums of the values and of their squares are made at
    // once; where the mean is so large that their difference loses more than 4
    // bits, or the squares leave binary32, the squares of the differences from it are
    // summed after it.
    auto moments = [&](const Pair (&v)[kPairs], const Side &side, float *m, float *rstd) {
        Pair sum = both(0.0f), squares = both(0.0f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {  // columns past the row's end hold 0
            sum = pair_add(sum, v[j]);
            squares = pair_fma(v[j], v[j], squares);
        }
        float s[2] = {pair_sum(sum), pair_sum(squares)};
        row_sum(s, sums[id], id, turn);
        *m = 0.0f;
        float var = s[1] * p.per_d;
        if (side.kind == RA_NORM_LAYER) {
            *m = s[0] * p.per_d;
            const float left = fmaf(-*m, *m, var);
            if (!(left * 16.0f >= var && var < INFINITY) && var > 0.0f) {  // the same for the whole row
                s[0] = s[1] = 0.0f;
#pragma unroll
                for (int j = 0; j < kOwn; ++j) {
                    float a, b;
                    apart(v[j / 2], a, b);
                    const float c = (j & 1 ? b : a) - *m;
                    if (j < count) s[0] = fmaf(c, c, s[0]);
                }
                row_sum(s, sums[id], id, turn);
                var = s[0] * p.per_d;
            } else {
                var = left;
            }
        }
        *rstd = rsqrtf(var + side.eps);
    };

    for (uint32_t r = first; r < last; r += step) {
        Own<TX, C> x;
        Own<TF, C> f, g;
        const int at = stage * stage_bytes;
        if constexpr (kRing) {
            fetch(r + kAhead * step, stage == 0 ? kAhead : stage - 1);
            await_copies<kAhead>();
            if constexpr (JOIN) f.take(mine_f + at, kThreads, count);
            stage = stage == kAhead ? 0 : stage + 1;
        } else {
            cache(r + 2 * step);
            x.load(row_of_matrix<WIDE>(static_cast<const TX *>(p.x), p.ld_x, r), col, count);
            if constexpr (JOIN) {
                f.load(row_of_matrix<WIDE>(static_cast<const TF *>(p.f), p.ld_f, r), col, count);
                if (by_matrix) g.load(row_of_matrix<WIDE>(static_cast<const TF *>(p.gate), p.ld_gate, r), col, count);
            }
        }
        Pair v[kPairs];
        float m_f = 0.0f, rstd_f = 0.0f, m_x = 0.0f, rstd_x = 0.0f;
        if constexpr (JOIN) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) v[j] = f.two(j);
            const bool normed = p.post.kind != RA_NORM_NONE;
            if (normed) moments(v, p.post, &m_f, &rstd_f);
            if constexpr (kRing) {
                if (by_matrix) g.take(mine_f + at + kRowF, kThreads, count);
                x.take(mine_x + at, kThreads, count);
            }
            const Pair scale = both(normed ? rstd_f : 1.0f), off = both(-m_f), alpha = both(p.alpha);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                v[j] = pair_fma(pair_add(v[j], off), pair_mul(scale, a_post[j]), b_post[j]);
                if (by_matrix) v[j] = pair_mul(v[j], g.two(j));
                v[j] = pair_fma(alpha, x.two(j), v[j]);
            }
            x.set(v);
            x.store(row_of_matrix<WIDE>(static_cast<TX *>(p.x_out), p.ld_x_out, r), col, count);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {  // the norm is that of the row as stored
                v[j] = x.two(j);
                if (!WIDE || kOwn > 8) v[j] = pair(2 * j < count ? x[2 * j] : 0.0f, 2 * j + 1 < count ? x[2 * j + 1] : 0.0f);
            }
        } else {
            if constexpr (kRing) x.take(mine_x + at, kThreads, count);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) v[j] = x.two(j);
        }
        if (p.pre.kind != RA_NORM_NONE) {
            moments(v, p.pre, &m_x, &rstd_x);
            const Pair scale = both(rstd_x), off = both(-m_x);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) v[j] = pair_fma(pair_add(v[j], off), pair_mul(scale, a_pre[j]), b_pre[j]);
            f.set(v);
            f.store(row_of_matrix<WIDE>(static_cast<TF *>(p.h), p.ld_h, r), col, count);
        }
        if (p.kept != nullptr && col.first == 0) reinterpret_cast<float4 *>(p.kept)[r] = make_float4(m_f, rstd_f, m_x, rstd_x);
    }
}

template <class TX, class TF, bool JOIN>
cudaError_t launch_norm(const NormParams &p, bool wide, cudaStream_t s) {
    const Shape sh(p.d, kOwn);
    return with_shape(sh, [&](auto warps, auto cluster) {
        constexpr int kWarps = decltype(warps)::value;
        constexpr bool kCluster = decltype(cluster)::value != 0;
        const int64_t grid = sh.shares(p.rows) * sh.cluster;
        if (!wide) return launch_clusters(norm_kernel<TX, TF, false, kWarps, JOIN, kCluster>, grid, sh.cluster, sh.threads(), 0, s, p);
        const int rows = kCluster ? 0 : norm_stages<TX, TF, JOIN>() * sh.threads();
        const cudaError_t e = opt_in_smem<norm_kernel<TX, TF, true, kWarps, JOIN, kCluster>>(rows * norm_bytes<TX, TF, JOIN>(JOIN));
        if (e != cudaSuccess) return e;
        return launch_clusters(norm_kernel<TX, TF, true, kWarps, JOIN, kCluster>, grid, sh.cluster, sh.threads(),
                               rows * norm_bytes<TX, TF, JOIN>(p.gate_kind == RA_GATE_MATRIX), s, p);
    });
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
    const NormParams p{a.x, a.f, a.gate, a.x_out, a.h, a.kept, a.ld_x, a.ld_f, a.ld_gate, a.ld_x_out, a.ld_h, a.rows, (int)a.d, gate, post, ahead,
                       gate == RA_GATE_VECTOR && a.gate_dtype == RA_F32, a.alpha, a.beta, 1.0f / (float)a.d};
    const bool wide = all_wide(rows, a.d);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(join ? launch_norm<true>(p, a.x_dtype, a.f_dtype, wide, s) : launch_norm<false>(p, a.x_dtype, a.f_dtype, wide, s));
}
