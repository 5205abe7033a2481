// op_norm_grad.cu -- the gradients of the join behind a block and of the norm
// before the next one: ra_norm_block_grad.
#include "op_norm.cuh"

namespace ra {
namespace op {
namespace {

// As forward, a row's threads keep their columns from row to row, here also for the
// sums over the rows, which stay in their registers until the block leaves them as
// its part; parts_kernel adds the parts.  16 columns a thread would need 64 registers
// for the sums alone, so there are 8, and 122 registers, 16 warps an SM.  8192 x 2048
// bf16 take 58 us (30 at the copy's rate): about 49 in rows and 9 in parts.  Neither
// memory (46 % busy) nor issue (41 %) bounds the rows but their two sums in turn, of
// which the second needs the first, in so few warps.
constexpr int kOwn = 8;  // columns a thread has, in every row: their sums stay in its registers

// What is summed over the rows, with v and w the normed x' and f and D the whole
// gradient of x': dh v, dh, and D w, D (with a matrix's gate: D gate w, D gate).  The
// gradients of post's gain and bias, and of a vector's gate, follow from the last
// two, as the gate and beta are the same for all rows of a column.
enum { kDhUnit, kDh, kDUnit, kD, kSumsMost };

// A thread's values of a vector of parameters.
template <class C>
__device__ __forceinline__ void load_vector(const void *v, bool f32, const C &col, int count, float none, float (&out)[kOwn]) {
    if (v != nullptr && count == kOwn && C::kEach > 1 && reinterpret_cast<uintptr_t>(v) % 16 == 0) {
#pragma unroll
        for (int i = 0; i < C::kParts; ++i) {
            float w[C::kEach];
            if (f32)
                load_w<float, C::kEach>(static_cast<const float *>(v) + col[i * C::kEach], w);
            else
                load_w<uint16_t, C::kEach>(static_cast<const uint16_t *>(v) + col[i * C::kEach], w);
#pragma unroll
            for (int j = 0; j < C::kEach; ++j) out[i * C::kEach + j] = w[j];
        }
    } else {
        load_param(v, f32, col, count, none, out);
    }
}

struct NormGradParams {
    const void *dh, *dx_new, *x, *f, *gate;
    const float *kept;
    void *dx, *df, *dgate;  // dgate: a matrix's
    float *parts;           // shares x (kSumsMost or 2) x d, or null
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
// bytes a thread needs for a row: kept, dh, x, dx_new, f, the gate
template <class TX, class TF, bool JOIN>
__host__ __device__ constexpr int grad_bytes(bool gate_matrix) {
    return 16 + kOwn * (int)(sizeof(TF) * ((JOIN ? 2 : 1) + (gate_matrix ? 1 : 0)) + 2 * sizeof(TX));
}

template <class TX, class TF, bool WIDE, int WARPS, bool JOIN, bool CLUSTER>
__global__ void __launch_bounds__(WARPS == 16 ? 512 : kNormThreads, WARPS == 16 ? 1 : 2) norm_grad_kernel(const NormGradParams p) {
    constexpr int kThreads = WARPS == 16 ? 512 : kNormThreads, kGroups = kThreads / (WARPS * 32), kSums = JOIN ? kSumsMost : 2;
    constexpr int kAhead = grad_stages<TX, TF>() - 1, kPairs = kOwn / 2;
    constexpr int kEach = each_of<TX, TF, WIDE>();
    constexpr bool kRing = WIDE && !CLUSTER;
    using C = Columns<kOwn, kEach, WARPS, CLUSTER>;
    __shared__ RowSums<WARPS, CLUSTER> sums[kGroups];
    __shared__ float joined[kGroups > 1 ? WARPS * 32 * kOwn : 1];
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_enter();
    if constexpr (CLUSTER) cluster_meet();
    const int id = threadIdx.x / (WARPS * 32);
    const C col(p.d);
    const int count = col.count();
    int turn = 0;
    const bool by_matrix = JOIN && p.gate_kind == RA_GATE_MATRIX, has_pre = p.dh != nullptr, has_new = p.dx_new != nullptr;
    const bool normed = JOIN && p.post.kind != RA_NORM_NONE;

    const int blocks = CLUSTER ? gridDim.x / cluster_blocks() : gridDim.x, block = CLUSTER ? blockIdx.x / cluster_blocks() : blockIdx.x;
    // (below 2^31 rows: no sum of these wraps)
    const uint32_t first = block * kGroups + id, step = blocks * kGroups, last = (uint32_t)p.rows;
    // a stage: kept, dh, x, dx_new, f, the gate; the threads' pieces of each side by side
    constexpr int kRowF = kOwn * (int)sizeof(TF) * kThreads, kRowX = kOwn * (int)sizeof(TX) * kThreads;
    constexpr int kAtDh = 16 * kThreads, kAtX = kAtDh + kRowF, kAtNew = kAtX + kRowX, kAtF = kAtNew + kRowX, kAtGate = kAtF + kRowF;
    const int stage_bytes = grad_bytes<TX, TF, JOIN>(by_matrix) * kThreads;
    const uint32_t base = smem_addr(ring), mine = base + threadIdx.x * 16, mine_f = base + threadIdx.x * kEach * (int)sizeof(TF),
                   mine_x = base + threadIdx.x * kEach * (int)sizeof(TX);
    auto fetch = [&](uint32_t r, int stage) {
        if (r < last) {
            const int to = stage * stage_bytes;
            if (p.kept != nullptr) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + to), "l"(p.kept + (int64_t)r * 4) : "memory");
            if (has_pre) {
                copy_own(mine_f + to + kAtDh, kThreads, row_of_matrix<WIDE>(static_cast<const TF *>(p.dh), p.ld_dh, r), col, count);
                copy_own(mine_x + to + kAtX, kThreads, row_of_matrix<WIDE>(static_cast<const TX *>(p.x), p.ld_x, r), col, count);
            }
            if (has_new) copy_own(mine_x + to + kAtNew, kThreads, row_of_matrix<WIDE>(static_cast<const TX *>(p.dx_new), p.ld_dx_new, r), col, count);
            if constexpr (JOIN) {
                copy_own(mine_f + to + kAtF, kThreads, row_of_matrix<WIDE>(static_cast<const TF *>(p.f), p.ld_f, r), col, count);
                if (by_matrix) copy_own(mine_f + to + kAtGate, kThreads, row_of_matrix<WIDE>(static_cast<const TF *>(p.gate), p.ld_gate, r), col, count);
            }
        }
        copies_done();
    };
    auto cache = [&](uint32_t r) {
        if (WARPS == 1 || r >= last) return;
        if (has_pre) {
            cache_own(row_of_matrix<WIDE>(static_cast<const TF *>(p.dh), p.ld_dh, r), col);
            cache_own(row_of_matrix<WIDE>(static_cast<const TX *>(p.x), p.ld_x, r), col);
        }
        if (has_new) cache_own(row_of_matrix<WIDE>(static_cast<const TX *>(p.dx_new), p.ld_dx_new, r), col);
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
        cache(first);
        cache(first + step);
    }

    // pre's gain; and beta times the gate times post's gain (without a matrix's gate)
    Pair gain[kPairs], back[JOIN ? kPairs : 1], acc[kSums][kPairs];
    {
        float a[kOwn], b[kOwn];
        load_vector(p.pre.gain, p.pre.f32, col, count, 1.0f, a);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) gain[j] = pair(a[2 * j], a[2 * j + 1]);
        if constexpr (JOIN) {
            load_vector(p.post.gain, p.post.f32, col, count, 1.0f, a);
            load_vector(p.gate_kind == RA_GATE_VECTOR ? p.gate : nullptr, p.gate_f32, col, count, 1.0f, b);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) back[j] = pair(p.beta * b[2 * j] * a[2 * j], p.beta * b[2 * j + 1] * a[2 * j + 1]);
        }
    }
#pragma unroll
    for (int a = 0; a < kSums; ++a)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) acc[a][j] = both(0.0f);

    for (uint32_t r = first; r < last; r += step) {
        Own<TX, C> x;
        Own<TF, C> h;
        float4 kept = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int at = stage * stage_bytes;
        if constexpr (kRing) {
            fetch(r + kAhead * step, stage == 0 ? kAhead : stage - 1);
            await_copies<kAhead>();
            if (p.kept != nullptr) asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(kept.x), "=f"(kept.y), "=f"(kept.z), "=f"(kept.w) : "r"(mine + at) : "memory");
            stage = stage == kAhead ? 0 : stage + 1;
        } else {
            cache(r + 2 * step);
            if (p.kept != nullptr) kept = reinterpret_cast<const float4 *>(p.kept)[r];
        }
        // the rest of a row's values, where they are needed
        auto read = [&](auto &to, const auto *from, int64_t ld, int place) {
            if constexpr (kRing)
                to.take((place == kAtX || place == kAtNew ? mine_x : mine_f) + at + place, kThreads, count);
            else
                to.load(row_of_matrix<WIDE>(from, ld, r), col, count);
        };
        // Columns past the row's end hold 0, and add 0 to the sums; but where m rstd is no
        // binary32 number (huge equal values) their units would be infinite: 0 then.
        auto no_units = [&](Pair (&unit)[kPairs], float m, float rstd) {
            if (fabsf(m) * rstd > 3.402823466e38f) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    float a, b;
                    apart(unit[j], a, b);
                    unit[j] = pair(2 * j < count ? a : 0.0f, 2 * j + 1 < count ? b : 0.0f);
                }
            }
        };

        Pair full[kPairs];
        {
            Pair unit[kPairs], by_unit = both(0.0f), plain = both(0.0f);
            if (has_pre) {
                read(h, static_cast<const TF *>(p.dh), p.ld_dh, kAtDh);
                read(x, static_cast<const TX *>(p.x), p.ld_x, kAtX);
                const Pair off = both(-kept.z), scale = both(kept.w);
                Pair s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) unit[j] = pair_mul(pair_add(x.two(j), off), scale);
                no_units(unit, kept.z, kept.w);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const Pair dh = h.two(j);
                    full[j] = pair_mul(dh, gain[j]);
                    s0 = pair_fma(full[j], unit[j], s0);
                    s1 = pair_add(s1, full[j]);
                    acc[kDhUnit][j] = pair_fma(dh, unit[j], acc[kDhUnit][j]);
                    acc[kDh][j] = pair_add(acc[kDh][j], dh);
                }
                float s[2] = {pair_sum(s0), pair_sum(s1)};
                row_sum(s, sums[id], id, turn);
                by_unit = both(-s[0] * p.per_d);
                plain = both(p.pre.kind == RA_NORM_LAYER ? -s[1] * p.per_d : 0.0f);
            }
            Own<TX, C> d;
            if (has_new) {
                read(d, static_cast<const TX *>(p.dx_new), p.ld_dx_new, kAtNew);
            } else {
#pragma unroll
                for (int i = 0; i < C::kParts; ++i) d.v[i].zero();
            }
            const Pair scale = both(kept.w);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) full[j] = has_pre ? pair_fma(pair_fma(unit[j], by_unit, pair_add(full[j], plain)), scale, d.two(j)) : d.two(j);
        }
        if (p.dx != nullptr) {
            const Pair alpha = both(JOIN ? p.alpha : 1.0f);
            Pair y[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) y[j] = pair_mul(full[j], alpha);
            x.set(y);
            x.store(row_of_matrix<WIDE>(static_cast<TX *>(p.dx), p.ld_dx, r), col, count);
        }
        if constexpr (JOIN) {
            Own<TF, C> f;
            read(f, static_cast<const TF *>(p.f), p.ld_f, kAtF);
            Pair unit[kPairs], s0 = both(0.0f), s1 = both(0.0f);
            const Pair off = both(normed ? -kept.x : 0.0f), scale = both(normed ? kept.y : 1.0f);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) unit[j] = pair_mul(pair_add(f.two(j), off), scale);
            no_units(unit, kept.x, kept.y);
            if (by_matrix) {
                float a[kOwn], b[kOwn];
                load_vector(p.post.gain, p.post.f32, col, count, 1.0f, a);
                load_vector(p.post.bias, p.post.f32, col, count, 0.0f, b);
                Own<TF, C> g;
                read(g, static_cast<const TF *>(p.gate), p.ld_gate, kAtGate);
                const Pair beta = both(p.beta);
                Pair dg[kPairs];
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    dg[j] = pair_mul(pair_mul(beta, full[j]), pair_fma(unit[j], pair(a[2 * j], a[2 * j + 1]), pair(b[2 * j], b[2 * j + 1])));
                    full[j] = pair_mul(full[j], g.two(j));
                }
                if (p.dgate != nullptr) {
                    g.set(dg);
                    g.store(row_of_matrix<WIDE>(static_cast<TF *>(p.dgate), p.ld_dgate, r), col, count);
                }
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                if (count < kOwn) {
                    float a, b;
                    apart(full[j], a, b);
                    full[j] = pair(2 * j < count ? a : 0.0f, 2 * j + 1 < count ? b : 0.0f);
                }
                acc[kDUnit][j] = pair_fma(full[j], unit[j], acc[kDUnit][j]);
                acc[kD][j] = pair_add(acc[kD][j], full[j]);
                full[j] = pair_mul(full[j], back[j]);
                s0 = pair_fma(full[j], unit[j], s0);
                s1 = pair_add(s1, full[j]);
            }
            if (normed) {
                float s[2] = {pair_sum(s0), pair_sum(s1)};
                row_sum(s, sums[id], id, turn);
                const Pair by_unit = both(-s[0] * p.per_d), plain = both(p.post.kind == RA_NORM_LAYER ? -s[1] * p.per_d : 0.0f);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) full[j] = pair_mul(pair_fma(unit[j], by_unit, pair_add(full[j], plain)), scale);
            }
            if (p.df != nullptr) {
                f.set(full);
                f.store(row_of_matrix<WIDE>(static_cast<TF *>(p.df), p.ld_df, r), col, count);
            }
        }
    }

    if (p.parts == nullptr) return;
    float *const part = p.parts + (int64_t)block * kSums * p.d;
#pragma unroll
    for (int a = 0; a < kSums; ++a) {
        float v[kOwn];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) apart(acc[a][j], v[2 * j], v[2 * j + 1]);
        if constexpr (kGroups > 1) {  // the groups' sums in their order
            for (int k = 0; k < kGroups; ++k) {
                __syncthreads();
                if (id != k) continue;
#pragma unroll
                for (int j = 0; j < kOwn; ++j) {
                    float &to = joined[col[j]];
                    to = k == 0 ? v[j] : to + v[j];
                }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.d; c += kThreads) part[(int64_t)a * p.d + c] = joined[c];
        } else if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < C::kParts; ++i) {
                float w[C::kEach];
#pragma unroll
                for (int j = 0; j < C::kEach; ++j) w[j] = v[i * C::kEach + j];
                if (i * C::kEach < count) store_w<float, C::kEach>(part + (int64_t)a * p.d + col[i * C::kEach], w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
                if (j < count) part[(int64_t)a * p.d + col[j]] = v[j];
        }
    }
}

// The blocks' sums, added in their order, and the gradients they give: a block takes
// 32 columns, kPartWarps warps each of the sums, warp w of these every kPartWarps-th part
// from w on, kPartFlight in flight.
struct PartsParams {
    const float *parts;
    float *dpre_gain, *dpre_bias, *dpost_gain, *dpost_bias, *dgate;
    const void *post_gain, *post_bias, *gate;
    int64_t count, d;  // parts
    int sums, accumulate;
    bool post_f32, gate_f32;
    float beta;
};
constexpr int kPartWarps = 8, kPartFlight = 16;
__global__ void __launch_bounds__(kSumsMost *kPartWarps * 32) parts_kernel(const PartsParams p) {
    __shared__ float sum[kSumsMost][kPartWarps][32];
    pdl_enter();
    const int lane = threadIdx.x & 31, a = threadIdx.x / (32 * kPartWarps), w = threadIdx.x / 32 % kPartWarps;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < p.d && a < p.sums) {
        const float *at = p.parts + a * p.d + c;
        const int64_t pitch = p.sums * p.d;
        for (int64_t b = w; b < p.count; b += kPartFlight * kPartWarps) {
            float v[kPartFlight];
#pragma unroll
            for (int k = 0; k < kPartFlight; ++k) v[k] = b + k * kPartWarps < p.count ? at[(b + k * kPartWarps) * pitch] : 0.0f;
#pragma unroll
            for (int k = 0; k < kPartFlight; ++k) s += v[k];
        }
    }
    sum[a][w][lane] = s;
    __syncthreads();
    if (threadIdx.x >= 32 || c >= p.d) return;
    float t[kSumsMost];
#pragma unroll
    for (int k = 0; k < kSumsMost; ++k) {
        t[k] = sum[k][0][lane];
#pragma unroll
        for (int i = 1; i < kPartWarps; ++i) t[k] += sum[k][i][lane];
    }
    auto value = [&](const void *v, bool f32, float none) {
        return v == nullptr ? none : f32 ? static_cast<const float *>(v)[c] : to_f32<uint16_t>(static_cast<const uint16_t *>(v)[c]);
    };
    auto put = [&](float *to, float v) {
        if (p.count == 0) v = 0.0f;  // no rows: 0, whatever it was multiplied with
        if (to != nullptr) to[c] = p.accumulate ? to[c] + v : v;
    };
    const float by = p.beta * value(p.gate, p.gate_f32, 1.0f);
    put(p.dpre_gain, t[kDhUnit]);
    put(p.dpre_bias, t[kDh]);
    put(p.dpost_gain, by * t[kDUnit]);
    put(p.dpost_bias, by * t[kD]);
    if (p.dgate != nullptr) put(p.dgate, p.beta * fmaf(value(p.post_gain, p.post_f32, 1.0f), t[kDUnit], value(p.post_bias, p.post_f32, 0.0f) * t[kD]));
}

// ---------------------------------------------------------------------------
// host

// blocks (or clusters) that share the rows, each with a part of the sums
int64_t grad_parts(int64_t rows, int64_t d) { return Shape(d, kOwn).shares(rows); }

template <class TX, class TF, bool JOIN>
cudaError_t launch_grad(const NormGradParams &p, bool wide, cudaStream_t s) {
    const Shape sh(p.d, kOwn);
    return with_shape(sh, [&](auto warps, auto cluster) {
        constexpr int kWarps = decltype(warps)::value;
        constexpr bool kCluster = decltype(cluster)::value != 0;
        const int64_t grid = grad_parts(p.rows, p.d) * sh.cluster;
        if (!wide) return launch_clusters(norm_grad_kernel<TX, TF, false, kWarps, JOIN, kCluster>, grid, sh.cluster, sh.threads(), 0, s, p);
        const int rows = kCluster ? 0 : grad_stages<TX, TF>() * sh.threads();
        const cudaError_t e = opt_in_smem<norm_grad_kernel<TX, TF, true, kWarps, JOIN, kCluster>>(rows * grad_bytes<TX, TF, JOIN>(JOIN));
        if (e != cudaSuccess) return e;
        return launch_clusters(norm_grad_kernel<TX, TF, true, kWarps, JOIN, kCluster>, grid, sh.cluster, sh.threads(),
                               rows * grad_bytes<TX, TF, JOIN>(p.gate_kind == RA_GATE_MATRIX), s, p);
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
    return (size_t)(grad_parts(rows, d) * kSumsMost * d * 4);
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
    const Mat all[] = {dh, dx_new, x, f, gm, kept, dx, df, dgate, vector_of(a.dpre_gain, a.d, 4), vector_of(a.dpre_bias, a.d, 4), vector_of(a.dpost_gain, a.d, 4),
                       vector_of(a.dpost_bias, a.d, 4)};
    for (const Mat &m : all)
        if (!mat_ok(m)) return RA_ERR_INVALID_ARG;
    if (!wide_at(a.kept)) return RA_ERR_INVALID_ARG;
    if (a.d > RA_NORM_MAX_D) return RA_ERR_UNSUPPORTED;
    const bool sums = a.dpre_gain || a.dpre_bias || a.dpost_gain || a.dpost_bias || (by_vector && a.dgate);
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
    const PartsParams q{static_cast<const float *>(a.ws), a.dpre_gain, a.dpre_bias, a.dpost_gain, a.dpost_bias, by_vector ? static_cast<float *>(a.dgate) : nullptr,
                        behind.gain, behind.bias, by_vector ? a.gate : nullptr, none ? 0 : grad_parts(a.rows, a.d), a.d, join ? kSumsMost : 2, a.accumulate, behind.f32,
                        by_vector && a.gate_dtype == RA_F32, a.beta};
    return cuda_status(launch_pdl(parts_kernel, ceil_div<int64_t>(a.d, 32), kSumsMost * kPartWarps * 32, 0, s, q));
}

}  // extern "C"
