// op_logprobs.cu -- log probabilities of given tokens with their distribution's
// entropy and its most likely alternatives, and the logits' gradient:
// ra_logprobs and ra_logprobs_grad.
#include "op_rows.cuh"

namespace ra {
namespace op {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = INFINITY;

// ---------------------------------------------------------------------------
// forward

struct LogParams {
    const void *logits, *ids;
    float *logp, *lse, *entropy, *top_logp;
    int64_t *top_ids;
    int64_t ld, rows, vocab;
    float scale, scale2;  // scale2: scale / ln 2
    int top, id_bytes;
};

// A share of a row: m the largest logit, s the sum of 2^y, w that of y 2^y, with
// y = (z - m) scale2 held to at least kLeast, where 2^y is 0 (the exponential
// flushes what is below 2^-126): so a token that cannot be, or is that far off,
// adds 0 and no 0 * infinity.  A NaN stays one.
struct Share {
    float m, s, w;
};
constexpr float kLeast = -160.0f;
__device__ __forceinline__ float at_least(float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(kLeast));
    return r;
}
// what is taken out before the exponential: 0 where the largest is minus infinity
__device__ __forceinline__ float base_of(float m) { return m == -kInf ? 0.0f : m; }
__device__ __forceinline__ void rebase(Share &a, float m, float scale2) {
    const float y = at_least((a.m - base_of(m)) * scale2), f = fast_exp2(y);
    a.w = f * fmaf(y, a.s, a.w);
    a.s = f * a.s;
    a.m = m;
}
__device__ __forceinline__ Share join(Share a, Share b, float scale2) {
    const float m = fmaxf(a.m, b.m);
    rebase(a, m, scale2);
    rebase(b, m, scale2);
    return Share{m, a.s + b.s, a.w + b.w};
}
__device__ __forceinline__ void add(Share &a, float z, float scale2) {
    if (z > a.m) rebase(a, z, scale2);
    const float y = at_least((z - base_of(a.m)) * scale2), e = fast_exp2(y);
    a.s += e;
    a.w = fmaf(e, y, a.w);
}

// A logit and its index as a number that orders as the alternatives do: by
// value (a NaN first), among equals by falling index.  0 comes after every
// token that can be.
__device__ __forceinline__ uint64_t rank_of(float z, uint32_t i) {
    if (z == -kInf) return 0;
    const uint32_t b = __float_as_uint(z + 0.0f);  // one zero
    const uint32_t key = z != z ? 0xff800001u : (b & 0x80000000u ? ~b : b | 0x80000000u);
    return (uint64_t)key << 32 | (uint32_t)~i;
}

template <class T, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 256 : WARPS * 32) logprobs_kernel(const LogParams p) {
    constexpr int kThreads = WARPS * 32, kGroups = WARPS == 1 ? 8 : 1;
    __shared__ Share shares[WARPS];
    __shared__ uint64_t best[WARPS];
    pdl_enter();
    const int t = threadIdx.x % kThreads, id = threadIdx.x / kThreads;
    for (int64_t r = (int64_t)blockIdx.x * kGroups + id; r < p.rows; r += (int64_t)gridDim.x * kGroups) {
        const T *row = static_cast<const T *>(p.logits) + r * p.ld;
        Share a{-kInf, 0.0f, 0.0f};
        for (int64_t c = t; c < p.vocab; c += kThreads) add(a, to_f32<T>(row[c]), p.scale2);
#pragma unroll
        for (int o = 16; o > 0; o /= 2)
            a = join(a, Share{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.w, o)}, p.scale2);
        if constexpr (WARPS > 1) {
            __syncthreads();
            if (t % 32 == 0) shares[t / 32] = a;
            __syncthreads();
            a = shares[0];
            for (int w = 1; w < WARPS; ++w) a = join(a, shares[w], p.scale2);
        }
        const bool none = a.m == -kInf && a.s == 0.0f;
        const float base = base_of(a.m), log_s = logf(a.s);
        if (t == 0) {
            const float lse = none ? -kInf : fmaf(base, p.scale, log_s);
            p.lse[r] = lse;
            if (p.entropy != nullptr) {
                const float h = none ? 0.0f : log_s - a.w / a.s * kLn2;
                p.entropy[r] = h < 0.0f ? 0.0f : h;  // by the roundings of a certain token's row
            }
            if (p.logp != nullptr) {
                const int64_t id = p.id_bytes == 8 ? static_cast<const int64_t *>(p.ids)[r] : static_cast<const int32_t *>(p.ids)[r];
                float y = 0.0f;
                if (id >= 0 && id < p.vocab) y = none ? -kInf : (to_f32<T>(row[id]) - base) * p.scale - log_s;
                p.logp[r] = y;
            }
        }
        uint64_t last = ~0ull;
        for (int k = 0; k < p.top; ++k) {
            uint64_t mine = 0;
            for (int64_t c = t; c < p.vocab; c += kThreads) {
                const uint64_t rank = rank_of(to_f32<T>(row[c]), (uint32_t)c);
                if (rank < last && rank > mine) mine = rank;
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2) {
                const uint64_t other = __shfl_xor_sync(0xffffffffu, mine, o);
                mine = other > mine ? other : mine;
            }
            if constexpr (WARPS > 1) {
                __syncthreads();
                if (t % 32 == 0) best[t / 32] = mine;
                __syncthreads();
                for (int w = 0; w < WARPS; ++w) mine = best[w] > mine ? best[w] : mine;
            }
            if (t == 0) {
                const uint32_t i = ~(uint32_t)mine;
                p.top_ids[r * p.top + k] = mine ? (int64_t)i : -1;
                p.top_logp[r * p.top + k] = mine ? (to_f32<T>(row[i]) - base) * p.scale - log_s : -kInf;
            }
            last = mine;
        }
    }
}

// ---------------------------------------------------------------------------
// backward

struct LogGradParams {
    const void *logits, *ids;
    const float *lse, *entropy, *g, *ge;
    void *out;
    int64_t ld, ld_out, rows, vocab;
    float scale;
    int id_bytes;
};

template <class T, class TO>
__global__ void __launch_bounds__(256) logprobs_grad_kernel(const LogGradParams p) {
    pdl_enter();
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T *row = static_cast<const T *>(p.logits) + r * p.ld;
        TO *out = static_cast<TO *>(p.out) + r * p.ld_out;
        const int64_t id = p.g == nullptr ? -1 : p.id_bytes == 8 ? static_cast<const int64_t *>(p.ids)[r] : static_cast<const int32_t *>(p.ids)[r];
        const bool given = id >= 0 && id < p.vocab;
        const float lse = p.lse[r], g = given ? p.g[r] : 0.0f, ge = p.ge != nullptr ? p.ge[r] : 0.0f, h = p.ge != nullptr ? p.entropy[r] : 0.0f;
        for (int64_t c = threadIdx.x; c < p.vocab; c += 256) {
            const float z = to_f32<T>(row[c]);
            const float logp = fmaf(z, p.scale, -lse);
            const float q = fast_exp2(logp * kLog2e);
            float d = given ? -g * q : 0.0f;
            if (given && c == id) d += g;
            if (p.ge != nullptr && z != -kInf) d = fmaf(-ge * q, logp + h, d);
            out[c] = from_f32<TO>(lse == -kInf ? 0.0f : d * p.scale);
        }
    }
}

bool ids_ok(const void *ids, int id_bytes, int64_t rows) {
    return (id_bytes == 4 || id_bytes == 8) && (rows == 0 || (ids != nullptr && reinterpret_cast<uintptr_t>(ids) % id_bytes == 0));
}
bool scale_ok(float scale) { return scale > 0.0f && scale * kLog2e < kInf; }
bool floats_ok(const void *v) { return reinterpret_cast<uintptr_t>(v) % 4 == 0; }
Mat line(const void *v, int64_t n, int esz) { return Mat{v, v ? 1 : 0, n, n, esz}; }

}  // namespace
}  // namespace op
}  // namespace ra

extern "C" {

ra_status ra_logprobs(const void *logits, int64_t ld, int dtype, int64_t rows, int64_t vocab, const void *ids, int id_bytes,
                      float scale, float *logp, float *lse, float *entropy, int top, int64_t *top_ids, float *top_logp,
                      void *stream) {
    using namespace ra;
    using namespace ra::op;
    const int esz = esize(dtype);
    if (esz == 0 || !scale_ok(scale) || top < 0 || top > RA_LOGPROBS_MAX_TOP) return RA_ERR_INVALID_ARG;
    const Mat a{logits, rows, vocab, ld, esz};
    if (!mat_ok(a)) return RA_ERR_INVALID_ARG;
    if (rows == 0) return RA_OK;
    if (lse == nullptr || !floats_ok(lse) || !floats_ok(logp) || !floats_ok(entropy) || (logp != nullptr && !ids_ok(ids, id_bytes, rows))) return RA_ERR_INVALID_ARG;
    if (top > 0 && (top_ids == nullptr || top_logp == nullptr || !floats_ok(top_logp) || reinterpret_cast<uintptr_t>(top_ids) % 8 != 0)) return RA_ERR_INVALID_ARG;
    const Mat i = line(logp ? ids : nullptr, rows, id_bytes);
    const Mat out[] = {line(logp, rows, 4), line(lse, rows, 4), line(entropy, rows, 4), line(top ? top_ids : nullptr, rows * top, 8),
                       line(top ? top_logp : nullptr, rows * top, 4)};
    for (int o = 0; o < 5; ++o) {
        if (mats_overlap(out[o], a) || mats_overlap(out[o], i)) return RA_ERR_OVERLAP;
        for (int q = 0; q < o; ++q)
            if (mats_overlap(out[o], out[q])) return RA_ERR_OVERLAP;
    }
    const LogParams p{logits, ids, logp, lse, entropy, top_logp, top_ids, ld, rows, vocab, scale, scale * kLog2e, top, id_bytes};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool narrow = vocab <= 1024;
    const int64_t blocks = narrow ? ceil_div<int64_t>(rows, 8) : rows, grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    if (dtype == RA_F32)
        return cuda_status(narrow ? launch_pdl(logprobs_kernel<float, 1>, grid, 256, 0, s, p) : launch_pdl(logprobs_kernel<float, 16>, grid, 512, 0, s, p));
    return cuda_status(narrow ? launch_pdl(logprobs_kernel<uint16_t, 1>, grid, 256, 0, s, p) : launch_pdl(logprobs_kernel<uint16_t, 16>, grid, 512, 0, s, p));
}

ra_status ra_logprobs_grad(const void *logits, int64_t ld, int dtype, int64_t rows, int64_t vocab, const void *ids,
                           int id_bytes, float scale, const float *lse, const float *entropy, const float *grad_logp,
                           const float *grad_entropy, void *out, int64_t ld_out, int out_dtype, void *stream) {
    using namespace ra;
    using namespace ra::op;
    const int esz = esize(dtype), eso = esize(out_dtype);
    if (esz == 0 || eso == 0 || !scale_ok(scale)) return RA_ERR_INVALID_ARG;
    const Mat a{logits, rows, vocab, ld, esz}, b{out, rows, vocab, ld_out, eso};
    if (!mat_ok(a) || !mat_ok(b)) return RA_ERR_INVALID_ARG;
    if (a.empty()) return RA_OK;
    if (lse == nullptr || !floats_ok(lse) || !floats_ok(entropy) || !floats_ok(grad_logp) || !floats_ok(grad_entropy) ||
        (grad_logp != nullptr && !ids_ok(ids, id_bytes, rows)))
        return RA_ERR_INVALID_ARG;
    if (grad_entropy != nullptr && entropy == nullptr) return RA_ERR_INVALID_ARG;
    const Mat in[] = {line(grad_logp ? ids : nullptr, rows, id_bytes), line(lse, rows, 4), line(grad_entropy ? entropy : nullptr, rows, 4), line(grad_logp, rows, 4),
                      line(grad_entropy, rows, 4)};
    for (const Mat &m : in)
        if (mats_overlap(b, m)) return RA_ERR_OVERLAP;
    if (mats_overlap(a, b) && !same_mat(a, b)) return RA_ERR_OVERLAP;
    const LogGradParams p{logits, ids, lse, entropy, grad_logp, grad_entropy, out, ld, ld_out, rows, vocab, scale, id_bytes};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == RA_F32)
        return cuda_status(out_dtype == RA_F32 ? launch_pdl(logprobs_grad_kernel<float, float>, rows, 256, 0, s, p)
                                               : launch_pdl(logprobs_grad_kernel<float, uint16_t>, rows, 256, 0, s, p));
    return cuda_status(out_dtype == RA_F32 ? launch_pdl(logprobs_grad_kernel<uint16_t, float>, rows, 256, 0, s, p)
                                           : launch_pdl(logprobs_grad_kernel<uint16_t, uint16_t>, rows, 256, 0, s, p));
}

}  // extern "C"
