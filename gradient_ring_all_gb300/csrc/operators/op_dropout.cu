// op_dropout.cu -- values dropped by a counter-based generator, with the
// residual they are added to: ra_dropout.
//
// y = residual + (u >= t ? x * scale : 0), u 16 bits of Philox4x32-10 (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)
// for the counter (column / 8, site, row) under the seed.  One evaluation, ten
// rounds of two wide multiplications, makes the bits of 8 neighbouring values, so
// the mask costs no memory, and memory bounds the kernel: 8192 x 8192 bf16 takes
// 44 us (6.1 TB/s, issue slots 56 % busy), 8192 x 2048 with a residual 16.  16 bits a value keep the drop probability to a
// 65536th; the scale is that of the rounded probability, so the mean is exact.
#include "op_common.cuh"

namespace ra {
namespace op {
namespace {

constexpr int kDropThreads = 256;

// u / d for any 32-bit u by a multiplication: with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, u / d = (umulhi(u, m) + u) >> s without
// the sum's overflow (Granlund and Montgomery, "Division by invariant integers
// using multiplication", 1994).
struct Divisor {
    uint32_t d, m;
    int s1, s2;
    explicit Divisor(uint32_t by) : d(by) {
        int s = 0;
        while (((uint64_t)1 << s) < by) ++s;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - by)) / by + 1);
        s1 = s < 1 ? s : 1;
        s2 = s < 1 ? 0 : s - 1;
    }
    __device__ __forceinline__ uint32_t of(uint32_t u) const {
        const uint32_t h = __umulhi(u, m);
        return (h + ((u - h) >> s1)) >> s2;
    }
};

struct DropParams {
    const void *x, *residual;
    void *y;
    const uint64_t *seed_at;
    int64_t ldx, ldr, ldy, rows, cols, first_row;
    int64_t units, per_row;  // pieces of work, and how many a row has
    Divisor by;              // per_row
    uint64_t seed;
    uint32_t keys[20];  // each round's two, from the seed (without seed_at)
    uint32_t site, t;   // a value is kept where its 16 bits are >= t / 65536
    float scale;
    bool none, dense;  // nothing is kept; each matrix is one run of rows without gaps
};

// What a round adds to the key: the golden ratio's and sqrt(3)'s fractions.
constexpr uint32_t kWeyl0 = 0x9E3779B9u, kWeyl1 = 0xBB67AE85u;

// AT: the key is made from the seed in device memory; else it is in the constants.
template <bool AT>
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, const DropParams &p, uint64_t seed) {
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ (AT ? k0 : p.keys[2 * round]);
        c2 = (uint32_t)(a >> 32) ^ c3 ^ (AT ? k1 : p.keys[2 * round + 1]);
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        k0 += kWeyl0;
        k1 += kWeyl1;
    }
    return make_uint4(c0, c1, c2, c3);
}

// the bits of group g of row r
template <bool AT>
__device__ __forceinline__ uint4 bits_of(const DropParams &p, uint64_t seed, int64_t r, uint32_t g) {
    const uint64_t row = (uint64_t)(p.first_row + r);
    return philox<AT>(g, p.site, (uint32_t)row, (uint32_t)(row >> 32), p, seed);
}

// whether value j of a group is kept: its half of the word, in the high bits, against t
__device__ __forceinline__ bool kept_of(const uint4 &w, int j, uint32_t t) {
    const uint32_t word = j < 4 ? (j < 2 ? w.x : w.y) : (j < 6 ? w.z : w.w);
    return (j & 1 ? word : word << 16) >= t;
}

template <bool AT>
__device__ __forceinline__ uint64_t seed_of(const DropParams &p) {
    return AT ? p.seed + *p.seed_at : p.seed;
}

// A unit's row and its place in the row.
__device__ __forceinline__ void place_of(const DropParams &p, int64_t u, int64_t *r, int64_t *k) {
    if (p.units <= 0xffffffffll) {
        *r = p.by.of((uint32_t)u);
        *k = (uint32_t)u - (uint32_t)*r * p.by.d;
    } else {
        *r = u / p.per_row;
        *k = u - *r * p.per_row;
    }
}

// TR: the residual's type, void for none
template <class TR>
struct Residual {
    using T = TR;
    static constexpr bool on = true;
};
template <>
struct Residual<void> {
    using T = float;
    static constexpr bool on = false;
};

// SPAN neighbours of a row, 8 or 16, as they lie in memory; rows on 16-byte
// boundaries, or on 32-byte ones where that is the access (whole sectors).
template <class T, int SPAN>
struct Span {
    uint32_t w[SPAN * sizeof(T) / 4];
    template <bool SECTOR>
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (SECTOR) {
#pragma unroll
            for (int i = 0; i < (int)(SPAN * sizeof(T)) / 32; ++i) {
                uint32_t s[8];
                load_sector(reinterpret_cast<const char *>(p) + 32 * i, s);
#pragma unroll
                for (int k = 0; k < 8; ++k) w[8 * i + k] = s[k];
            }
        } else {
#pragma unroll
            for (int i = 0; i < (int)(SPAN * sizeof(T)) / 16; ++i) {
                const uint4 v = load_16(reinterpret_cast<const char *>(p) + 16 * i);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[j]);
        else
            return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    }
    __device__ __forceinline__ void set(int j, float a, float b) {
        if constexpr (sizeof(T) == 4) {
            w[j] = __float_as_uint(a);
            w[j + 1] = __float_as_uint(b);
        } else {
            w[j / 2] = pack2(a, b);
        }
    }
    template <bool SECTOR>
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (SECTOR) {
#pragma unroll
            for (int i = 0; i < (int)(SPAN * sizeof(T)) / 32; ++i) {
                uint32_t s[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] = w[8 * i + k];
                store_sector(reinterpret_cast<char *>(p) + 32 * i, s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < (int)(SPAN * sizeof(T)) / 16; ++i)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
};

// Whole groups of 8 (SPAN 8, rows on 16-byte boundaries) or pairs of groups (SPAN
// 16, rows on 32-byte boundaries, whole sectors an access: 8192 x 8192 bf16 50 us
// with 8, 44 with 16): a thread takes kFlight spans at a time, 64 bytes or more of
// loads under way.
template <class TX, class TR, class TY, bool AT, int SPAN>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const DropParams p) {
    pdl_enter();
    using R = Residual<TR>;
    constexpr int kFlight = SPAN == 16 ? (R::on ? 1 : 2) : (R::on ? 2 : 4);
    constexpr bool kSector = SPAN == 16;
    const uint64_t seed = seed_of<AT>(p);
    constexpr int64_t kPer = kDropThreads * kFlight;
    auto at = [&](auto *base, int64_t ld, int64_t u) {
        if (p.dense) return base + u * SPAN;
        int64_t r, k;
        place_of(p, u, &r, &k);
        return base + r * ld + k * SPAN;
    };
    for (int64_t u0 = (int64_t)blockIdx.x * kPer + threadIdx.x; u0 < p.units; u0 += (int64_t)gridDim.x * kPer) {
        Span<TX, SPAN> x[kFlight];
        Span<typename R::T, SPAN> res[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const int64_t u = u0 + j * kDropThreads;
            if (u < p.units) {
                x[j].template load<kSector>(at(static_cast<const TX *>(p.x), p.ldx, u));
                if constexpr (R::on) res[j].template load<kSector>(at(static_cast<const typename R::T *>(p.residual), p.ldr, u));
            }
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const int64_t u = u0 + j * kDropThreads;
            if (u >= p.units) break;
            int64_t r, k;
            place_of(p, u, &r, &k);
            Span<TY, SPAN> out;
#pragma unroll
            for (int g = 0; g < SPAN / 8; ++g) {
                const uint4 w = bits_of<AT>(p, seed, r, (uint32_t)k * (SPAN / 8) + g);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const int c = 8 * g + i;
                    float y0 = kept_of(w, i, p.t) && !p.none ? x[j][c] * p.scale : 0.0f, y1 = kept_of(w, i + 1, p.t) && !p.none ? x[j][c + 1] * p.scale : 0.0f;
                    if constexpr (R::on) {
                        y0 += res[j][c];
                        y1 += res[j][c + 1];
                    }
                    out.set(c, y0, y1);
                }
            }
            out.template store<kSector>(at(static_cast<TY *>(p.y), p.ldy, u));
        }
    }
}

// Any stride, width and alignment (8192 x 2047 bf16 with a residual 28 us, where rows
// of 2048 take 16): a warp takes 256 neighbouring columns of a
// row.  A lane makes the bits of one group, and the lanes read and write the
// groups' values side by side.
template <class TX, class TR, class TY, bool AT>
__global__ void __launch_bounds__(kDropThreads) dropout_scalar_kernel(const DropParams p) {
    pdl_enter();
    using R = Residual<TR>;
    const uint64_t seed = seed_of<AT>(p);
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kDropThreads / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kDropThreads / 32) + threadIdx.x / 32; u < p.units; u += step) {
        int64_t r, k;
        place_of(p, u, &r, &k);
        const int64_t c0 = k * 256 + lane;
        Raw<TX, 1> x[8];
        Raw<typename R::T, 1> res[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 32 * j;
            if (c >= p.cols) break;
            x[j].load(static_cast<const TX *>(p.x) + r * p.ldx + c);
            if constexpr (R::on) res[j].load(static_cast<const typename R::T *>(p.residual) + r * p.ldr + c);
        }
        const uint4 w = bits_of<AT>(p, seed, r, (uint32_t)(k * 32 + lane));
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) mine |= kept_of(w, j, p.t) && !p.none ? 1u << j : 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t group = __shfl_sync(0xffffffffu, mine, 4 * j + lane / 8);
            const int64_t c = c0 + 32 * j;
            if (c < p.cols) {
                float y = (group >> (lane % 8)) & 1 ? x[j][0] * p.scale : 0.0f;
                if constexpr (R::on) y += res[j][0];
                static_cast<TY *>(p.y)[r * p.ldy + c] = from_f32<TY>(y);
            }
        }
    }
}

// values a thread takes at once: 16, 8, or (any stride, width and alignment) 0
template <class TX, class TR, class TY, bool AT>
cudaError_t launch_drop(const DropParams &p, int span, cudaStream_t s) {
    const int64_t each = span == 0 ? kDropThreads / 32 : kDropThreads * (32 / span) / (p.residual ? 2 : 1);
    const int64_t blocks = ceil_div<int64_t>(p.units, each), grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    return launch_pdl(span == 16 ? dropout_kernel<TX, TR, TY, AT, 16> : span == 8 ? dropout_kernel<TX, TR, TY, AT, 8> : dropout_scalar_kernel<TX, TR, TY, AT>, grid,
                      kDropThreads, 0, s, p);
}
template <class TX, class TR, class TY>
cudaError_t launch_drop(const DropParams &p, int span, cudaStream_t s) {
    return p.seed_at != nullptr ? launch_drop<TX, TR, TY, true>(p, span, s) : launch_drop<TX, TR, TY, false>(p, span, s);
}

template <class TX, class TY>
cudaError_t launch_drop(const DropParams &p, int res_dtype, int span, cudaStream_t s) {
    if (p.residual == nullptr) return launch_drop<TX, void, TY>(p, span, s);
    return res_dtype == RA_F32 ? launch_drop<TX, float, TY>(p, span, s) : launch_drop<TX, uint16_t, TY>(p, span, s);
}

}  // namespace
}  // namespace op
}  // namespace ra

extern "C" ra_status ra_dropout(const void *x, int64_t ld_x, int x_dtype, int64_t rows, int64_t cols, double p, uint64_t seed,
                                const uint64_t *seed_at, uint32_t site, int64_t first_row, const void *residual, int64_t ld_res,
                                int res_dtype, void *y, int64_t ld_y, int y_dtype, void *stream) {
    using namespace ra;
    using namespace ra::op;
    if (esize(x_dtype) == 0 || esize(y_dtype) == 0 || (residual != nullptr && esize(res_dtype) == 0)) return RA_ERR_INVALID_ARG;
    if (!(p >= 0.0 && p <= 1.0) || first_row < 0 || reinterpret_cast<uintptr_t>(seed_at) % 8 != 0) return RA_ERR_INVALID_ARG;
    const Mat a{x, rows, cols, ld_x, esize(x_dtype)}, b{y, rows, cols, ld_y, esize(y_dtype)};
    const Mat c{residual, residual ? rows : 0, cols, ld_res, residual ? esize(res_dtype) : 4};
    if (!mat_ok(a) || !mat_ok(b) || !mat_ok(c) || first_row > INT64_MAX - rows) return RA_ERR_INVALID_ARG;
    if (a.empty()) return RA_OK;
    const Mat at{seed_at, seed_at ? 1 : 0, 1, 1, 8};
    if ((mats_overlap(a, b) && !same_mat(a, b)) || (mats_overlap(c, b) && !same_mat(c, b)) || mats_overlap(at, b)) return RA_ERR_OVERLAP;
    auto aligned = [&](int bytes) { return cols % (bytes / 2) == 0 && a.aligned(bytes) && b.aligned(bytes) && (residual == nullptr || c.aligned(bytes)); };
    const int span = aligned(32) ? 16 : aligned(16) ? 8 : 0;
    const int64_t per_row = span ? cols / span : ceil_div<int64_t>(cols, 256);
    const uint32_t t = (uint32_t)nearbyint(65536.0 * p);
    const bool dense = rows == 1 || (ld_x == cols && ld_y == cols && (residual == nullptr || ld_res == cols));
    DropParams q{x, residual, y, seed_at, ld_x, ld_res, ld_y, rows, cols, first_row, rows * per_row, per_row, Divisor((uint32_t)per_row), seed, {}, site, t << 16,
                 t < 65536 ? (float)(65536.0 / (65536 - (int)t)) : 0.0f, t == 65536, dense};
    for (uint32_t k = 0; k < 10; ++k) {
        q.keys[2 * k] = (uint32_t)seed + k * kWeyl0;
        q.keys[2 * k + 1] = (uint32_t)(seed >> 32) + k * kWeyl1;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (x_dtype == RA_F32)
        return cuda_status(y_dtype == RA_F32 ? launch_drop<float, float>(q, res_dtype, span, s) : launch_drop<float, uint16_t>(q, res_dtype, span, s));
    return cuda_status(y_dtype == RA_F32 ? launch_drop<uint16_t, float>(q, res_dtype, span, s)
                                         : launch_drop<uint16_t, uint16_t>(q, res_dtype, span, s));
}
