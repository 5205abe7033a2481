// op_common.cuh -- what the training-step operators share: argument checks
// on the host, element types, activations and the 8-bit checkpoint format on
// the device.
#pragma once

#include <math.h>

#include <atomic>

#include "../../../include/ra_operators.h"
#include "../ra_internal.h"
#include "../ra_kernels.cuh"

namespace ra {
namespace op {

// ---------------------------------------------------------------------------
// host: argument checks

inline int esize(int dtype) { return dtype == RA_F32 ? 4 : (dtype == RA_BF16 ? 2 : 0); }

// a row-major matrix in device memory: element (r, c) at data[r * ld + c]
struct Mat {
    const void *data;
    int64_t rows, cols, ld;
    int esz;
    bool empty() const { return rows == 0 || cols == 0; }
    int64_t pitch() const { return ld * esz; }
    int64_t row_bytes() const { return cols * esz; }
    // bytes from the first element to the end of the last
    int64_t span() const { return empty() ? 0 : (rows - 1) * pitch() + row_bytes(); }
    bool aligned(int bytes) const {
        return reinterpret_cast<uintptr_t>(data) % bytes == 0 && (rows <= 1 || pitch() % bytes == 0);
    }
};

constexpr int64_t kMaxExtent = (int64_t)1 << 31;  // rows and columns stay below 2^31
constexpr int64_t kMaxSpan = (int64_t)1 << 46;    // so that no byte offset can wrap

inline bool size_ok(const Mat &a) {
    if (a.rows < 0 || a.cols < 0 || a.rows >= kMaxExtent || a.cols >= kMaxExtent) return false;
    return a.rows <= 1 || a.cols == 0 || (a.ld >= a.cols && a.ld <= kMaxSpan / a.rows / a.esz);
}
inline bool mat_ok(const Mat &a) {
    return size_ok(a) && (a.empty() || (a.data != nullptr && reinterpret_cast<uintptr_t>(a.data) % a.esz == 0));
}

// Whether two matrices share a byte.  Views with one pitch (column slices of
// one array) interleave without sharing any, and a single row can lie between
// another's; every other pair is judged by the byte ranges that it spans.
inline bool mats_overlap(const Mat &a, const Mat &b) {
    if (a.empty() || b.empty()) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.data), pb = reinterpret_cast<uintptr_t>(b.data);
    if (pa + (uintptr_t)a.span() <= pb || pb + (uintptr_t)b.span() <= pa) return false;
    const int64_t pitch = a.rows > 1 ? a.pitch() : b.pitch();
    if ((a.rows > 1 || b.rows > 1) && (a.rows <= 1 || b.rows <= 1 || a.pitch() == b.pitch())) {
        const int64_t d = pb >= pa ? (int64_t)((pb - pa) % (uintptr_t)pitch)
                                   : (pitch - (int64_t)((pa - pb) % (uintptr_t)pitch)) % pitch;
        if (d >= a.row_bytes() && d + b.row_bytes() <= pitch) return false;
    }
    return true;
}

// the same matrix by address, type and stride (which a single row does not have)
inline bool same_mat(const Mat &a, const Mat &b) { return a.data == b.data && a.esz == b.esz && (a.pitch() == b.pitch() || a.rows <= 1); }

inline ra_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return RA_OK;
    record_cuda_error(e);
    return RA_ERR_CUDA;
}

// dynamic shared memory past 48 KB, asked for once per kernel and device
template <auto KERNEL>
inline cudaError_t opt_in_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_acq_rel);
    return e;
}

template <class I>
__host__ __device__ constexpr I ceil_div(I a, I b) {
    return (a + b - 1) / b;
}

// ---------------------------------------------------------------------------
// device: scalars of either type

// two values as bf16, the first in the low half: one conversion
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 32 bytes, a whole sector, in one access; p on a 32-byte boundary
__device__ __forceinline__ void load_sector(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p) : "memory");
}
__device__ __forceinline__ void store_sector(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_bits_to_f32(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return (uint16_t)f32_to_bf16_bits(v); }

// Ordinary loads of 16 to 2 bytes, here and everywhere: the read-only path is
// for memory that nobody writes while the kernel lives, and a kernel launched
// early lives while its predecessor writes.  As volatile instructions they keep
// their place behind the wait for that predecessor, and in their group (left to
// the compiler, the table gradient of 65521 tokens took 71 us instead of 67).
__device__ __forceinline__ uint4 load_16(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint2 load_8(const void *p) {
    uint2 v;
    asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_4(const void *p) {
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_2(const void *p) {
    uint16_t v;
    asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    return v;
}

// W consecutive elements as they lie in memory, so that many can be in flight
// in few registers; aligned to the access width (at most 16 bytes an access)
template <class T, int W>
struct Raw {
    static constexpr int kBytes = W * sizeof(T), kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int g = 0; g < kBytes / 16; ++g) {
                const uint4 v = load_16(reinterpret_cast<const char *>(p) + 16 * g);
                w[4 * g] = v.x;
                w[4 * g + 1] = v.y;
                w[4 * g + 2] = v.z;
                w[4 * g + 3] = v.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 v = load_8(p);
            w[0] = v.x;
            w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = load_4(p);
        } else {
            w[0] = load_2(p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) w[k] = 0;
    }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[j]);
        else
            return j & 1 ? __uint_as_float(w[j / 2] & 0xffff0000u) : __uint_as_float(w[j / 2] << 16);
    }
};

template <class T, int W>
__device__ __forceinline__ void load_w(const T *p, float (&x)[W]) {
    Raw<T, W> r;
    r.load(p);
#pragma unroll
    for (int j = 0; j < W; ++j) x[j] = r[j];
}

template <class T, int W>
__device__ __forceinline__ void store_w(T *p, const float (&x)[W]) {
    if constexpr (W * sizeof(T) >= 16) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int g = 0; g < W / V; ++g) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (sizeof(T) == 4)
                    w[k] = __float_as_uint(x[g * 4 + k]);
                else
                    w[k] = pack2(x[g * 8 + 2 * k], x[g * 8 + 2 * k + 1]);
            }
            reinterpret_cast<uint4 *>(p)[g] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else if constexpr (W * sizeof(T) == 8) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
    } else if constexpr (W * sizeof(T) == 4 && sizeof(T) == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack2(x[0], x[1]);
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) p[k] = from_f32<T>(x[k]);
    }
}

// ---------------------------------------------------------------------------
// device: activations, in binary32

// 1 / x and 2^x by the hardware's approximations (a unit or two in the last place)
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float logistic(float z) { return fast_rcp(1.0f + fast_exp2(z * -1.4426950408889634f)); }

// Two binary32 values in one register pair, and arithmetic on both at once
// (each rounded to nearest, as the scalar instructions round).
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
    __device__ __forceinline__ void get(float *a, float *b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v)); }
};
__device__ __forceinline__ Two operator+(Two a, Two b) {
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
    return a;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
    return a;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.v) : "l"(b.v), "l"(c.v));
    return a;
}

// The normal distribution function of two values, and through *bell
// exp(-z^2 / 2).  The tail 1 - cdf(|z|) is half of Abramowitz and Stegun's
// 7.1.26 for erfc(|z| / sqrt 2): a polynomial in 1 / (1 + c |z|) times the
// exponential, within 0.75e-7, without a branch.  In pairs it takes 10
// instructions a value.  (erff takes two paths that most warps both walk: 8192 x
// 8192 restored through gelu took 73 us with it.)
__device__ __forceinline__ void gauss_cdf(float z0, float z1, float *cdf0, float *cdf1, Two *bell) {
    const Two z(z0, z1), x = z * z * Two(-0.72134752044448170f);
    float e0, e1;
    x.get(&e0, &e1);
    const Two e(fast_exp2(e0), fast_exp2(e1));
    constexpr float c = 0.3275911f * 0.70710678118654752f;
    const Two t(fast_rcp(fmaf(fabsf(z0), c, 1.0f)), fast_rcp(fmaf(fabsf(z1), c, 1.0f)));
    Two s = fma2(t, Two(0.5f * 1.061405429f), Two(0.5f * -1.453152027f));
    s = fma2(t, s, Two(0.5f * 1.421413741f));
    s = fma2(t, s, Two(0.5f * -0.284496736f));
    s = fma2(t, s, Two(0.5f * 0.254829592f));
    float tail0, tail1;
    (s * t * e).get(&tail0, &tail1);
    *cdf0 = z0 > 0.0f ? 1.0f - tail0 : tail0;
    *cdf1 = z1 > 0.0f ? 1.0f - tail1 : tail1;
    *bell = e;
}

template <int ACT>
__device__ __forceinline__ void act_values(float &z0, float &z1) {
    if constexpr (ACT == RA_ACT_RELU) {  // a NaN stays one
        z0 = z0 < 0.0f ? 0.0f : z0;
        z1 = z1 < 0.0f ? 0.0f : z1;
    } else if constexpr (ACT == RA_ACT_GELU) {
        float c0, c1;
        Two bell(0.0f);
        gauss_cdf(z0, z1, &c0, &c1, &bell);
        z0 *= c0;
        z1 *= c1;
    } else if constexpr (ACT == RA_ACT_SILU) {
        z0 *= logistic(z0);
        z1 *= logistic(z1);
    }
}

// v *= act'(z)
template <int ACT>
__device__ __forceinline__ void times_slopes(float &v0, float &v1, float z0, float z1) {
    if constexpr (ACT == RA_ACT_RELU) {
        v0 *= z0 > 0.0f ? 1.0f : (z0 <= 0.0f ? 0.0f : z0);
        v1 *= z1 > 0.0f ? 1.0f : (z1 <= 0.0f ? 0.0f : z1);
    } else if constexpr (ACT == RA_ACT_GELU) {
        float c0, c1;
        Two bell(0.0f);
        gauss_cdf(z0, z1, &c0, &c1, &bell);
        (Two(v0, v1) * fma2(Two(z0, z1) * Two(0.3989422804014327f), bell, Two(c0, c1))).get(&v0, &v1);
    } else if constexpr (ACT == RA_ACT_SILU) {
        const float p0 = logistic(z0), p1 = logistic(z1);
        v0 *= p0 * fmaf(z0, 1.0f - p0, 1.0f);
        v1 *= p1 * fmaf(z1, 1.0f - p1, 1.0f);
    }
}

// every value of an array of pairs
template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += 2) act_values<ACT>(v[j], v[j + 1]);
}

// f(Const<ACT>) for a runtime activation
template <int V>
struct Const {
    static constexpr int value = V;
};
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
        case RA_ACT_RELU: f(Const<RA_ACT_RELU>()); break;
        case RA_ACT_GELU: f(Const<RA_ACT_GELU>()); break;
        case RA_ACT_SILU: f(Const<RA_ACT_SILU>()); break;
        default: f(Const<RA_ACT_NONE>()); break;
    }
}

inline bool act_ok(int act) { return act >= RA_ACT_NONE && act <= RA_ACT_SILU; }

// ---------------------------------------------------------------------------
// device: the 8-bit checkpoint.  kGroup neighbours of a row share the step
// 2^(e - 127), e the group's byte: 6 below the exponent of the group's largest
// magnitude, one more where that magnitude would round to 128 steps.  The
// largest magnitude is found on the bit patterns, whose order is the
// magnitudes' with NaN above infinity, so a group that holds either is marked
// (kStepNan) and reads back as NaN throughout.

constexpr int kGroup = RA_CHECKPOINT8_GROUP;
constexpr uint32_t kStepNan = 255;

__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// the largest magnitude of three values, as bits; a NaN counts as the largest
__device__ __forceinline__ uint32_t top_of(uint32_t top, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(__uint_as_float(top)), "f"(a), "f"(b));
    return __float_as_uint(r) & 0x7fffffffu;
}

// A group's byte and the factor that turns its values into steps: 2^(127 - e),
// with which the product is exact.  A marked group's factor is 0.  At the very
// top of binary32, where 128 steps would be infinite, the values are taken
// times 127/128.
struct Step {
    uint32_t e;
    float inverse;
};
__device__ __forceinline__ Step step_of(uint32_t top) {
    if (top >= 0x7f7f0000u) return top >= 0x7f800000u ? Step{kStepNan, 0.0f} : Step{248u, 0x1.fcp-122f};
    const int e = (int)((top + 0x10000u) >> 23) - 6;
    const uint32_t byte = e < 1 ? 1u : (uint32_t)e;
    return Step{byte, __uint_as_float((254u - byte) << 23)};
}
// 2^(e - 127), infinity for a marked group (0 * inf reads back as NaN)
__device__ __forceinline__ float step_value(uint32_t e) { return __uint_as_float(e << 23); }

// x / step rounded to nearest even: adding 1.5 * 2^23 leaves the whole number
// in the low bits of the sum, in two's complement
__device__ __forceinline__ uint32_t steps_bits(float x, float inverse) {
    return __float_as_uint(__fmaf_rn(x, inverse, 12582912.0f));
}
__device__ __forceinline__ uint32_t quantise(float x, Step s) { return s.e == kStepNan ? 0u : steps_bits(x, s.inverse) & 0xffu; }
// four values as the bytes of a word
__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d, Step s) {
    const uint32_t ab = __byte_perm(steps_bits(a, s.inverse), steps_bits(b, s.inverse), 0x0040);
    const uint32_t cd = __byte_perm(steps_bits(c, s.inverse), steps_bits(d, s.inverse), 0x0040);
    return s.e == kStepNan ? 0u : __byte_perm(ab, cd, 0x5410);
}
// A word of four: each byte, offset by 128, as the low bits of 2^23, less
// 2^23 + 128.  (An integer conversion shares the slow unit with the activations'
// exponentials and reciprocals.)
__device__ __forceinline__ uint32_t offset_bytes(uint32_t word) { return word ^ 0x80808080u; }
__device__ __forceinline__ float offset_float(uint32_t offset_word, int k) {
    return __uint_as_float(__byte_perm(offset_word, 0x4b000000u, 0x7650 + k));
}
__device__ __forceinline__ void dequantise4(uint32_t word, float step, float *v) {
    const uint32_t w = offset_bytes(word);
#pragma unroll
    for (int k = 0; k < 4; k += 2) ((Two(offset_float(w, k), offset_float(w, k + 1)) + Two(-8388736.0f)) * Two(step)).get(v + k, v + k + 1);
}
__device__ __forceinline__ float dequantise(uint32_t offset_word, int k, float step) { return (offset_float(offset_word, k) - 8388736.0f) * step; }

struct PackParams {
    const void *x;  // pack: the activation
    void *out;      // unpack: the restored activation
    int64_t ld;     // elements between the rows of x or out
    int8_t *q;
    uint8_t *e;
    int64_t rows, cols, groups;  // groups a row
    int act;
};

// Unit number -> row and unit within it.  32-bit division where the numbers
// fit (an ordinary size): a 64-bit one costs as much as the rest of a unit's
// work.
__device__ __forceinline__ void row_of(int64_t u, int64_t per_row, int64_t total, int64_t *r, int64_t *k) {
    if (total <= 0x7fffffff) {
        const uint32_t q = (uint32_t)u / (uint32_t)per_row;
        *r = q;
        *k = (uint32_t)u - q * (uint32_t)per_row;
    } else {
        *r = u / per_row;
        *k = u - *r * per_row;
    }
}

// 32 neighbouring values of either type, by whole sectors (p on a 32-byte boundary)
template <class T>
__device__ __forceinline__ void load_group(const T *p, float (&x)[kGroup]) {
    constexpr int kEach = 32 / sizeof(T);
#pragma unroll
    for (int g = 0; g < kGroup / kEach; ++g) {
        uint32_t w[8];
        load_sector(p + g * kEach, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (sizeof(T) == 4) {
                x[g * 8 + k] = __uint_as_float(w[k]);
            } else {
                x[g * 16 + 2 * k] = __uint_as_float(w[k] << 16);
                x[g * 16 + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    }
}
template <class T>
__device__ __forceinline__ void store_group(T *p, const float (&x)[kGroup]) {
    constexpr int kEach = 32 / sizeof(T);
#pragma unroll
    for (int g = 0; g < kGroup / kEach; ++g) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (sizeof(T) == 4)
                w[k] = __float_as_uint(x[g * 8 + k]);
            else
                w[k] = pack2(x[g * 16 + 2 * k], x[g * 16 + 2 * k + 1]);
        }
        store_sector(p + g * kEach, w);
    }
}

// Threads `first`, `first` + `stride`, .. restore a group each, to rows on
// 32-byte boundaries.
template <class T>
__device__ __forceinline__ void unpack_groups(const PackParams &p, int64_t first, int64_t stride) {
    const int64_t total = p.rows * p.groups;
    for (int64_t u = first; u < total; u += stride) {
        const uint4 q0 = load_16(p.q + u * kGroup), q1 = load_16(p.q + u * kGroup + 16);
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        const float step = step_value(p.e[u]);
        int64_t r, k;
        row_of(u, p.groups, total, &r, &k);
        float v[kGroup];
#pragma unroll
        for (int j = 0; j < 8; ++j) dequantise4(w[j], step, v + 4 * j);
        with_act(p.act, [&](auto a) { act_all<decltype(a)::value>(v); });
        T *dst = static_cast<T *>(p.out) + r * p.ld + k * kGroup;
        const int64_t left = p.cols - k * kGroup;
        if (left >= kGroup) {
            store_group(dst, v);
        } else {
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (j < left) dst[j] = from_f32<T>(v[j]);
        }
    }
}

}  // namespace op
}  // namespace ra
