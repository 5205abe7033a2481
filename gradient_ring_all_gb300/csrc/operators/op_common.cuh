// op_common.cuh -- what the training-step operators share: argument checks
// on the host, element types, activations and the 8-bit checkpoint format on
// the device.
#pragma once

#include <math.h>

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

inline bool mat_ok(const Mat &a) {
    if (a.rows < 0 || a.cols < 0 || a.rows >= kMaxExtent || a.cols >= kMaxExtent) return false;
    if (a.empty()) return true;
    if (a.rows > 1 && a.ld < a.cols) return false;
    if (a.data == nullptr || reinterpret_cast<uintptr_t>(a.data) % a.esz != 0) return false;
    return a.rows <= 1 || a.ld <= kMaxSpan / a.rows / a.esz;
}

// Whether two matrices share a byte.  Views with one pitch (column slices of
// one array) interleave without sharing any; every other pair is judged by
// the byte ranges that it spans.
inline bool mats_overlap(const Mat &a, const Mat &b) {
    if (a.empty() || b.empty()) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.data), pb = reinterpret_cast<uintptr_t>(b.data);
    if (pa + (uintptr_t)a.span() <= pb || pb + (uintptr_t)b.span() <= pa) return false;
    if (a.pitch() == b.pitch() && a.rows > 1 && b.rows > 1) {
        const int64_t pitch = a.pitch();
        const int64_t d = pb >= pa ? (int64_t)((pb - pa) % (uintptr_t)pitch)
                                   : (pitch - (int64_t)((pa - pb) % (uintptr_t)pitch)) % pitch;
        if (d >= a.row_bytes() && d + b.row_bytes() <= pitch) return false;
    }
    return true;
}

inline bool same_mat(const Mat &a, const Mat &b) { return a.data == b.data && a.pitch() == b.pitch() && a.esz == b.esz; }

inline ra_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return RA_OK;
    record_cuda_error(e);
    return RA_ERR_CUDA;
}

template <class I>
__host__ __device__ constexpr I ceil_div(I a, I b) {
    return (a + b - 1) / b;
}

// ---------------------------------------------------------------------------
// device: scalars of either type

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

// W consecutive elements as binary32; `W * sizeof(T)` bytes, aligned to the
// access width (at most 16 bytes an access)
template <class T, int W>
__device__ __forceinline__ void load_w(const T *p, float (&x)[W]) {
    if constexpr (W * sizeof(T) >= 16) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int g = 0; g < W / V; ++g) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + g);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (sizeof(T) == 4) {
                    x[g * 4 + k] = __uint_as_float(w[k]);
                } else {
                    x[g * 8 + 2 * k] = bf16_bits_to_f32(w[k] & 0xffffu);
                    x[g * 8 + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                }
            }
        }
    } else if constexpr (W == 4 && sizeof(T) == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        x[0] = bf16_bits_to_f32(v.x & 0xffffu);
        x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = bf16_bits_to_f32(v.y & 0xffffu);
        x[3] = __uint_as_float(v.y & 0xffff0000u);
    } else if constexpr (W == 2 && sizeof(T) == 2) {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t *>(p));
        x[0] = bf16_bits_to_f32(v & 0xffffu);
        x[1] = __uint_as_float(v & 0xffff0000u);
    } else if constexpr (W == 2 && sizeof(T) == 4) {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
        x[0] = v.x;
        x[1] = v.y;
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) x[k] = to_f32<T>(__ldg(p + k));
    }
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
                    w[k] = pack_bf16x2(x[g * 8 + 2 * k], x[g * 8 + 2 * k + 1]);
            }
            reinterpret_cast<uint4 *>(p)[g] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else if constexpr (W * sizeof(T) == 8) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    } else if constexpr (W * sizeof(T) == 4 && sizeof(T) == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(x[0], x[1]);
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) p[k] = from_f32<T>(x[k]);
    }
}

// ---------------------------------------------------------------------------
// device: activations, in binary32

__device__ __forceinline__ float gauss_cdf(float z) { return fmaf(0.5f, erff(z * 0.70710678118654752f), 0.5f); }
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == RA_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
    if constexpr (ACT == RA_ACT_GELU) return z * gauss_cdf(z);
    if constexpr (ACT == RA_ACT_SILU) return z * logistic(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == RA_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == RA_ACT_GELU) return fmaf(z, 0.3989422804014327f * __expf(-0.5f * z * z), gauss_cdf(z));
    if constexpr (ACT == RA_ACT_SILU) {
        const float p = logistic(z);
        return p * fmaf(z, 1.0f - p, 1.0f);
    }
    return 1.0f;
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
__device__ __forceinline__ float dequantise(uint32_t word, int k, float step) {
    return (float)(int)(int8_t)(word >> (8 * k)) * step;
}

}  // namespace op
}  // namespace ra
