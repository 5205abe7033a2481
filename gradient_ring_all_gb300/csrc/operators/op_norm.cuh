// op_norm.cuh -- what the norms' forward and backward kernels share.
#pragma once

#include "op_rows.cuh"

namespace ra {
namespace op {

constexpr int kNormThreads = 256;  // of a block, unless a row takes more

// A norm as the kernels take it.  *_wide: on 16-byte boundaries.
struct Side {
    const void *gain, *bias;
    int kind;
    float eps;
    bool f32, gain_wide, bias_wide;
};

// W neighbouring values of a vector of parameters, `none` without one
template <int W>
__device__ __forceinline__ void load_param(const void *v, bool f32, bool wide, int64_t c, float none, float (&out)[W]) {
    if (v == nullptr) {
#pragma unroll
        for (int j = 0; j < W; ++j) out[j] = none;
    } else if (W > 1 && wide) {
        if (f32)
            load_w<float, W>(static_cast<const float *>(v) + c, out);
        else
            load_w<uint16_t, W>(static_cast<const uint16_t *>(v) + c, out);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
            out[j] = f32 ? static_cast<const float *>(v)[c + j] : to_f32<uint16_t>(static_cast<const uint16_t *>(v)[c + j]);
    }
}

// The columns of thread t of a row's threads: vectors of W, `kStep` apart.
template <int W, int N, int WARPS, bool CLUSTER>
struct Columns {
    static constexpr int kThreads = WARPS * 32, kStep = kThreads * W, kMost = kStep * N;
    int first;
    __device__ __forceinline__ Columns() : first((CLUSTER ? (int)cluster_block() * kMost : 0) + threadIdx.x % kThreads * W) {}
    __device__ __forceinline__ int operator[](int i) const { return first + i * kStep; }
};

// ---------------------------------------------------------------------------
// host

inline bool side_ok(const ra_norm &n) {
    if (n.kind < RA_NORM_NONE || n.kind > RA_NORM_RMS) return false;
    if (n.kind == RA_NORM_NONE) return true;
    const int esz = esize(n.dtype);
    return n.reserved == 0 && n.eps >= 0.0f && esz != 0 && reinterpret_cast<uintptr_t>(n.gain) % esz == 0 && reinterpret_cast<uintptr_t>(n.bias) % esz == 0;
}
inline Mat vector_of(const void *v, int64_t d, int esz) { return Mat{v, v ? 1 : 0, d, d, esz}; }
inline bool wide_at(const void *v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; }
inline Side side_of(const ra_norm &n) {
    return Side{n.kind ? n.gain : nullptr, n.kind ? n.bias : nullptr, n.kind, n.eps, n.dtype == RA_F32, wide_at(n.gain), wide_at(n.bias)};
}

inline bool types_ok(int x_dtype, int f_dtype) { return esize(x_dtype) != 0 && esize(f_dtype) != 0 && !(x_dtype == RA_BF16 && f_dtype == RA_F32); }
inline bool sizes_ok(int64_t rows, int64_t d) { return rows >= 0 && d >= 0 && rows < kMaxExtent && d < kMaxExtent; }

// whether every matrix given can be read by vectors of 8
template <int K>
bool all_wide(const Mat (&m)[K], int64_t d) {
    if (d % 8 != 0) return false;
    for (const Mat &a : m)
        if (!a.empty() && !a.aligned(16)) return false;
    return true;
}

struct Shape {
    int warps, cluster;
    int64_t groups() const { return warps * 32 < kNormThreads ? kNormThreads / (warps * 32) : 1; }
    int threads() const { return warps * 32 < kNormThreads ? kNormThreads : warps * 32; }
};

}  // namespace op
}  // namespace ra
