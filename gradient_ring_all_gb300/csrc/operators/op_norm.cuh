// op_norm.cuh -- what the norms' forward and backward kernels share.
#pragma once

#include "op_rows.cuh"

namespace ra {
namespace op {

constexpr int kNormThreads = 256;  // of a block, unless a row takes more

// A norm as the kernels take it.
struct Side {
    const void *gain, *bias;
    int kind;
    float eps;
    bool f32;
};

constexpr int kOwn = 8;  // columns a thread has, in every row

// The columns of a thread: 8 neighbours (WIDE: rows on 16-byte boundaries, d a
// multiple of 8), or 8 that are the row's threads apart.
template <bool WIDE, int WARPS, bool CLUSTER>
struct Columns {
    static constexpr int kThreads = WARPS * 32;
    int first;
    __device__ __forceinline__ Columns()
        : first((CLUSTER ? (int)cluster_block() * kThreads * kOwn : 0) + (int)threadIdx.x % kThreads * (WIDE ? kOwn : 1)) {}
    __device__ __forceinline__ int operator[](int j) const { return first + j * (WIDE ? 1 : kThreads); }
    // how many of them are within a row of d
    __device__ __forceinline__ int count(int d) const {
        return WIDE ? (first < d ? kOwn : 0) : max(0, min(kOwn, ceil_div(d - first, kThreads)));
    }
};

// a thread's values of a vector of parameters, `none` where there is no vector
template <class C>
__device__ __forceinline__ void load_param(const void *v, bool f32, const C &col, int count, float none, float (&out)[kOwn]) {
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        out[j] = none;
        if (v != nullptr && j < count) out[j] = f32 ? static_cast<const float *>(v)[col[j]] : to_f32<uint16_t>(static_cast<const uint16_t *>(v)[col[j]]);
    }
}

// A thread's values of one row of a matrix as they lie in memory.
template <class T, bool WIDE>
struct Own {
    Raw<T, WIDE ? kOwn : 1> v[WIDE ? 1 : kOwn];
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (WIDE)
            return v[0][j];
        else
            return v[j][0];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < (WIDE ? 1 : kOwn); ++j) v[j].zero();
    }
    template <class C>
    __device__ __forceinline__ void load(const T *row, const C &col, int count) {
        zero();
        if constexpr (WIDE) {
            if (count > 0) v[0].load(row + col.first);
        } else {
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
                if (j < count) v[j].load(row + col[j]);
        }
    }
    // from the thread's own place in shared memory
    __device__ __forceinline__ void take(uint32_t shared, int pitch) {
        static_assert(WIDE, "take");
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0].w[4 * k]), "=r"(v[0].w[4 * k + 1]), "=r"(v[0].w[4 * k + 2]), "=r"(v[0].w[4 * k + 3]) : "r"(shared + k * pitch) : "memory");
    }
};
template <class T, bool WIDE, class C>
__device__ __forceinline__ void store_own(T *row, const C &col, int count, const float (&v)[kOwn]) {
    if constexpr (WIDE) {
        if (count > 0) store_w<T, kOwn>(row + col.first, v);
    } else {
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (j < count) row[col[j]] = from_f32<T>(v[j]);
    }
}

// Rows read ahead (WIDE): every thread copies its own values of the next rows
// asynchronously to places of its own in shared memory, 16 bytes each, kThreads
// places apart, and reads them from there: nobody waits for another's copies.
template <class T>
constexpr int places() {  // of 8 values
    return sizeof(T) / 2;
}
template <class T>
__device__ __forceinline__ uint32_t copy_own(uint32_t to, int pitch, const T *from) {
#pragma unroll
    for (int k = 0; k < places<T>(); ++k)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * pitch), "l"(from + k * (16 / (int)sizeof(T))) : "memory");
    return to + places<T>() * pitch;
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void await_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

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
    return Side{n.kind ? n.gain : nullptr, n.kind ? n.bias : nullptr, n.kind, n.eps, n.dtype == RA_F32};
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

// How a row of d is shared: 8 columns a thread, up to 512 threads a block (blocks of
// 256 where a row takes fewer, several rows at a time), beyond that the blocks of a
// cluster.
struct Shape {
    int warps, cluster;
    explicit Shape(int64_t d) : warps(d <= 256 ? 1 : d <= 512 ? 2 : d <= 1024 ? 4 : d <= 2048 ? 8 : 16), cluster(d <= 4096 ? 1 : d <= 8192 ? 2 : d <= 16384 ? 4 : 8) {}
    int64_t groups() const { return warps * 32 < kNormThreads ? kNormThreads / (warps * 32) : 1; }
    int threads() const { return warps * 32 < kNormThreads ? kNormThreads : warps * 32; }
    // blocks, or clusters, that share the rows; at most `each` blocks an SM
    int64_t shares(int64_t rows, int each) const {
        const int64_t most = 152 * (warps == 16 && each > 1 ? each / 2 : each) / cluster, blocks = ceil_div<int64_t>(rows, groups());
        return blocks < most ? blocks : most;
    }
};
// f(a constant for the warps, whether in clusters)
template <class F>
cudaError_t with_shape(const Shape &sh, F &&f) {
    switch (sh.warps) {
        case 1: return f(Const<1>(), Const<0>());
        case 2: return f(Const<2>(), Const<0>());
        case 4: return f(Const<4>(), Const<0>());
        case 8: return f(Const<8>(), Const<0>());
        default: return sh.cluster == 1 ? f(Const<16>(), Const<0>()) : f(Const<16>(), Const<1>());
    }
}

}  // namespace op
}  // namespace ra
