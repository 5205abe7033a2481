// op_norm.cuh -- what the norms' forward and backward kernels share.
#pragma once

#include "op_rows.cuh"

namespace ra {
namespace op {

constexpr int kNormThreads = 256;  // of a block, unless a row takes more

// neighbours a thread takes at a time: 16 bytes of the wider of two types
template <class TX, class TF, bool WIDE>
constexpr int each_of() {
    return !WIDE ? 1 : sizeof(TX) == 4 || sizeof(TF) == 4 ? 4 : 8;
}

// A norm as the kernels take it.
struct Side {
    const void *gain, *bias;
    int kind;
    float eps;
    bool f32;
};

// The columns of a thread, OWN of them: EACH neighbours at a time (WIDE: rows on
// 16-byte boundaries, d a multiple of 8), or single ones that are the row's threads
// apart.  EACH is 16 bytes of the wider type, so that the lanes' accesses lie side by
// side: with 8 of binary32 8192 rows of 2048 took 66 us forward and 138 backward,
// with 4 they take 48 and 97.  The blocks of a cluster have equal shares.
template <int OWN, int EACH, int WARPS, bool CLUSTER>
struct Columns {
    static constexpr int kThreads = WARPS * 32, kOwn = OWN, kEach = EACH, kParts = OWN / kEach;
    int begin, end, first;  // of the block, and the thread's first
    __device__ __forceinline__ explicit Columns(int d) : begin(0), end(d) {
        if constexpr (CLUSTER) {
            const int share = ceil_div(d, 8 * (int)cluster_blocks()) * 8;
            begin = (int)cluster_block() * share;
            end = min(d, begin + share);
        }
        first = begin + (int)threadIdx.x % kThreads * kEach;
    }
    __device__ __forceinline__ int operator[](int j) const { return first + j / kEach * (kEach * kThreads) + j % kEach; }
    // how many of them are within the block's share
    __device__ __forceinline__ int count() const { return max(0, min(kParts, ceil_div(end - first, kEach * kThreads))) * kEach; }
};

// a thread's values of a vector of parameters, `none` where there is no vector
template <class C>
__device__ __forceinline__ void load_param(const void *v, bool f32, const C &col, int count, float none, float (&out)[C::kOwn]) {
#pragma unroll
    for (int j = 0; j < C::kOwn; ++j) {
        out[j] = none;
        if (v != nullptr && j < count) out[j] = f32 ? static_cast<const float *>(v)[col[j]] : to_f32<uint16_t>(static_cast<const uint16_t *>(v)[col[j]]);
    }
}

// Row r of a matrix.  WIDE: rows and the bytes between them fit 31 bits each (the
// host sees to it), so that the place is one multiplication; else 64-bit ones.
template <bool WIDE, class T>
__device__ __forceinline__ T *row_of_matrix(T *base, int64_t ld, int64_t r) {
    if constexpr (WIDE)
        return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(base) + (uint64_t)(uint32_t)r * ((uint32_t)ld * (uint32_t)sizeof(T)));
    else
        return base + r * ld;
}

// A thread's values of one row of a matrix as they lie in memory.
template <class T, class C>
struct Own {
    Raw<T, C::kEach> v[C::kParts];
    __device__ __forceinline__ float operator[](int j) const { return v[j / C::kEach][j % C::kEach]; }
    __device__ __forceinline__ Pair two(int j) const { return pair((*this)[2 * j], (*this)[2 * j + 1]); }
    // values past the row's end are 0
    __device__ __forceinline__ void load(const T *row, const C &col, int count) {
#pragma unroll
        for (int i = 0; i < C::kParts; ++i) {
            v[i].zero();
            if (i * C::kEach < count) v[i].load(row + col[i * C::kEach]);
        }
    }
    // from the thread's own places in shared memory
    __device__ __forceinline__ void take(uint32_t shared, int threads, int count) {
        constexpr int kBytes = C::kEach * (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < C::kParts; ++i) {
            v[i].zero();
            if (i * C::kEach < count) {
                const uint32_t at = shared + i * threads * kBytes;
                if constexpr (kBytes == 16)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[i].w[0]), "=r"(v[i].w[1]), "=r"(v[i].w[2]), "=r"(v[i].w[3]) : "r"(at) : "memory");
                else
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[i].w[0]), "=r"(v[i].w[1]) : "r"(at) : "memory");
            }
        }
    }
    // the values rounded to T
    __device__ __forceinline__ void set(const Pair (&p)[C::kOwn / 2]) {
#pragma unroll
        for (int j = 0; j < C::kOwn; j += 2) {
            float a, b;
            apart(p[j / 2], a, b);
            if constexpr (sizeof(T) == 4) {
                v[j / C::kEach].w[j % C::kEach] = __float_as_uint(a);
                v[(j + 1) / C::kEach].w[(j + 1) % C::kEach] = __float_as_uint(b);
            } else if constexpr (C::kEach > 1) {
                v[j / C::kEach].w[j % C::kEach / 2] = pack2(a, b);
            } else {
                const uint32_t w = pack2(a, b);
                v[j].w[0] = w & 0xffffu;
                v[j + 1].w[0] = w >> 16;
            }
        }
    }
    __device__ __forceinline__ void store(T *row, const C &col, int count) const {
#pragma unroll
        for (int i = 0; i < C::kParts; ++i) {
            if (i * C::kEach >= count) continue;
            T *to = row + col[i * C::kEach];
            if constexpr (C::kEach * sizeof(T) == 16) {
                *reinterpret_cast<uint4 *>(to) = make_uint4(v[i].w[0], v[i].w[1], v[i].w[2], v[i].w[3]);
            } else if constexpr (C::kEach > 1) {
                *reinterpret_cast<uint2 *>(to) = make_uint2(v[i].w[0], v[i].w[1]);
            } else if constexpr (sizeof(T) == 4) {
                *to = __uint_as_float(v[i].w[0]);
            } else {
                *to = (T)v[i].w[0];
            }
        }
    }
};

// Rows read ahead (WIDE): every thread copies its own values of the next rows
// asynchronously to places of its own in shared memory, beside the other threads',
// and reads them from there: nobody waits for another's copies.
template <class T, class C>
__device__ __forceinline__ void copy_own(uint32_t to, int threads, const T *row, const C &col, int count) {
    constexpr int kBytes = C::kEach * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < C::kParts; ++i)
        if (i * C::kEach < count) {
            if constexpr (kBytes == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * threads * kBytes), "l"(row + col[i * C::kEach]) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + i * threads * kBytes), "l"(row + col[i * C::kEach]) : "memory");
        }
}
// Other rows, and a cluster's: only into the L2 cache, a line of 128 bytes a thread
// (8192 rows of 2047 bf16 backward: 136 us without, 95 with, and 84 since; rows of one
// warp, 18 and 19 at 250 columns, go without).  A cluster's blocks meet once a sum, and
// a meeting waits for the copies under way: with them 2048 rows of 8192 bf16 took 125
// us backward, and 87 without a join, with this 107 and 59.
template <class T, class C>
__device__ __forceinline__ void cache_own(const T *row, const C &col) {
    const int at = col.begin + (int)threadIdx.x % C::kThreads * (128 / (int)sizeof(T));
    if (at < col.end) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + at) : "memory");
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

// whether every matrix given can be read by vectors of 8, its rows' places by 32-bit
// numbers
template <int K>
bool all_wide(const Mat (&m)[K], int64_t d) {
    if (d % 8 != 0) return false;
    for (const Mat &a : m)
        if (!a.empty() && (!a.aligned(16) || (a.rows > 1 && a.pitch() >= kMaxExtent))) return false;
    return true;
}

// How a row of d is shared: `own` columns a thread, up to 512 threads a block (blocks
// of 256 where a row takes fewer, several rows at a time), beyond that the blocks of
// a cluster.
struct Shape {
    int warps, cluster;
    Shape(int64_t d, int own) : warps(1), cluster(1) {
        while (warps < 16 && warps * 32 * own < d) warps *= 2;
        cluster = (int)ceil_div<int64_t>(d, warps * 32 * own);
    }
    int64_t groups() const { return warps * 32 < kNormThreads ? kNormThreads / (warps * 32) : 1; }
    int threads() const { return warps * 32 < kNormThreads ? kNormThreads : warps * 32; }
    // blocks, or clusters, that share the rows: as many as run at once, with two blocks
    // of 256 an SM or one of 512 (what the occupancy query gives for clusters, which
    // stay within a GPC's SMs)
    int64_t shares(int64_t rows) const {
        constexpr int kClusters[kMostBlocks] = {152, 76, 46, 36, 28, 23, 15, 15};
        const int64_t most = warps == 16 ? kClusters[cluster - 1] : 304, blocks = ceil_div<int64_t>(rows, groups());
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
