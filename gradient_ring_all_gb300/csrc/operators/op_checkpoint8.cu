// op_checkpoint8.cu -- activation checkpoints in 8 bits: ra_checkpoint8_pack
// and ra_checkpoint8_unpack.
#include "op_common.cuh"

namespace ra {
namespace op {
namespace {

constexpr int kThreadsCkpt = 256;

// Rows and q on 32-byte boundaries: a thread takes a group, by whole sectors.
// Bound by memory: x once in (2 or 4 bytes a value), 33/32 byte out, and back:
// 8192 x 8192 bf16 31 and 34 us (6.5 and 6.0 TB/s; half a group a thread, with
// 16-byte stores, 36 and 39).
template <class T>
__global__ void __launch_bounds__(kThreadsCkpt) pack_kernel(const PackParams p) {
    pdl_enter();
    const int64_t total = p.rows * p.groups, stride = (int64_t)gridDim.x * kThreadsCkpt;
    for (int64_t u = (int64_t)blockIdx.x * kThreadsCkpt + threadIdx.x; u < total; u += stride) {
        int64_t r, k;
        row_of(u, p.groups, total, &r, &k);
        const T *src = static_cast<const T *>(p.x) + r * p.ld + k * kGroup;
        const int64_t left = p.cols - k * kGroup;
        float x[kGroup];
        if (left >= kGroup) {
            load_group(src, x);
        } else {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) x[j] = j < left ? to_f32<T>(src[j]) : 0.0f;
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kGroup; j += 2) top = top_of(top, x[j], x[j + 1]);
        const Step step = step_of(top);
        uint32_t w[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) w[g] = quantise4(x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3], step);
        store_sector(p.q + u * kGroup, w);
        p.e[u] = (uint8_t)step.e;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreadsCkpt) unpack_kernel(const PackParams p) {
    pdl_enter();
    unpack_groups<T>(p, (int64_t)blockIdx.x * kThreadsCkpt + threadIdx.x, (int64_t)gridDim.x * kThreadsCkpt);
}

// Byte j of the result is byte (lane mod 4) of lane j's word, of the four
// lanes that differ in their low two bits: a 4 x 4 transposition.
__device__ __forceinline__ uint32_t transpose4(uint32_t w, int lane) {
    uint32_t o = __shfl_xor_sync(0xffffffffu, w, 1);
    w = lane & 1 ? __byte_perm(o, w, 0x7351) : __byte_perm(w, o, 0x6240);
    o = __shfl_xor_sync(0xffffffffu, w, 2);
    return lane & 2 ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
}

// Any stride and alignment (333 x 1001 binary32: 2.2 us each way, a launch's
// time): a warp takes four groups, a lane one value of
// each, so the loads are coalesced whatever the row's start; the transposition
// makes words of the bytes.
template <class T>
__global__ void __launch_bounds__(kThreadsCkpt) pack_scalar_kernel(const PackParams p) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t quads = ceil_div<int64_t>(p.groups, 4), total = p.rows * quads;
    const int64_t stride = (int64_t)gridDim.x * (kThreadsCkpt / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreadsCkpt / 32) + threadIdx.x / 32; u < total; u += stride) {
        int64_t r, k;
        row_of(u, quads, total, &r, &k);
        const T *src = static_cast<const T *>(p.x) + r * p.ld;
        float x[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int64_t c = (k * 4 + g) * kGroup + lane;
            x[g] = c < p.cols ? to_f32<T>(src[c]) : 0.0f;
        }
        uint32_t w = 0, e = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const Step step = step_of(__reduce_max_sync(0xffffffffu, magnitude_bits(x[g])));
            w |= quantise(x[g], step) << (8 * g);
            if (lane == g) e = step.e;
        }
        w = transpose4(w, lane);  // four neighbouring values of group lane % 4
        const int64_t first = r * p.groups + k * 4;
        if (k * 4 + (lane & 3) < p.groups) reinterpret_cast<uint32_t *>(p.q + (first + (lane & 3)) * kGroup)[lane / 4] = w;
        if (lane < 4 && k * 4 + lane < p.groups) p.e[first + lane] = (uint8_t)e;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreadsCkpt) unpack_scalar_kernel(const PackParams p) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t quads = ceil_div<int64_t>(p.groups, 4), total = p.rows * quads;
    const int64_t stride = (int64_t)gridDim.x * (kThreadsCkpt / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreadsCkpt / 32) + threadIdx.x / 32; u < total; u += stride) {
        int64_t r, k;
        row_of(u, quads, total, &r, &k);
        const int64_t first = r * p.groups + k * 4;
        const bool in = k * 4 + (lane & 3) < p.groups;
        const uint32_t e = in ? p.e[first + (lane & 3)] : 1;
        uint32_t w = in ? reinterpret_cast<const uint32_t *>(p.q + (first + (lane & 3)) * kGroup)[lane / 4] : 0;
        w = offset_bytes(transpose4(w, lane));  // the lane's value of each of the four groups
        T *dst = static_cast<T *>(p.out) + r * p.ld;
        float v[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            v[g] = dequantise(w, g, step_value(__shfl_sync(0xffffffffu, e, g)));
        }
        with_act(p.act, [&](auto a) { act_all<decltype(a)::value>(v); });
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int64_t c = (k * 4 + g) * kGroup + lane;
            if (c < p.cols) dst[c] = from_f32<T>(v[g]);
        }
    }
}

template <class T>
ra_status launch_ckpt(bool pack, bool wide, const PackParams &p, cudaStream_t s) {
    const int64_t blocks = wide ? ceil_div<int64_t>(p.rows * p.groups, kThreadsCkpt)
                                : ceil_div<int64_t>(p.rows * ceil_div<int64_t>(p.groups, 4), kThreadsCkpt / 32);
    const int64_t grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    return cuda_status(wide ? launch_pdl(pack ? pack_kernel<T> : unpack_kernel<T>, grid, kThreadsCkpt, 0, s, p)
                            : launch_pdl(pack ? pack_scalar_kernel<T> : unpack_scalar_kernel<T>, grid, kThreadsCkpt, 0, s, p));
}

ra_status run_ckpt(bool pack, const void *x, int64_t ld, int dtype, int64_t rows, int64_t cols, int8_t *q, uint8_t *e,
                   int act, void *stream) {
    const int esz = esize(dtype);
    if (esz == 0 || !act_ok(act)) return RA_ERR_INVALID_ARG;
    const Mat a{x, rows, cols, ld, esz};
    if (!mat_ok(a)) return RA_ERR_INVALID_ARG;
    if (a.empty()) return RA_OK;
    if (q == nullptr || e == nullptr || reinterpret_cast<uintptr_t>(q) % 16 != 0) return RA_ERR_INVALID_ARG;
    const int64_t groups = ceil_div<int64_t>(cols, kGroup);
    const Mat mq{q, rows, groups * kGroup, groups * kGroup, 1}, me{e, rows, groups, groups, 1};
    if (mats_overlap(a, mq) || mats_overlap(a, me) || mats_overlap(mq, me)) return RA_ERR_OVERLAP;
    const PackParams p{x, const_cast<void *>(x), ld, q, e, rows, cols, groups, act};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool wide = a.aligned(32) && reinterpret_cast<uintptr_t>(q) % 32 == 0;
    return dtype == RA_F32 ? launch_ckpt<float>(pack, wide, p, s) : launch_ckpt<uint16_t>(pack, wide, p, s);
}

}  // namespace
}  // namespace op
}  // namespace ra

extern "C" {

ra_status ra_checkpoint8_pack(const void *x, int64_t ld, int dtype, int64_t rows, int64_t cols, int8_t *q, uint8_t *e,
                              void *stream) {
    return ra::op::run_ckpt(true, x, ld, dtype, rows, cols, q, e, RA_ACT_NONE, stream);
}

ra_status ra_checkpoint8_unpack(const int8_t *q, const uint8_t *e, int64_t rows, int64_t cols, int act, void *out,
                                int64_t ld, int dtype, void *stream) {
    return ra::op::run_ckpt(false, out, ld, dtype, rows, cols, const_cast<int8_t *>(q), const_cast<uint8_t *>(e), act, stream);
}

}  // extern "C"
