// op_checkpoint8.cu -- activation checkpoints in 8 bits: ra_checkpoint8_pack
// and ra_checkpoint8_unpack.
#include "op_common.cuh"

namespace ra {
namespace op {
namespace {

constexpr int kThreadsCkpt = 256;

struct PackParams {
    const void *x;  // pack: the activation; unpack: unused
    void *out;      // unpack: the restored activation
    int64_t ld;     // elements between the rows of x or out
    int8_t *q;
    uint8_t *e;
    int64_t rows, cols, groups;  // groups a row
    int act;
};

// One warp a group, a lane an element: any stride and alignment.
template <class T>
__global__ void __launch_bounds__(kThreadsCkpt) pack_scalar_kernel(const PackParams p) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t total = p.rows * p.groups, step = (int64_t)gridDim.x * (kThreadsCkpt / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreadsCkpt / 32) + threadIdx.x / 32; u < total; u += step) {
        const int64_t r = u / p.groups, c = (u - r * p.groups) * kGroup + lane;
        const float x = c < p.cols ? to_f32<T>(static_cast<const T *>(p.x)[r * p.ld + c]) : 0.0f;
        const Step step8 = step_of(__reduce_max_sync(0xffffffffu, magnitude_bits(x)));
        p.q[u * kGroup + lane] = (int8_t)quantise(x, step8);
        if (lane == 0) p.e[u] = (uint8_t)step8.e;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreadsCkpt) unpack_scalar_kernel(const PackParams p) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t total = p.rows * p.groups, step = (int64_t)gridDim.x * (kThreadsCkpt / 32);
    for (int64_t u = (int64_t)blockIdx.x * (kThreadsCkpt / 32) + threadIdx.x / 32; u < total; u += step) {
        const int64_t r = u / p.groups, c = (u - r * p.groups) * kGroup + lane;
        float v = (float)p.q[u * kGroup + lane] * step_value(p.e[u]);
        with_act(p.act, [&](auto a) { v = act_value<decltype(a)::value>(v); });
        if (c < p.cols) static_cast<T *>(p.out)[r * p.ld + c] = from_f32<T>(v);
    }
}

ra_status launch_ckpt(bool pack, int dtype, const PackParams &p, cudaStream_t s) {
    const int64_t blocks = ceil_div<int64_t>(p.rows * p.groups, kThreadsCkpt / 32);
    const int64_t grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    if (dtype == RA_F32)
        return cuda_status(launch_pdl(pack ? pack_scalar_kernel<float> : unpack_scalar_kernel<float>, grid, kThreadsCkpt, 0, s, p));
    return cuda_status(launch_pdl(pack ? pack_scalar_kernel<uint16_t> : unpack_scalar_kernel<uint16_t>, grid, kThreadsCkpt, 0, s, p));
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
    return launch_ckpt(pack, dtype, p, static_cast<cudaStream_t>(stream));
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
