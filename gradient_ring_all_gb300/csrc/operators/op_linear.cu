// op_linear.cu -- the linear layer and its gradients: ra_linear,
// ra_linear_dgrad and ra_linear_wgrad.
#include "op_common.cuh"

namespace ra {
namespace op {
namespace {

enum Mode { kForward = 0, kDgrad = 1, kWgrad = 2 };

// the epilogue's operands; an output row is out[r * ldo ..]
struct Epilogue {
    void *out;
    const void *bias, *res;
    int8_t *q;   // forward: written; dgrad: read
    uint8_t *e;
    int64_t ldo, ldr, groups;
    int out_f32, bias_f32, res_f32, act;
};

__device__ __forceinline__ float load_any(const void *p, int64_t i, int f32) {
    return f32 ? static_cast<const float *>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]);
}

// 32 neighbouring columns of one output row, from column n0 (a multiple of
// 32) on; `count` of them exist.
template <int MODE>
__device__ __forceinline__ void finish32(const Epilogue &ep, int64_t row, int64_t n0, int count, float (&v)[32]) {
    if constexpr (MODE == kForward) {
        if (ep.bias)
            for (int j = 0; j < count; ++j) v[j] += load_any(ep.bias, n0 + j, ep.bias_f32);
        if (ep.q) {
            uint32_t top = 0;
            for (int j = 0; j < 32; ++j) top = max(top, j < count ? magnitude_bits(v[j]) : 0u);
            const Step step = step_of(top);
            const int64_t u = row * ep.groups + n0 / kGroup;
            for (int j = 0; j < 32; ++j) ep.q[u * kGroup + j] = j < count ? (int8_t)quantise(v[j], step) : 0;
            ep.e[u] = (uint8_t)step.e;
        }
        with_act(ep.act, [&](auto a) {
            for (int j = 0; j < 32; ++j) v[j] = act_value<decltype(a)::value>(v[j]);
        });
    }
    if constexpr (MODE == kDgrad) {
        if (ep.q) {
            const int64_t u = row * ep.groups + n0 / kGroup;
            const float step = step_value(ep.e[u]);
            with_act(ep.act, [&](auto a) {
                for (int j = 0; j < 32; ++j) v[j] *= act_slope<decltype(a)::value>((float)ep.q[u * kGroup + j] * step);
            });
        }
    }
    for (int j = 0; j < count; ++j) {
        if (ep.res) v[j] += load_any(ep.res, row * ep.ldr + n0 + j, ep.res_f32);
        if (ep.out_f32)
            static_cast<float *>(ep.out)[row * ep.ldo + n0 + j] = v[j];
        else
            static_cast<uint16_t *>(ep.out)[row * ep.ldo + n0 + j] = (uint16_t)f32_to_bf16_bits(v[j]);
    }
}

// out[rows, cols] = sum over kk of A(row, kk) * B(kk, col); A(i, j) is at
// a[i * a_row + j * a_k] and so on, and A may be an 8-bit checkpoint read
// across its rows (act(z), rounded to bf16 as the tensor cores take it)
struct Product {
    const uint16_t *a, *b;
    const int8_t *aq;
    const uint8_t *ae;
    int64_t a_row, a_k, b_k, b_col, a_groups;
    int64_t rows, cols, k;
    int a_act;
    Epilogue ep;
};

template <int MODE>
__global__ void __launch_bounds__(128) product_kernel(const Product p) {
    __shared__ float ta[32][65], tb[32][65], acc_s[64][65];
    pdl_enter();
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const int tr = threadIdx.x / 16 * 8, tc = threadIdx.x % 16 * 4;
    float acc[8][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += 32) {
        for (int u = threadIdx.x; u < 32 * 64; u += 128) {
            const int i = u % 64, kk = u / 64;
            float av = 0.0f, bv = 0.0f;
            if (k0 + kk < p.k && r0 + i < p.rows) {
                if (p.aq) {
                    const int64_t t = k0 + kk, c = r0 + i, g = t * p.a_groups + c / kGroup;
                    float z = (float)p.aq[g * kGroup + c % kGroup] * step_value(p.ae[g]);
                    with_act(p.a_act, [&](auto a) { z = act_value<decltype(a)::value>(z); });
                    av = round_bf16(z);
                } else {
                    av = bf16_bits_to_f32(p.a[(r0 + i) * p.a_row + (k0 + kk) * p.a_k]);
                }
            }
            if (k0 + kk < p.k && c0 + i < p.cols) bv = bf16_bits_to_f32(p.b[(k0 + kk) * p.b_k + (c0 + i) * p.b_col]);
            ta[kk][i] = av;
            tb[kk][i] = bv;
        }
        __syncthreads();
        for (int kk = 0; kk < 32; ++kk)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ta[kk][tr + i], tb[kk][tc + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 8; ++i)
        for (int j = 0; j < 4; ++j) acc_s[tr + i][tc + j] = acc[i][j];
    __syncthreads();
    const int64_t row = r0 + threadIdx.x % 64, n0 = c0 + threadIdx.x / 64 * 32;
    if (row >= p.rows || n0 >= p.cols) return;
    float v[32];
    for (int j = 0; j < 32; ++j) v[j] = acc_s[threadIdx.x % 64][threadIdx.x / 64 * 32 + j];
    finish32<MODE>(p.ep, row, n0, (int)(p.cols - n0 < 32 ? p.cols - n0 : 32), v);
}

__global__ void __launch_bounds__(128) column_sum_kernel(const uint16_t *dy, int64_t ld, int64_t m, int64_t n, int accumulate, float *db) {
    pdl_enter();
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (c >= n) return;
    float s = 0.0f;
    for (int64_t r = 0; r < m; ++r) s += bf16_bits_to_f32(dy[r * ld + c]);
    db[c] = accumulate ? db[c] + s : s;
}

template <int MODE>
cudaError_t launch_product(const Product &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div<int64_t>(p.cols, 64), (unsigned)ceil_div<int64_t>(p.rows, 64));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RA_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, product_kernel<MODE>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// the checkpoint's two arrays as matrices
struct Kept {
    Mat q, e;
    bool ok;
};
Kept kept_mats(const int8_t *q, const uint8_t *e, int64_t rows, int64_t cols) {
    const int64_t groups = ceil_div<int64_t>(cols, kGroup);
    Kept k{{q, rows, groups * kGroup, groups * kGroup, 1}, {e, rows, groups, groups, 1}, true};
    k.ok = q != nullptr && e != nullptr && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    return k;
}

}  // namespace
}  // namespace op
}  // namespace ra

using namespace ra;
using namespace ra::op;

extern "C" {

size_t ra_linear_workspace_bytes(int64_t m, int64_t k, int64_t n) {
    if (m < 0 || k < 0 || n < 0 || m >= kMaxExtent || k >= kMaxExtent || n >= kMaxExtent) return 0;
    return 0;
}

ra_status ra_linear(const void *x, int64_t ld_x, const void *w, int64_t ld_w, int64_t m, int64_t k, int64_t n,
                    const void *bias, int bias_dtype, int act, const void *residual, int64_t ld_res, int res_dtype,
                    int8_t *save_q, uint8_t *save_e, void *y, int64_t ld_y, int y_dtype, void *ws, size_t ws_bytes,
                    void *stream) {
    (void)ws;
    (void)ws_bytes;
    const int ysz = esize(y_dtype);
    if (ysz == 0 || !act_ok(act)) return RA_ERR_INVALID_ARG;
    if ((bias && esize(bias_dtype) == 0) || (residual && esize(res_dtype) == 0)) return RA_ERR_INVALID_ARG;
    const Mat mx{x, m, k, ld_x, 2}, mw{w, k, n, ld_w, 2}, my{y, m, n, ld_y, ysz};
    const Mat mb{bias, 1, bias ? n : 0, n, bias ? esize(bias_dtype) : 1};
    const Mat mr{residual, residual ? m : 0, n, residual ? ld_res : n, residual ? esize(res_dtype) : 1};
    if (!mat_ok(mx) || !mat_ok(mw) || !mat_ok(my) || !mat_ok(mb) || !mat_ok(mr)) return RA_ERR_INVALID_ARG;
    const Kept kept = kept_mats(save_q, save_e, m, n);
    if ((save_q || save_e) && !my.empty() && !kept.ok) return RA_ERR_INVALID_ARG;
    if (my.empty()) return RA_OK;
    if (mats_overlap(my, mx) || mats_overlap(my, mw) || mats_overlap(my, mb)) return RA_ERR_OVERLAP;
    if (mats_overlap(my, mr) && !same_mat(my, mr)) return RA_ERR_OVERLAP;
    if (save_q) {
        const Mat *all[] = {&mx, &mw, &my, &mb, &mr};
        for (const Mat *o : all)
            if (mats_overlap(kept.q, *o) || mats_overlap(kept.e, *o)) return RA_ERR_OVERLAP;
        if (mats_overlap(kept.q, kept.e)) return RA_ERR_OVERLAP;
    }
    Product p = {};
    p.a = static_cast<const uint16_t *>(x);
    p.b = static_cast<const uint16_t *>(w);
    p.a_row = ld_x;
    p.a_k = 1;
    p.b_k = ld_w;
    p.b_col = 1;
    p.rows = m;
    p.cols = n;
    p.k = k;
    p.ep = Epilogue{y, bias, residual, save_q, save_e, ld_y, ld_res, ceil_div<int64_t>(n, kGroup), y_dtype == RA_F32, bias_dtype == RA_F32, res_dtype == RA_F32, act};
    return cuda_status(launch_product<kForward>(p, static_cast<cudaStream_t>(stream)));
}

ra_status ra_linear_dgrad(const void *dy, int64_t ld_dy, const void *w, int64_t ld_w, int64_t m, int64_t k, int64_t n,
                          const int8_t *z_q, const uint8_t *z_e, int act, const void *residual, int64_t ld_res, int res_dtype,
                          void *dx, int64_t ld_dx, int dx_dtype, void *ws, size_t ws_bytes, void *stream) {
    (void)ws;
    (void)ws_bytes;
    const int xsz = esize(dx_dtype);
    if (xsz == 0 || !act_ok(act) || (residual && esize(res_dtype) == 0)) return RA_ERR_INVALID_ARG;
    const Mat md{dy, m, n, ld_dy, 2}, mw{w, k, n, ld_w, 2}, mx{dx, m, k, ld_dx, xsz};
    const Mat mr{residual, residual ? m : 0, k, residual ? ld_res : k, residual ? esize(res_dtype) : 1};
    if (!mat_ok(md) || !mat_ok(mw) || !mat_ok(mx) || !mat_ok(mr)) return RA_ERR_INVALID_ARG;
    const Kept kept = kept_mats(z_q, z_e, m, k);
    if (mx.empty()) return RA_OK;
    if (act != RA_ACT_NONE && !kept.ok) return RA_ERR_INVALID_ARG;
    if (mats_overlap(mx, md) || mats_overlap(mx, mw)) return RA_ERR_OVERLAP;
    if (mats_overlap(mx, mr) && !same_mat(mx, mr)) return RA_ERR_OVERLAP;
    if (act != RA_ACT_NONE && (mats_overlap(mx, kept.q) || mats_overlap(mx, kept.e))) return RA_ERR_OVERLAP;
    Product p = {};
    p.a = static_cast<const uint16_t *>(dy);
    p.b = static_cast<const uint16_t *>(w);
    p.a_row = ld_dy;
    p.a_k = 1;
    p.b_k = 1;
    p.b_col = ld_w;
    p.rows = m;
    p.cols = k;
    p.k = n;
    p.ep = Epilogue{dx, nullptr, residual, act ? const_cast<int8_t *>(z_q) : nullptr, const_cast<uint8_t *>(z_e), ld_dx, ld_res,
                    ceil_div<int64_t>(k, kGroup), dx_dtype == RA_F32, 0, res_dtype == RA_F32, act};
    return cuda_status(launch_product<kDgrad>(p, static_cast<cudaStream_t>(stream)));
}

ra_status ra_linear_wgrad(const void *x, int64_t ld_x, const int8_t *z_q, const uint8_t *z_e, int act, const void *dy,
                          int64_t ld_dy, int64_t m, int64_t k, int64_t n, int accumulate, void *dw, int64_t ld_dw,
                          int dw_dtype, float *db, void *ws, size_t ws_bytes, void *stream) {
    (void)ws;
    (void)ws_bytes;
    const int wsz = esize(dw_dtype);
    const bool from_kept = x == nullptr && (z_q != nullptr || z_e != nullptr);
    if (wsz == 0 || !act_ok(act) || (!from_kept && act != RA_ACT_NONE)) return RA_ERR_INVALID_ARG;
    if (x != nullptr && (z_q != nullptr || z_e != nullptr)) return RA_ERR_INVALID_ARG;
    const Mat mx{x, from_kept ? 0 : m, k, from_kept ? k : ld_x, 2}, md{dy, m, n, ld_dy, 2}, mw{dw, k, n, ld_dw, wsz};
    const Mat mb{db, 1, db ? n : 0, n, 4};
    if (!mat_ok(mx) || !mat_ok(md) || !mat_ok(mw) || !mat_ok(mb)) return RA_ERR_INVALID_ARG;
    if (m < 0 || m >= kMaxExtent) return RA_ERR_INVALID_ARG;
    const Kept kept = kept_mats(z_q, z_e, m, k);
    if (from_kept && !kept.q.empty() && !kept.ok) return RA_ERR_INVALID_ARG;
    const Mat *in[] = {&mx, &md, &kept.q, &kept.e};
    for (int i = 0; i < (from_kept ? 4 : 2); ++i)
        if (mats_overlap(mw, *in[i]) || mats_overlap(mb, *in[i])) return RA_ERR_OVERLAP;
    if (mats_overlap(mw, mb)) return RA_ERR_OVERLAP;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!mw.empty()) {
        Product p = {};
        p.a = static_cast<const uint16_t *>(x);
        p.aq = from_kept ? z_q : nullptr;
        p.ae = z_e;
        p.a_groups = ceil_div<int64_t>(k, kGroup);
        p.a_act = act;
        p.b = static_cast<const uint16_t *>(dy);
        p.a_row = 1;
        p.a_k = ld_x;
        p.b_k = ld_dy;
        p.b_col = 1;
        p.rows = k;
        p.cols = n;
        p.k = m;
        p.ep = Epilogue{dw, nullptr, accumulate ? dw : nullptr, nullptr, nullptr, ld_dw, ld_dw, 0, dw_dtype == RA_F32, 0, dw_dtype == RA_F32, 0};
        const cudaError_t e = launch_product<kWgrad>(p, s);
        if (e != cudaSuccess) return cuda_status(e);
    }
    if (!mb.empty()) {
        cudaLaunchConfig_t cfg = {};
        (void)cfg;
        return cuda_status(launch_pdl(column_sum_kernel, ceil_div<int64_t>(n, 128), 128, 0, s, static_cast<const uint16_t *>(dy), ld_dy, m, n, accumulate, db));
    }
    return RA_OK;
}

}  // extern "C"
