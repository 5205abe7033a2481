// op_linear.cu -- the linear layer and its gradients on the tensor cores:
// ra_linear, ra_linear_dgrad and ra_linear_wgrad.
//
// All three are out = epilogue(A B) with A rows x k and B k x cols, bf16 in,
// binary32 sums:
//   forward  A = x   (a row's k values are neighbours)       "K-major"
//            B = w   (the columns of one k are neighbours)   "MN-major"
//   dgrad    A = dy, B = w^T: both K-major
//   wgrad    A = x^T, B = dy: both MN-major
// The tensor cores take either order from shared memory, so nothing is
// transposed: TMA lays 128-byte swizzled tiles of 64 k by 128 rows and by BN
// columns, one warp issues tcgen05.mma on them, the sums stay in TMEM, and
// the epilogue warps read them from there.
//
// A step of 64 k of a pair's 256 x 256 tile is 512 clocks of the tensor core and
// 64 KB of loads; 7 such steps are in flight.  Large products run into the
// power limit, the more the warmer the GPU is: on normal values, without a
// residual, 8192 x 2048 x 8192 takes 148-165 us, 8192 x 8192 x 2048 149-169 us,
// 8192^3 550-630 us; on zeros 127, 131 and 469 us (2.34 PFLOP/s at 2070 MHz).
// Small ones are bound by the rate at which an SM takes tiles in and by a
// launch's start: one 64-column step alone takes 3 us, of which the first loads
// take 0.9 and the epilogue 0.7.  A single token's forward product has a kernel
// of its own.
#include <cuda.h>

#include <cooperative_groups.h>

#include "op_common.cuh"

namespace ra {
namespace op {
namespace {

enum Mode { kForward = 0, kDgrad = 1, kWgrad = 2 };

// How blocks share tiles: one tile a block, one for a pair of blocks that work
// as one tensor core, or one for a cluster that splits k, of single blocks or of
// pairs.  kSkinny is kSplit for up to kSkinnyRows rows.
enum Kind { kSingle = 0, kPair = 1, kSplit = 2, kSkinny = 3, kPairSplit = 4 };
constexpr int kSkinnyRows = 16;

// ---------------------------------------------------------------------------
// epilogue

// what becomes of the sums; an output row is out[r * ldo ..]
struct Epilogue {
    void *out;
    const void *bias, *res;
    int8_t *q;   // forward: the checkpoint of z, written; dgrad: read
    uint8_t *e;
    int64_t ldo, ldr, groups;
    int bias_f32, res_f32, act;
    // 32: rows of out and res on 32-byte boundaries; 16: bf16 rows of out alone, on 16-byte ones; 0: others
    int rows_aligned;
    int bias_aligned, q_aligned;  // on 32-byte boundaries
};

// v += the 32 values from p on
template <bool F32>
__device__ __forceinline__ void add32(const void *p, float (&v)[32]) {
#pragma unroll
    for (int g = 0; g < (F32 ? 4 : 2); ++g) {
        uint32_t w[8];
        load_sector(static_cast<const char *>(p) + 32 * g, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (F32) {
                v[8 * g + k] += __uint_as_float(w[k]);
            } else {
                v[16 * g + 2 * k] += __uint_as_float(w[k] << 16);
                v[16 * g + 2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    }
}

// 32 values of 32 lanes, crosswise: lane l's v[k] becomes lane k's v[l]
__device__ __forceinline__ void transpose32(float (&v)[32], int lane) {
#pragma unroll
    for (int s = 16; s > 0; s /= 2) {
        const bool high = lane & s;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j & s) continue;
            const float got = __shfl_xor_sync(0xffffffffu, high ? v[j] : v[j + s], s);
            if (high)
                v[j] = got;
            else
                v[j + s] = got;
        }
    }
}

// The 32 values of a lane's row lie in N pieces of 16 bytes; N neighbouring
// lanes trade theirs: lane l's piece i becomes piece l % N of the i-th of their
// rows.  Doing it again takes it back.
template <int N>
__device__ __forceinline__ void trade(uint32_t (&w)[4 * N], int lane) {
#pragma unroll
    for (int s = 1; s < N; s *= 2) {
        const bool high = lane & s;
#pragma unroll
        for (int j = 0; j < 4 * N; ++j) {
            if (j / 4 & s) continue;
            const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[j] : w[j + 4 * s], s);
            if (high)
                w[j] = got;
            else
                w[j + 4 * s] = got;
        }
    }
}

// 32 columns of bf16 rows on 16-byte boundaries, a row a lane: `rows` rows and
// `pieces` pieces of 16 bytes of each are there.  An access takes 8 rows whole:
// a lane's sectors would be shared with its row's next columns.
__device__ __forceinline__ void store_pieces(uint16_t *p, int64_t ld, int rows, int pieces, const float (&v)[32], int lane) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack2(v[2 * j], v[2 * j + 1]);
    trade<4>(w, lane);
    const int r0 = lane / 4 * 4, c = lane % 4;
    p += r0 * ld + 8 * c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r0 + i < rows && c < pieces) *reinterpret_cast<uint4 *>(p + i * ld) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

__device__ __forceinline__ float load_any(const void *p, int64_t i, int f32) {
    return f32 ? static_cast<const float *>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]);
}

// v[i] += p[i * ld], i < rows; eight loads at a time (sixteen were no faster)
template <class T>
__device__ __forceinline__ void add_column(const T *p, int64_t ld, int rows, float (&v)[32]) {
#pragma unroll
    for (int i0 = 0; i0 < 32; i0 += 8) {
        T x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i0 + i < rows ? p[(i0 + i) * ld] : T(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i0 + i] += to_f32<T>(x[i]);
    }
}

// A warp finishes 32 neighbouring columns of 32 output rows, from column n0 (a
// multiple of 32, so one checkpoint group) and row row0 on, a row a lane;
// `count` columns and `rows` rows of them exist.  The sums of columns that do
// not exist are not looked at: they are zero, or NaN where A's row holds an
// infinity.  Each lane reads and writes its row by whole sectors.  Rows that
// start elsewhere, and the last columns, are taken crosswise, so that the lanes
// of an access are neighbours (one lane a row cost 568 x 3688 x 2440 20 of its
// 44 us); where they start on 16-byte boundaries and the result is bf16, four
// lanes trade pieces of their rows, which is less work (that product: 22.7 -> 20.9 us).
// Returns the group's step byte (forward, with a checkpoint), which the caller
// stores with its neighbours'.
template <int MODE, bool F32>
__device__ __forceinline__ uint32_t finish32(const Epilogue &ep, int64_t row0, int rows, int64_t n0, int count, float (&v)[32]) {
    const int lane = threadIdx.x & 31;
    const int64_t row = row0 + lane;
    uint32_t step_byte = 0;
    if constexpr (MODE == kForward) {
        if (ep.bias) {
            if (count == 32 && ep.bias_aligned) {
                if (ep.bias_f32)
                    add32<true>(static_cast<const float *>(ep.bias) + n0, v);
                else
                    add32<false>(static_cast<const uint16_t *>(ep.bias) + n0, v);
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j < count) v[j] += load_any(ep.bias, n0 + j, ep.bias_f32);
            }
        }
        if (ep.q) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j >= count) v[j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; j += 2) top = top_of(top, v[j], v[j + 1]);
            const Step step = step_of(top);
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = quantise4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], step);
            if (lane < rows) {
                int8_t *q = ep.q + (row * ep.groups + n0 / kGroup) * kGroup;
                if (ep.q_aligned) {
                    store_sector(q, w);
                } else {
                    reinterpret_cast<uint4 *>(q)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    reinterpret_cast<uint4 *>(q)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            step_byte = step.e;
        }
        with_act(ep.act, [&](auto a) { act_all<decltype(a)::value>(v); });
    }
    if constexpr (MODE == kDgrad) {
        if (ep.q && lane < rows) {
            const int64_t u = row * ep.groups + n0 / kGroup;
            const float step = step_value(ep.e[u]);
            uint32_t w[8];
            if (ep.q_aligned) {
                load_sector(ep.q + u * kGroup, w);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = reinterpret_cast<const uint32_t *>(ep.q + u * kGroup)[k];
            }
            with_act(ep.act, [&](auto a) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float z[4];
                    dequantise4(w[k], step, z);
                    times_slopes<decltype(a)::value>(v[4 * k], v[4 * k + 1], z[0], z[1]);
                    times_slopes<decltype(a)::value>(v[4 * k + 2], v[4 * k + 3], z[2], z[3]);
                }
            });
        }
    }
    if (count == 32 && ep.rows_aligned == 32) {
        if (lane < rows) {
            if (ep.res) {
                if (ep.res_f32)
                    add32<true>(static_cast<const float *>(ep.res) + row * ep.ldr + n0, v);
                else
                    add32<false>(static_cast<const uint16_t *>(ep.res) + row * ep.ldr + n0, v);
            }
            char *p = static_cast<char *>(ep.out) + (row * ep.ldo + n0) * (F32 ? 4 : 2);
#pragma unroll
            for (int g = 0; g < (F32 ? 4 : 2); ++g) {
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = F32 ? __float_as_uint(v[8 * g + k]) : pack2(v[16 * g + 2 * k], v[16 * g + 2 * k + 1]);
                store_sector(p + 32 * g, w);
            }
        }
        __syncwarp();
        return step_byte;
    }
    if constexpr (!F32) {
        if (count % 8 == 0 && ep.rows_aligned == 16) {
            store_pieces(static_cast<uint16_t *>(ep.out) + row0 * ep.ldo + n0, ep.ldo, rows, count / 8, v, lane);
            __syncwarp();
            return step_byte;
        }
    }
    transpose32(v, lane);  // v[i]: row row0 + i, column n0 + lane
    if (lane < count) {
        if (ep.res) {
            const int64_t at = row0 * ep.ldr + n0 + lane;
            if (ep.res_f32)
                add_column(static_cast<const float *>(ep.res) + at, ep.ldr, rows, v);
            else
                add_column(static_cast<const uint16_t *>(ep.res) + at, ep.ldr, rows, v);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (i >= rows) break;
            const int64_t at = (row0 + i) * ep.ldo + n0 + lane;
            if constexpr (F32)
                static_cast<float *>(ep.out)[at] = v[i];
            else
                static_cast<uint16_t *>(ep.out)[at] = (uint16_t)f32_to_bf16_bits(v[i]);
        }
    }
    __syncwarp();
    return step_byte;
}

// the step bytes of COLS / 32 neighbouring groups of a row, in one store where
// all are there and the place allows it
template <int COLS>
__device__ __forceinline__ void store_steps(const Epilogue &ep, int64_t row, int64_t n0, uint32_t bytes) {
    constexpr int kCount = COLS / 32;
    const int64_t g = n0 / kGroup;
    uint8_t *p = ep.e + row * ep.groups + g;
    if (kCount == 2 && g + 1 < ep.groups && reinterpret_cast<uintptr_t>(p) % 2 == 0) {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)bytes;
    } else {
#pragma unroll
        for (int k = 0; k < kCount; ++k)
            if (g + k < ep.groups) p[k] = (uint8_t)(bytes >> (8 * k));
    }
}

// ---------------------------------------------------------------------------
// tcgen05, TMA and mbarrier instructions

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Wait for a phase, for `limit` ns at most, from `t0` on where that is given; the
// clock is read only where the phase is not over yet.
__device__ __forceinline__ bool phase_over(uint32_t bar, uint32_t parity) {
    uint32_t over;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(over) : "r"(bar), "r"(parity) : "memory");
    return over;
}
__device__ __forceinline__ bool phase_seen(uint32_t bar, uint32_t parity) {
    uint32_t over;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(over) : "r"(bar), "r"(parity) : "memory");
    return over;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint64_t limit, uint64_t t0 = 0) {
    if (phase_over(bar, parity)) return true;
    if (t0 == 0) t0 = global_ns();
    while (!phase_over(bar, parity))
        if (global_ns() - t0 > limit) return false;
    return true;
}
// One lane of a converged warp.  The TMA and MMA warps stay whole and choose a
// lane for the instructions alone, so their operands stay in uniform registers:
// a loop of one lane on its own issued a 256 x 256 x 64 step in about 700
// cycles instead of the tensor core's 512.
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one;
}
// the same shared-memory place in another block of the cluster, and in the
// first of this block's pair
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) { return in_block(addr, cluster_rank() & ~1); }
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// PAIR: two blocks of a cluster on neighbouring SMs work as one tensor core
// (cta_group::2).  The loads of both count on the first one's barrier, and a
// commit reaches the same barrier in both (`blocks`: a bit for each in the cluster).
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar, [[maybe_unused]] uint16_t blocks = 0) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"(blocks)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    if constexpr (PAIR)
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
    else
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
}
template <bool PAIR, int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t slot) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "n"(COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "n"(COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <bool PAIR, int COLS>
__device__ __forceinline__ void tmem_free(uint32_t tmem) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS));
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory operand descriptor of a 128-byte swizzled tile: start
// address, the two strides between 8-row (1024-byte) swizzle atoms, in 16-byte
// units.  K-major: atoms of 8 rows x 64 k, `sbo` from one 8 rows to the next,
// lbo unused.  MN-major: atoms of 64 rows x 8 k, `lbo` from one 64 rows to the
// next, `sbo` from one 8 k to the next.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// the next of the two sums in TMEM
__device__ __forceinline__ void flip(int &acc, uint32_t &phase) {
    acc ^= 1;
    if (acc == 0) phase ^= 1;
}
// a warp has read its part of a sum (the barrier is the first block's)
template <bool PAIR>
__device__ __forceinline__ void release(uint32_t bar, int lane) {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    if (lane == 0) {
        if constexpr (PAIR)
            mbar_arrive_remote(bar);
        else
            mbar_arrive(bar);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// the product

constexpr int kBM = 128, kBK = 64;
// The tensor core adds to its binary32 sums by truncation: of a product that is
// small beside the sum, bits are lost below the sum's last place.  A sum over k
// comes out short of itself by about 1e-9 k where signs are mixed (2.3e-7 at k = 256,
// 4.4e-6 at 4096, 3.8e-5 at 32768), and by 5e-9 to 2e-8 k where all products have one
// sign (7.5e-5 at 16384, 1.6e-3 to 6e-3 at 262144).  Up to kLongSum of k that is at most a
// fifth of half a bf16 step.  A binary32 result, and a longer sum, is made in chunks: the
// tensor core sums 512 of k at a time, and the epilogue warps add the chunks in
// registers with rounding to nearest, while the next chunk is made (8192 x 16384 x
// 2048 into bf16: 301 us, 289 without; 2048 x 32000 x 2048 160 either way).
constexpr int kChunk64 = 8;
constexpr int64_t kLongSum = 16384;
enum Sums { kBf16 = 0, kF32 = 1, kBf16Long = 2 };  // the result's type, and whether bf16 ones are made in chunks
constexpr int kGroupM = 8;  // row tiles that share the columns' tiles in L2

// A tile is BN columns wide and 128 rows high per block; in a pair each block
// holds its own rows of A and half of B's columns, which the two share.
template <int BN, int KIND>
struct Shape {
    static constexpr bool kIsPair = KIND == kPair || KIND == kPairSplit, kIsSplit = KIND == kSplit || KIND == kSkinny || KIND == kPairSplit;
    // Rows of A that are loaded.  For a few rows, only those: the tensor core
    // reads 128 all the same, whatever lies there, into sums that nothing uses.
    static constexpr int kARows = KIND == kSkinny ? kSkinnyRows : kBM;
    static constexpr int kBlocks = kIsPair ? 2 : 1, kRows = kBM * kBlocks, kBCols = BN / kBlocks;
    static constexpr int kABytes = kARows * kBK * 2, kBBytes = kBCols * kBK * 2;
    // Steps of 64 k a stage holds, side by side.  A round of the loading and of the
    // issuing warp (wait, elect, instructions, commit) takes some 300 clocks
    // whatever it moves, so the smaller tiles take two steps a round.
    static constexpr int kSub = kIsPair && BN == 256 ? 1 : 2;
    static_assert(kSub <= 2, "the last stage has one step or all");
    static constexpr int kSubBytes = kABytes + kBBytes, kStageBytes = kSub * kSubBytes;
    // all of an SM's shared memory, or half of it where two blocks share an SM
    static constexpr int kStages = (KIND == kSkinny ? 9 : KIND == kSplit ? 4 : kSubBytes > 24576 ? 7 : 8) / kSub;
    static constexpr int kBlocksPerSm = kIsSplit && !kIsPair ? 2 : 1;
    // epilogue warps: four take the tile's 128 rows, and every further four share its columns
    static constexpr int kWarps = kBCols >= 128 ? 16 : 8, kCols = BN / (kWarps / 4), kThreads = (kWarps + 2) * 32;
    static constexpr int kTmemCols = 2 * BN;  // two tiles' sums: one is finished while the next is made
    static constexpr int kColumnBytes = 2 * kBCols * 4;  // column sums of the two halves of dy's rows
    // (the last stage of a skinny tile is read past its end)
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + 1024 + 256 + kColumnBytes + (kBM - kARows) * kBK * 2;
    static_assert(!kIsSplit || kStages * kStageBytes >= kBM * BN * 4, "room for a split tile's sums");
    static_assert(kSmem <= kMaxDynamicSmem && kWarps == kBCols / 16 * 2, "shared memory, warps for the column sums");
};

struct Product {
    CUtensorMap a, b;
    Epilogue ep;
    unsigned int *err;
    uint64_t wait_ns;  // the limit of each wait
    int stalled;       // self-test: the block that makes no copies (-1: none)
    int64_t rows, cols;
    int tiles_m, tiles_n;
    int k64, steps;               // 64s of k, and steps: stages along k
    int splits;                   // blocks, or pairs, that share a tile's steps
    // pairs: tiles from `whole` on, which would leave most SMs idle in a last
    // wave of their own, are made in `tail_parts` parts along k, each into its
    // own 256 x 256 of `partial` (column by column), and joined afterwards
    int whole, tail_parts;
    float *partial;
    // wgrad: the column sums of B (dy) are wanted too
    float *db;
    const uint16_t *dy;
    int64_t ld_dy, dy_rows;
    int db_add;
};

// tile number -> its row and column: bands of kGroupM row tiles, down the band first
__device__ __forceinline__ void tile_at(const Product &p, int tile, int *tm, int *tn) {
    const int band = kGroupM * p.tiles_n;
    const int first = tile / band * kGroupM;
    const int height = p.tiles_m - first < kGroupM ? p.tiles_m - first : kGroupM;
    const int in = tile - tile / band * band;
    *tm = first + in % height;
    *tn = in / height;
}

// 32 sums of a row of a split tile, column by column, over the stages (whose
// products are done by then): the lanes of a warp are neighbours
__device__ __forceinline__ void keep_sums(unsigned char *smem, int col, int row, const float (&v)[32]) {
    float *to = reinterpret_cast<float *>(smem) + col * kBM + row;
#pragma unroll
    for (int j = 0; j < 32; ++j) to[j * kBM] = v[j];
}

// The sums of a tile of a few rows lie row by row.  The rows' distance is an odd
// number of 16 bytes, so the lanes' stores meet in no bank.
template <int BN>
__device__ __forceinline__ uint32_t sums_at(int row, int col) {
    return (uint32_t)(row * (BN + 4) + col) * 4;
}
template <int BN>
__device__ __forceinline__ void keep_rows(unsigned char *smem, int col, int row, const float (&v)[32]) {
    float4 *to = reinterpret_cast<float4 *>(smem + sums_at<BN>(row, col));
#pragma unroll
    for (int j = 0; j < 8; ++j) to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// Whether a wait in one of a cluster's `blocks` blocks has run out: lane l's look
// at block l (nothing for others), after the cluster has met.  What such a block
// left is no sum, so none of them stores anything.  The look is taken beside the
// first reads of the sums, and used after them.
__device__ __forceinline__ uint32_t one_gave_up(const uint32_t *gave_up, int blocks, int lane) {
    uint32_t f = 0;
    if (lane < blocks) asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(f) : "r"(in_block(smem_addr(gave_up), lane)) : "memory");
    return f;
}

// What stands in the first of each 32 sums of a part that was not made because a
// wait ran out: a NaN that no arithmetic gives (the hardware's has all other bits set).
constexpr uint32_t kUnmade = 0x7fc0dead;

// 32 sums of a row of a tile's part, column by column
template <int ROWS>
__device__ __forceinline__ void keep_part(float *to, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) to[j * ROWS] = v[j];
}

// The bias gradient, by the epilogue warps of the blocks with the first row
// tile, while the tensor core makes its first tiles: the column sums of the block's
// kBCols columns of dy.  A warp takes 16 columns (a sector a row) and half of
// the rows, a lane every 32nd of these; then lanes and halves are added in a
// fixed order.  For up to kColumnRows rows: a warp's loads are few enough in
// flight to take longer than the tile's products past that.  Measured as what
// the sums add to a 2048 x 2048 bf16 weight gradient, here / in a launch of their
// own: 256 rows 2.6 / 3.5 us, 512 rows 3.3 / 5.0, 1024 rows 8.2 / 5.9, 4096 rows 32 / 6.8.
constexpr int64_t kColumnRows = 512;
template <class S>
__device__ __forceinline__ void column_sums(const Product &p, int64_t c0, float *half_sums, int warp, int lane) {
    const int64_t c = c0 + warp / 2 * 16;
    const int64_t r0 = warp % 2 ? p.dy_rows / 2 : 0, r1 = warp % 2 ? p.dy_rows : p.dy_rows / 2;
    float acc[16] = {};
    if (c + 16 <= p.cols) {
        constexpr int kFlight = 4;
        for (int64_t r = r0 + lane; r < r1; r += 32 * kFlight) {
            Raw<uint16_t, 16> x[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                if (r + 32 * f < r1)
                    x[f].load(p.dy + (r + 32 * f) * p.ld_dy + c);
                else
                    x[f].zero();
            }
#pragma unroll
            for (int f = 0; f < kFlight; ++f)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[j] += x[f][j];
        }
    } else if (c < p.cols) {
        for (int64_t r = r0 + lane; r < r1; r += 32)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < p.cols) acc[j] += bf16_bits_to_f32(p.dy[r * p.ld_dy + c + j]);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], d);
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) half_sums[warp % 2 * S::kBCols + warp / 2 * 16 + j] = acc[j];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(S::kWarps * 32) : "memory");  // the epilogue warps alone
    const int at = warp * 32 + lane;
    if (at < S::kBCols && c0 + at < p.cols) {
        const float sum = half_sums[at] + half_sums[S::kBCols + at];
        p.db[c0 + at] = p.db_add ? p.db[c0 + at] + sum : sum;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(S::kWarps * 32) : "memory");
}

// What a block makes in its n-th turn: a tile, and the part of it and the steps
// along k.
struct Work {
    int tile, part, k_begin, k_end;
};
template <int KIND>
__device__ __forceinline__ Work work_at(const Product &p, int unit) {
    if (KIND == kSplit || KIND == kSkinny || KIND == kPairSplit) {
        const int part = KIND == kPairSplit ? blockIdx.x / 2 % p.splits : blockIdx.x % p.splits;
        return Work{unit, part, p.steps * part / p.splits, p.steps * (part + 1) / p.splits};
    }
    if (KIND == kPair && unit >= p.whole) {
        const int u = unit - p.whole, part = u % p.tail_parts;
        return Work{p.whole + u / p.tail_parts, part, p.steps * part / p.tail_parts, p.steps * (part + 1) / p.tail_parts};
    }
    return Work{unit, 0, 0, p.steps};
}

template <int MODE, int BN, int KIND, int SUMS>
__global__ void __launch_bounds__(Shape<BN, KIND>::kThreads, Shape<BN, KIND>::kBlocksPerSm) product_kernel(const __grid_constant__ Product p) {
    using S = Shape<BN, KIND>;
    constexpr bool PAIR = S::kIsPair, CHUNKED = SUMS != kBf16, F32 = SUMS == kF32;
    constexpr bool kAmn = MODE == kWgrad, kBmn = MODE != kDgrad;
    constexpr int kChunk = kChunk64 / S::kSub, kStepK = kBK * S::kSub;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t tiles = smem_addr(smem);
    const uint32_t bars = tiles + S::kStages * S::kStageBytes;
    // full: a stage's copies have landed; empty: its products are done; done: a
    // tile's sums are; freed: they have been read; drained: all products are
    const uint32_t full = bars, empty = full + 8 * S::kStages, done = empty + 8 * S::kStages, freed = done + 16, drained = freed + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kStages * S::kStageBytes + 16 * S::kStages + 40);
    uint32_t *gave_up = tmem_slot + 1;  // whether a wait of the block did
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = PAIR ? blockIdx.x & 1 : 0;
    // the first unit of work and the distance to the next
    const int share = (S::kIsSplit ? p.splits : 1) * S::kBlocks;
    const int unit0 = blockIdx.x / share, unit_step = gridDim.x / share;

    if (warp == S::kWarps) {
        if (lane == 0) {
            for (int s = 0; s < S::kStages; ++s) {
                mbar_init(full + 8 * s, 1);
                mbar_init(empty + 8 * s, 1);
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(done + 8 * s, 1);
                mbar_init(freed + 8 * s, S::kWarps * S::kBlocks);
            }
            mbar_init(drained, 1);
            *gave_up = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
    } else if (warp == S::kWarps + 1) {
        tmem_alloc<PAIR, S::kTmemCols>(smem_addr(tmem_slot));
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    if constexpr (PAIR)
        cluster_sync();
    else
        __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    pdl_enter();

    const int tile_count = p.tiles_m * p.tiles_n, unit_count = KIND == kPair ? p.whole + (tile_count - p.whole) * p.tail_parts : tile_count;
    bool ok = true;
    if (warp == S::kWarps) {  // TMA
        int s = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        for (int unit = unit0; unit < unit_count && ok; unit += unit_step) {
            const Work work = work_at<KIND>(p, unit);
            int tm, tn;
            tile_at(p, work.tile, &tm, &tn);
            const int row = tm * S::kRows + rank * kBM, col = tn * BN + rank * S::kBCols;
            for (int k = work.k_begin; k < work.k_end; ++k) {
                ok = __all_sync(0xffffffffu, wait(empty + 8 * s, phase ^ 1, p.wait_ns));
                if (!ok) break;
                const uint32_t a = tiles + s * S::kStageBytes, b = a + S::kABytes;
                const uint32_t bar = PAIR ? in_leader(full + 8 * s) : full + 8 * s;
                if (elected()) {
                    const int subs = S::kSub == 1 || (k + 1) * S::kSub <= p.k64 ? S::kSub : 1;  // of the last stage
                    if (rank == 0) mbar_expect(full + 8 * s, subs * S::kSubBytes * S::kBlocks);
#pragma unroll
                    for (int u = 0; u < S::kSub; ++u) {
                        if (u >= subs || blockIdx.x == p.stalled) break;
                        const int at = k * kStepK + u * kBK;
                        const uint32_t au = a + u * S::kSubBytes, bu = b + u * S::kSubBytes;
                        if constexpr (kAmn) {
#pragma unroll
                            for (int j = 0; j < kBM / 64; ++j) tma_load<PAIR>(au + j * 8192, &p.a, row + j * 64, at, bar);
                        } else {
                            tma_load<PAIR>(au, &p.a, at, row, bar);
                        }
                        if constexpr (kBmn) {
#pragma unroll
                            for (int j = 0; j < S::kBCols / 64; ++j) tma_load<PAIR>(bu + j * 8192, &p.b, col + j * 64, at, bar);
                        } else {
                            tma_load<PAIR>(bu, &p.b, at, col, bar);
                        }
                    }
                }
                __syncwarp();
                ++issued;
                if (++s == S::kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // shared memory must outlive the copies and the products that read it
        for (int64_t i = issued > S::kStages ? issued - S::kStages : 0; i < issued && ok; ++i)
            ok = __all_sync(0xffffffffu, wait(empty + 8 * (uint32_t)(i % S::kStages), (uint32_t)(i / S::kStages) & 1, p.wait_ns));
        // Also where a wait gave up: then nobody may read the stages any more,
        // but copies can still be on their way.  A pair's all count on its
        // first block's barriers, which the second, waiting at the end, may have
        // asked for a round of stages more.
        if (!ok && rank == 0) {
            const uint64_t t0 = global_ns();
            for (int64_t i = issued > S::kStages ? issued - S::kStages : 0; i < issued + (PAIR ? S::kStages : 0); ++i)
                wait(full + 8 * (uint32_t)(i % S::kStages), (uint32_t)(i / S::kStages) & 1, p.wait_ns, t0);
        }
    } else if (warp == S::kWarps + 1) {  // tcgen05.mma
        if (rank == 0) {
            constexpr uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (kAmn ? 1u << 15 : 0) | (kBmn ? 1u << 16 : 0) | (BN / 8) << 17 | (S::kRows / 16) << 24;
            // 16 of k further on in a stage, a stage and a 64 of k further on, in the descriptors' 16-byte units
            constexpr uint32_t a_next = (kAmn ? 2048 : 32) >> 4, b_next = (kBmn ? 2048 : 32) >> 4, stage_next = S::kStageBytes >> 4,
                               sub_next = S::kSubBytes >> 4;
            const uint64_t a0 = operand(tiles, kAmn ? 8192 : 16, 1024), b0 = operand(tiles + S::kABytes, kBmn ? 8192 : 16, 1024);
            const bool lead = elected();
            const uint16_t both = PAIR ? 3 << cluster_rank() : 0;  // the pair's blocks (this is its first)
            int s = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool landed = false;  // whether stage s is known to have
            for (int unit = unit0; unit < unit_count && ok; unit += unit_step) {
                const Work work = work_at<KIND>(p, unit);
                const int steps = work.k_end - work.k_begin;
                for (int k = 0; k < steps || k == 0; ++k) {
                    const int in_sum = CHUNKED ? k % kChunk : k;
                    if (in_sum == 0) {  // a new sum
                        ok = __all_sync(0xffffffffu, wait(freed + 8 * acc, acc_phase ^ 1, p.wait_ns));
                        if (!ok) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    }
                    const bool last = k + 1 >= steps || (CHUNKED && in_sum == kChunk - 1);
                    if (steps > 0) {
                        if (!landed) {
                            ok = __all_sync(0xffffffffu, wait(full + 8 * s, phase, p.wait_ns));
                            if (!ok) break;
                        }
                        if (lead) {
                            const uint64_t a = a0 + s * stage_next, b = b0 + s * stage_next;
                            const uint32_t sum = tmem + acc * BN;
#pragma unroll
                            for (int j = 0; j < kBK / 16; ++j) mma_bf16<PAIR>(sum, a + j * a_next, b + j * b_next, idesc, in_sum > 0 || j > 0);
                            if (S::kSub > 1 && (work.k_begin + k + 1) * S::kSub <= p.k64) {  // not the last half of a stage
#pragma unroll
                                for (int j = 0; j < kBK / 16; ++j) mma_bf16<PAIR>(sum, a + sub_next + j * a_next, b + sub_next + j * b_next, idesc, 1);
                            }
                            mma_commit<PAIR>(empty + 8 * s, both);
                            if (last) mma_commit<PAIR>(done + 8 * acc, both);
                        }
                        if (++s == S::kStages) {
                            s = 0;
                            phase ^= 1;
                        }
                        // the next stage is looked at while these products run
                        landed = __all_sync(0xffffffffu, phase_seen(full + 8 * s, phase));
                    } else if (lead) {
                        mma_commit<PAIR>(done + 8 * acc, both);
                    }
                    if (last) flip(acc, acc_phase);
                }
            }
            __syncwarp();
            // TMEM must outlive the products, also where a wait gave up
            if (lead) {
                if constexpr (PAIR)
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drained) : "memory");
                else
                    mma_commit<false>(drained);
            }
            __syncwarp();
            ok &= wait(drained, 0, p.wait_ns);
        }
    } else {
        const uint32_t freed_bar = PAIR ? in_leader(freed) : freed;
        int acc = 0;
        uint32_t acc_phase = 0;
        const uint32_t mine = tmem + (warp / 4) * S::kCols + ((uint32_t)(warp % 4 * 32) << 16);
        // where a part's sums go, for the warp's first column and this lane's row
        [[maybe_unused]] auto part_at = [&](int unit) {
            return p.partial + ((int64_t)(unit - p.whole) * BN + warp / 4 * S::kCols) * S::kRows + rank * kBM + warp % 4 * 32 + lane;
        };
        if (MODE == kWgrad && p.db) {
            // All of the block's column sums before its first wait: they have
            // barriers for all epilogue warps, and each of these decides by
            // itself that a wait has run out.
            for (int unit = unit0; unit < unit_count; unit += unit_step) {
                const Work work = work_at<KIND>(p, unit);
                int tm, tn;
                tile_at(p, work.tile, &tm, &tn);
                if (tm == 0 && work.part == 0)
                    column_sums<S>(p, (int64_t)tn * BN + rank * S::kBCols, reinterpret_cast<float *>(smem + S::kStages * S::kStageBytes + 256), warp, lane);
            }
        }
        int unit = unit0;
        for (; unit < unit_count && ok; unit += unit_step) {
            const Work work = work_at<KIND>(p, unit);
            const int steps = work.k_end - work.k_begin;
            int tm, tn;
            tile_at(p, work.tile, &tm, &tn);
            const int64_t row0 = (int64_t)tm * S::kRows + rank * kBM + warp % 4 * 32, row = row0 + lane;
            const int rows = p.rows - row0 < 32 ? (int)(p.rows - row0) : 32;  // of the warp's 32 (none where not above 0)
            const int64_t c0 = (int64_t)tn * BN + warp / 4 * S::kCols;
            const bool tail = KIND == kPair && unit >= p.whole;
            float *to = tail ? part_at(unit) : nullptr;
            if constexpr (CHUNKED) {
                float sum[S::kCols / 32][32];
#pragma unroll
                for (int g = 0; g < S::kCols / 32; ++g)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[g][j] = 0.0f;
                for (int k = 0; k < steps || k == 0; k += kChunk) {
                    ok = __all_sync(0xffffffffu, wait(done + 8 * acc, acc_phase, p.wait_ns));
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (steps > 0) {
#pragma unroll
                        for (int g = 0; g < S::kCols / 16; ++g) {
                            float v[16];
                            tmem_load16(mine + acc * BN + g * 16, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[g / 2][g % 2 * 16 + j] += v[j];
                        }
                    }
                    release<PAIR>(freed_bar + 8 * acc, lane);
                    flip(acc, acc_phase);
                }
                if (!ok) break;
                if constexpr (S::kIsSplit) {
#pragma unroll
                    for (int g = 0; g < S::kCols / 32; ++g) {
                        if constexpr (KIND != kSkinny)
                            keep_sums(smem, warp / 4 * S::kCols + g * 32, warp % 4 * 32 + lane, sum[g]);
                        else if (warp % 4 == 0 && lane < kSkinnyRows)
                            keep_rows<BN>(smem, warp / 4 * S::kCols + g * 32, lane, sum[g]);
                    }
                    continue;
                }
                if (tail) {
#pragma unroll
                    for (int g = 0; g < S::kCols / 32; ++g) keep_part<S::kRows>(to + g * 32 * S::kRows, sum[g]);
                    continue;
                }
                uint32_t step_bytes = 0;
#pragma unroll
                for (int g = 0; g < S::kCols / 32; ++g) {
                    const int64_t n0 = c0 + g * 32;
                    if (rows > 0 && n0 < p.cols)
                        step_bytes |= finish32<MODE, F32>(p.ep, row0, rows, n0, (int)(p.cols - n0 < 32 ? p.cols - n0 : 32), sum[g]) << (8 * g);
                }
                if (MODE == kForward && !S::kIsSplit && !tail && p.ep.q && row < p.rows && c0 < p.cols) store_steps<S::kCols>(p.ep, row, c0, step_bytes);
                __syncwarp();
            } else {
                ok = __all_sync(0xffffffffu, wait(done + 8 * acc, acc_phase, p.wait_ns));
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                uint32_t step_bytes = 0;
#pragma unroll 1
                for (int g = 0; g < S::kCols / 32; ++g) {
                    const int64_t n0 = c0 + g * 32;
                    if (n0 >= p.cols) break;
                    float v[32];
                    tmem_load32(mine + acc * BN + g * 32, v);
                    if (steps == 0) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                    }
                    if constexpr (S::kIsSplit) {
                        if constexpr (KIND != kSkinny)
                            keep_sums(smem, warp / 4 * S::kCols + g * 32, warp % 4 * 32 + lane, v);
                        else if (warp % 4 == 0 && lane < kSkinnyRows)
                            keep_rows<BN>(smem, warp / 4 * S::kCols + g * 32, lane, v);
                        continue;
                    }
                    if (tail) {
                        keep_part<S::kRows>(to + g * 32 * S::kRows, v);
                        continue;
                    }
                    if (rows > 0) step_bytes |= finish32<MODE, F32>(p.ep, row0, rows, n0, (int)(p.cols - n0 < 32 ? p.cols - n0 : 32), v) << (8 * g);
                }
                if (MODE == kForward && !S::kIsSplit && !tail && p.ep.q && row < p.rows && c0 < p.cols) store_steps<S::kCols>(p.ep, row, c0, step_bytes);
                release<PAIR>(freed_bar + 8 * acc, lane);
                flip(acc, acc_phase);
            }
        }
        if constexpr (KIND == kPair)  // the parts that a wait which ran out leaves unmade
            for (; unit < unit_count; unit += unit_step)
                if (unit >= p.whole)
                    for (int g = 0; g < S::kCols / 32; ++g) part_at(unit)[g * 32 * S::kRows] = __uint_as_float(kUnmade);
    }
    if (!ok) {
        atomicOr(p.err, 1u);
        *reinterpret_cast<volatile uint32_t *>(gave_up) = 1;
    }
    __syncwarp();
    if constexpr (KIND == kSkinny) {
        // Every block's sums lie in its shared memory; the blocks share the work
        // of adding and finishing them, 32 columns of 32 / splits rows at a time.
        // Eight lanes read 128 bytes of a row of one split, and a lane's eight
        // reads are all on their way at once; then the splits are added across
        // the lanes, in a fixed order, and each lane gets its row.  With the first
        // block alone reading, a row a lane and four bytes at a time as below,
        // 16 x 2048 x 2048 took 8.2 us instead of 6.3.  (The 128 rows of a
        // whole tile are better read that way: this one's exchanges between
        // lanes then cost more than the reads, 7.3 against 6.5 us at 256 x 1024 x 1024.)
        cluster_sync();
        const uint32_t failed = one_gave_up(gave_up, p.splits, lane);
        const int part = blockIdx.x % p.splits, per_task = 32 / p.splits, tasks = BN / 32 * (S::kARows / per_task);
        int tm, tn;
        tile_at(p, unit0, &tm, &tn);
        const int sub = lane / 8, q0 = p.splits == 2 ? sub / 2 : sub, r0 = p.splits == 2 ? sub % 2 * 8 : 0;
        for (int t = part + warp * p.splits; t < tasks && warp < S::kWarps; t += S::kWarps * p.splits) {
            const int g = t % (BN / 32), in_tile = t / (BN / 32) * per_task;
            const int64_t row0 = (int64_t)tm * kBM + in_tile, n0 = (int64_t)tn * BN + g * 32;
            if (row0 >= p.rows || n0 >= p.cols) continue;
            const int rows = p.rows - row0 < per_task ? (int)(p.rows - row0) : per_task;
            const uint32_t from = tiles + sums_at<BN>(in_tile + r0, g * 32 + lane % 8 * 4);
            const uint32_t one = in_block(from, q0), two = p.splits == 8 ? in_block(from, (q0 + 4)) : one;
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // with eight splits four rows of each of two, else eight rows of one
                const uint32_t at = p.splits == 8 ? (i < 4 ? one : two) + sums_at<BN>(i % 4, 0) : one + sums_at<BN>(i, 0);
                asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3]) : "r"(at) : "memory");
            }
            if (__any_sync(0xffffffffu, failed)) break;
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]);
            if (p.splits == 8) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += v[j + 16];
            }
            if (p.splits > 2) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], 8);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j] + __shfl_xor_sync(0xffffffffu, v[j], 16));
            trade<8>(w, lane);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]);
            const uint32_t step_byte = finish32<MODE, F32>(p.ep, row0, rows, n0, (int)(p.cols - n0 < 32 ? p.cols - n0 : 32), v);
            if (MODE == kForward && p.ep.q && lane < rows) store_steps<32>(p.ep, row0 + lane, n0, step_byte);
        }
        __syncwarp();
    } else if constexpr (S::kIsSplit) {
        // every block's sums lie in its shared memory: each block adds and
        // finishes its share of the rows, the splits in their order
        cluster_sync();
        const uint32_t failed = one_gave_up(gave_up, p.splits * S::kBlocks, lane);
        const int height = kBM / p.splits, per_group = height > 32 ? height / 32 : 1;  // warps a column group
        const int g = warp / per_group, at0 = warp % per_group * 32;
        int tm, tn;
        tile_at(p, unit0, &tm, &tn);
        const int in_tile = blockIdx.x / S::kBlocks % p.splits * height + at0;
        const int64_t row0 = (int64_t)tm * S::kRows + rank * kBM + in_tile, n0 = (int64_t)tn * BN + g * 32;
        int rows = height < 32 ? height : 32;
        if (p.rows - row0 < rows) rows = (int)(p.rows - row0);
        if (g < BN / 32 && rows > 0 && n0 < p.cols) {
            float v[32];
            // (lanes past the block's rows read its neighbours' and drop them)
            for (int q = 0; q < p.splits; ++q) {
                const uint32_t from = in_block(tiles + (g * 32 * kBM + (in_tile + lane) % kBM) * 4, q * S::kBlocks + rank);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float x;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(from + j * kBM * 4) : "memory");
                    v[j] = q ? v[j] + x : x;
                }
            }
            if (!__any_sync(0xffffffffu, failed)) {
                const uint32_t step_byte = finish32<MODE, F32>(p.ep, row0, rows, n0, (int)(p.cols - n0 < 32 ? p.cols - n0 : 32), v);
                if (MODE == kForward && p.ep.q && lane < rows) store_steps<32>(p.ep, row0 + lane, n0, step_byte);
            }
        }
        __syncwarp();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    if constexpr (KIND != kSingle)
        cluster_sync();  // neither block's memory goes while the other may still reach it
    else
        __syncthreads();
    if (warp == S::kWarps + 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        tmem_free<PAIR, S::kTmemCols>(tmem);
    }
}

// The tiles made in parts: the sums of the parts in their order, then the
// epilogue; nothing where a part was not made.  A block a 32-column stripe of a
// tile, a warp 32 of its rows.
constexpr int kTailBN = 256, kTailRows = 2 * kBM, kTailThreads = kTailRows;
template <int MODE, bool F32>
__global__ void __launch_bounds__(kTailThreads) join_tail_kernel(const __grid_constant__ Product p) {
    pdl_enter();
    const int t = blockIdx.x / (kTailBN / 32), g = blockIdx.x % (kTailBN / 32);
    int tm, tn;
    tile_at(p, p.whole + t, &tm, &tn);
    const int64_t row0 = (int64_t)tm * kTailRows + threadIdx.x / 32 * 32, n0 = (int64_t)tn * kTailBN + g * 32;
    if (row0 >= p.rows || n0 >= p.cols) return;
    const float *from = p.partial + ((int64_t)t * p.tail_parts * kTailBN + g * 32) * kTailRows + threadIdx.x;
    float v[32];
    bool made = true;
    for (int q = 0; q < p.tail_parts; ++q, from += kTailBN * kTailRows) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(load_4(from + j * kTailRows));
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = q ? v[j] + x[j] : x[j];
        made = made && __float_as_uint(x[0]) != kUnmade;
    }
    if (!__all_sync(0xffffffffu, made)) return;
    const int rows = p.rows - row0 < 32 ? (int)(p.rows - row0) : 32, lane = threadIdx.x & 31;
    const uint32_t step_byte = finish32<MODE, F32>(p.ep, row0, rows, n0, (int)(p.cols - n0 < 32 ? p.cols - n0 : 32), v);
    if (MODE == kForward && p.ep.q && lane < rows) store_steps<32>(p.ep, row0 + lane, n0, step_byte);
}

// ---------------------------------------------------------------------------
// a single row

// The forward product of one row, a single token's: the weights are read once
// and all else is latency, so the multiplications are the ordinary ones and
// nothing of the tensor core is set up.  A block takes 64 columns and its share
// of k, in rounds of kTokenRound; eight lanes read 128 bytes of a weight row, a
// thread kTokenFlight rows at once.  The threads', the warps' and the cluster's sums
// are added in fixed orders.
constexpr int kTokenCols = 64, kTokenThreads = 256, kTokenFlight = 16, kTokenRound = kTokenThreads / 8 * kTokenFlight;
struct Token {
    const uint16_t *x, *w;
    int64_t ld_w, cols, k, k_each;  // k_each: k of a block, whole rounds
    Epilogue ep;
};

// `count` neighbouring bf16 values (none where it is not above 0), zeros after
// them; eight in one access
__device__ __forceinline__ uint4 load8(const uint16_t *p, int64_t count) {
    if (count >= 8) return load_16(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (2 * i < count ? p[2 * i] : 0u) | (2 * i + 1 < count ? (uint32_t)p[2 * i + 1] : 0u) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

template <bool F32>
__global__ void __launch_bounds__(kTokenThreads, 2) token_kernel(const __grid_constant__ Token p) {
    namespace cg = cooperative_groups;
    __shared__ float part[kTokenThreads / 32][kTokenCols], sum[kTokenCols];
    pdl_enter();
    const cg::cluster_group cluster = cg::this_cluster();
    const int splits = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t col0 = (int64_t)(blockIdx.x / splits) * kTokenCols, col = col0 + threadIdx.x % 8 * 8;
    const int64_t end = p.k < (rank + 1) * p.k_each ? p.k : (rank + 1) * p.k_each;
    float acc[8] = {};
    for (int64_t k = rank * p.k_each + threadIdx.x / 8 * kTokenFlight; k < end; k += kTokenRound) {
        uint4 w[kTokenFlight], x[kTokenFlight / 8];
#pragma unroll
        for (int u = 0; u < kTokenFlight; ++u) w[u] = load8(p.w + (k + u) * p.ld_w + col, k + u < end ? p.cols - col : 0);
#pragma unroll
        for (int u = 0; u < kTokenFlight / 8; ++u) x[u] = load8(p.x + k + 8 * u, end - k - 8 * u);
#pragma unroll
        for (int u = 0; u < kTokenFlight; ++u) {
            float wf[8], xf[8];
            unpack8(w[u], wf);
            unpack8(x[u / 8], xf);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(xf[u % 8], wf[j], acc[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 8);
        acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 16);
        if (lane < 8) part[warp][lane * 8 + j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < kTokenCols) {
        float t = part[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kTokenThreads / 32; ++w) t += part[w][threadIdx.x];
        sum[threadIdx.x] = t;
    }
    cluster.sync();
    // two warps of the cluster finish 32 columns each
    const int g = splits > 1 ? rank : warp;
    const int64_t n0 = col0 + g * 32;
    if ((splits == 1 || warp == 0) && g < kTokenCols / 32 && n0 < p.cols) {
        float t = 0.0f, v[32];
        for (int q = 0; q < splits; ++q) t += *cluster.map_shared_rank(&sum[g * 32 + lane], q);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __shfl_sync(0xffffffffu, t, j);
        const uint32_t step_byte = finish32<kForward, F32>(p.ep, 0, 1, n0, (int)(p.cols - n0 < 32 ? p.cols - n0 : 32), v);
        if (p.ep.q && lane == 0) store_steps<32>(p.ep, 0, n0, step_byte);
    }
    cluster.sync();  // no block's memory goes while another may read it
}

// ---------------------------------------------------------------------------
// operands that TMA cannot read where they lie

// An operand to bring into the workspace, as bf16 rows on 32-byte boundaries:
// a bf16 matrix of any stride, or an 8-bit checkpoint (through its activation).
struct Layout {
    const uint16_t *x;  // null: the checkpoint
    int64_t ld, rows, cols;
    uint16_t *out;
    int64_t ldo;
    PackParams kept;
    int64_t blocks;  // that work on it
};
struct Layouts {
    Layout a, b;
};

constexpr int kLayoutThreads = 256;

// Eight columns a thread.  A row may start at any 2-byte address: the two
// aligned 16-byte words around the eight values are loaded and shifted, except
// at the matrix's own ends, beyond which nothing is read.
__device__ __forceinline__ void lay_out(const Layout &l, int64_t block) {
    const int64_t units = ceil_div<int64_t>(l.cols, 8), total = l.rows * units;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(l.x), hi = reinterpret_cast<uintptr_t>(l.x + (l.rows - 1) * l.ld + l.cols);
    for (int64_t u = block * kLayoutThreads + threadIdx.x; u < total; u += l.blocks * kLayoutThreads) {
        int64_t r, c;
        row_of(u, units, total, &r, &c);
        c *= 8;
        const uint16_t *src = l.x + r * l.ld + c;
        const uintptr_t at = reinterpret_cast<uintptr_t>(src), word = at & ~(uintptr_t)15;
        uint32_t w[8];
        if (c + 8 <= l.cols && word >= lo && word + 32 <= hi) {
            const uint4 x = load_16(reinterpret_cast<const void *>(word)), y = load_16(reinterpret_cast<const void *>(word + 16));
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
            if (at & 8)
#pragma unroll
                for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
            if (at & 4)
#pragma unroll
                for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
            if (at & 2)
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t even = c + 2 * k < l.cols ? src[2 * k] : 0, odd = c + 2 * k + 1 < l.cols ? src[2 * k + 1] : 0;
                w[k] = even | odd << 16;
            }
        }
        *reinterpret_cast<uint4 *>(l.out + r * l.ldo + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__global__ void __launch_bounds__(kLayoutThreads) layout_kernel(const Layouts p) {
    pdl_enter();
    const bool first = blockIdx.x < p.a.blocks;
    const Layout &l = first ? p.a : p.b;
    const int64_t block = first ? blockIdx.x : blockIdx.x - p.a.blocks;
    if (l.x)
        lay_out(l, block);
    else
        unpack_groups<uint16_t>(l.kept, block * kLayoutThreads + threadIdx.x, l.blocks * kLayoutThreads);
}

// Column sums of a bf16 matrix (the bias gradient) in a launch of their own,
// for more than kColumnRows rows.  A block takes a strip of
// LANES * W columns, W at a time per thread, and its share of the rows; the
// blocks of a cluster share a strip, and the first of them adds the others'
// sums, in order, out of their shared memory.  Bound by reading dy once.
constexpr int kColumnThreads = 512;
template <int W, int LANES>
__global__ void __launch_bounds__(kColumnThreads) column_sum_kernel(const uint16_t *dy, int64_t ld, int64_t m, int64_t n, int accumulate, float *db) {
    constexpr int kRowsAtOnce = kColumnThreads / LANES, kCols = LANES * W, kFlight = 16;
    __shared__ float part[kRowsAtOnce][kCols + 1];
    __shared__ float sum[kCols];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    pdl_enter();
    const int share = blockIdx.y, shares = gridDim.y;
    const int64_t r0 = m * share / shares, r1 = m * (share + 1) / shares;
    const int64_t c = (int64_t)blockIdx.x * kCols + threadIdx.x % LANES * W;
    float acc[W] = {};
    if (c < n) {
        for (int64_t r = r0 + threadIdx.x / LANES; r < r1; r += kRowsAtOnce * kFlight) {
            Raw<uint16_t, W> x[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                if (r + f * kRowsAtOnce < r1)
                    x[f].load(dy + (r + f * kRowsAtOnce) * ld + c);
                else
                    x[f].zero();
            }
#pragma unroll
            for (int f = 0; f < kFlight; ++f)
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j] += x[f][j];
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j) part[threadIdx.x / LANES][threadIdx.x % LANES * W + j] = acc[j];
    __syncthreads();
    for (int half = kRowsAtOnce / 2; half > 0; half /= 2) {  // a fixed tree
        for (int u = threadIdx.x; u < half * kCols; u += kColumnThreads) part[u / kCols][u % kCols] += part[u / kCols + half][u % kCols];
        __syncthreads();
    }
    if (threadIdx.x < kCols) sum[threadIdx.x] = part[0][threadIdx.x];
    cluster.sync();
    if (share == 0 && threadIdx.x < kCols) {
        float s = sum[threadIdx.x];
        for (int q = 1; q < shares; ++q) s += cluster.map_shared_rank(sum, q)[threadIdx.x];
        const int64_t at = (int64_t)blockIdx.x * kCols + threadIdx.x;
        if (at < n) db[at] = accumulate ? db[at] + s : s;
    }
    cluster.sync();  // the sums stay until they are read
}

// ---------------------------------------------------------------------------
// host

// ra_selftest_linear_stall: what this thread's next product is to do
struct Stall {
    int block;
    uint64_t limit_ns;  // 0: nothing is asked for
};
thread_local Stall next_stall = {-1, 0};

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// 64 columns by box_rows rows of a row-major bf16 matrix, 128-byte swizzled; what lies outside reads as zero
cudaError_t tensor_map(CUtensorMap *map, const Mat &a, int box_rows) {
    const EncodeTiled f = encode_tiled();
    if (f == nullptr) return cudaErrorNotSupported;
    const int64_t pitch = a.rows > 1 ? a.pitch() : ceil_div<int64_t>(a.row_bytes(), 16) * 16;
    const cuuint64_t dims[2] = {(cuuint64_t)a.cols, (cuuint64_t)a.rows}, strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(a.data), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

bool tma_readable(const Mat &a) { return a.aligned(16) && (a.rows <= 1 || a.pitch() < ((int64_t)1 << 40)); }

// rows of whole sectors (TMA asks for 16 bytes, restoring a checkpoint for 32)
int64_t laid_out_ld(int64_t cols) { return ceil_div<int64_t>(cols, 16) * 16; }
int64_t laid_out_bytes(int64_t rows, int64_t cols) {
    if (rows > 0 && laid_out_ld(cols) > 2 * kMaxSpan / rows) return 4 * kMaxSpan;  // of a matrix that no call takes
    return ceil_div<int64_t>(rows * laid_out_ld(cols) * 2, 256) * 256;
}

// The caller's workspace, handed out front to back from its first 32-byte
// boundary on.
constexpr int64_t kWorkspaceSlack = 32;
struct Workspace {
    char *at, *end;
    bool ok;
    Workspace(void *ws, size_t bytes) : at(nullptr), end(nullptr), ok(ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 16 == 0) {
        if (ws == nullptr) return;
        const uintptr_t skip = -reinterpret_cast<uintptr_t>(ws) & 31;
        at = static_cast<char *>(ws) + (skip < bytes ? skip : bytes);
        end = static_cast<char *>(ws) + bytes;
    }
    void *take(int64_t bytes) {
        if (!ok || bytes > end - at) return nullptr;
        char *p = at;
        at += bytes;
        return p;
    }
};

// a place in the workspace for an operand that TMA cannot read in place
bool place(const Mat &a, Workspace *ws, Mat *out) {
    *out = a;
    if (a.empty() || tma_readable(a)) return true;
    out->ld = laid_out_ld(a.cols);
    out->data = ws->take(laid_out_bytes(a.rows, a.cols));
    return out->data != nullptr;
}

Layout layout_of(const Mat &a, const Mat &placed) {
    Layout l = {};
    if (a.data == placed.data) return l;
    l = Layout{static_cast<const uint16_t *>(a.data), a.ld, a.rows, a.cols, static_cast<uint16_t *>(const_cast<void *>(placed.data)), placed.ld, {}, 0};
    const int64_t blocks = ceil_div<int64_t>(a.rows * ceil_div<int64_t>(a.cols, 8), kLayoutThreads);
    l.blocks = blocks < kMaxGrid / 2 ? blocks : kMaxGrid / 2;
    return l;
}

Layout layout_of(const PackParams &kept) {
    Layout l = {};
    l.kept = kept;
    const int64_t blocks = ceil_div<int64_t>(kept.rows * kept.groups, kLayoutThreads);
    l.blocks = blocks < kMaxGrid / 2 ? blocks : kMaxGrid / 2;
    return l;
}

cudaError_t launch_layouts(const Layouts &p, cudaStream_t s) {
    if (p.a.blocks + p.b.blocks == 0) return cudaSuccess;
    return launch_pdl(layout_kernel, p.a.blocks + p.b.blocks, kLayoutThreads, 0, s, p);
}

cudaError_t sm_count(int *out) {
    static std::atomic<int> known{0};
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known.store(n, std::memory_order_relaxed);
    }
    *out = n;
    return cudaSuccess;
}

cudaError_t launch_column_sum(const Mat &dy, int accumulate, float *db, cudaStream_t s) {
    const bool wide = dy.aligned(16) && dy.cols % 8 == 0;
    auto kernel = wide ? column_sum_kernel<8, 16> : column_sum_kernel<1, 32>;
    // blocks along the rows: at least 256 rows each, at most a portable cluster
    // (16 a cluster were slower: 17 against 13 us at 8192 x 2048, 47 against 31 at 8192 x 8192)
    int shares = 1;
    while (shares < 8 && dy.rows / shares >= 512) shares *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div<int64_t>(dy.cols, wide ? 128 : 32), (unsigned)shares);
    cfg.blockDim = dim3(kColumnThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RA_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = (unsigned)shares;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint16_t *>(dy.data), dy.ld,
                                             dy.rows, dy.cols, accumulate, db);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// The last wave of the pairs' 256 x 256 tiles: how many there are, and in how
// many parts each is made.  In parts where these find SMs that would idle, and
// the steps saved are worth the sums' way through memory and a launch (about 8
// us): 8192 x 8192 x 2048, 256 tiles on 76 pairs, 131 us instead of 142 on zeros and 167
// instead of 181 on normal values.
struct Tail {
    int tiles, parts;
};
Tail tail_of(int64_t rows, int64_t cols, int64_t steps, int sms) {
    const int64_t tiles = ceil_div<int64_t>(rows, kTailRows) * ceil_div<int64_t>(cols, kTailBN), pairs = sms / 2;
    if (pairs == 0 || tiles < pairs || tiles % pairs == 0) return Tail{0, 1};
    const int64_t last = tiles % pairs, parts = pairs / last < 4 ? pairs / last : 4;
    if (parts < 2 || steps - steps / parts < 48) return Tail{0, 1};
    return Tail{(int)last, (int)parts};
}
int64_t tail_bytes(int64_t rows, int64_t cols, int64_t k, int sms) {
    const Tail t = tail_of(rows, cols, ceil_div<int64_t>(k, kBK), sms);
    return (int64_t)t.tiles * t.parts * kTailRows * kTailBN * 4;
}

template <int MODE, int BN, int KIND, int SUMS>
cudaError_t launch_tiles(Product &p, const Mat &a, const Mat &b, int sms, cudaStream_t s, int splits = 1) {
    using S = Shape<BN, KIND>;
    p.tiles_m = p.rows > 0 ? (int)ceil_div<int64_t>(p.rows, S::kRows) : 1;  // no rows: column sums alone
    p.tiles_n = (int)ceil_div<int64_t>(p.cols, BN);
    p.splits = splits;
    p.steps = (int)ceil_div<int64_t>(p.k64, S::kSub);
    cudaError_t e = cudaSuccess;
    if (p.steps > 0) {
        e = tensor_map(&p.a, a, MODE == kWgrad ? kBK : S::kARows);
        if (e == cudaSuccess) e = tensor_map(&p.b, b, MODE == kDgrad ? S::kBCols : kBK);
        if (e != cudaSuccess) return e;
    }
    e = opt_in_smem<product_kernel<MODE, BN, KIND, SUMS>>((int)S::kSmem);
    if (e != cudaSuccess) return e;
    const int cluster = splits * S::kBlocks;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, most = S::kIsSplit ? tiles : sms / S::kBlocks;
    const Tail tail = KIND == kPair && BN == kTailBN && p.partial ? tail_of(p.rows, p.cols, p.k64, sms) : Tail{0, 1};
    p.wait_ns = next_stall.limit_ns ? next_stall.limit_ns : kWaitLimitNs;
    p.stalled = next_stall.limit_ns ? next_stall.block : -1;
    next_stall = {-1, 0};
    p.whole = (int)(tiles - tail.tiles);
    p.tail_parts = tail.parts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * cluster));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RA_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = KIND == kSingle ? 1 : 2;
    e = cudaLaunchKernelEx(&cfg, product_kernel<MODE, BN, KIND, SUMS>, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess || tail.tiles == 0) return e;
    return launch_pdl(join_tail_kernel<MODE, SUMS == kF32>, tail.tiles * (kTailBN / 32), kTailThreads, 0, s, p);
}

// how many clusters of `blocks` blocks of a kernel the device holds at once (0: not known)
template <int MODE, int BN, int KIND, int SUMS>
int64_t clusters_at_once(int blocks) {
    using S = Shape<BN, KIND>;
    static std::atomic<int> known[64][9] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
    n = known[dev][blocks].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (opt_in_smem<product_kernel<MODE, BN, KIND, SUMS>>((int)S::kSmem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, product_kernel<MODE, BN, KIND, SUMS>, &cfg) != cudaSuccess) n = 0;
    known[dev][blocks].store(n, std::memory_order_relaxed);
    return n;
}

// The tile: the widest that leaves half of the SMs or more one.  What bounds
// the smaller products is the rate at which an SM takes tiles in, about 50 bytes
// a clock, so pairs, which share B, do better than single blocks of one width:
// 512 x 3712 x 2560 in a pair's 128 columns 13.3 us, in its 256 21.7; 1024 x 4096 x
// 4096 in 256 columns 24.4 us, in 128 34.0 / 42.2, in 64 75.  With a step or two
// of k the results' writes are all, and single blocks of 128 columns have more
// tiles finishing at once: 8192 x 64 x 4096 19.3 us, a pair's 256 columns 25.2.
// Where even the narrowest tiles leave half of the SMs idle and k is
// long enough, clusters of 2 to 8 blocks split it: the exchange of the sums
// costs about what 8 steps do.  With one row tile, where the weights' stream is
// what counts, up to two blocks an SM.  Split / whole, us (GB300, graph replay):
// 256 x 1024 x 1024 6.8 / 7.4, 512 x 2048 x 512 8.7 / 11.8, 128 x 4096 x 4096
// 11.9 / 20.9, 16 x 2448 x 160 7.3 / 13.2; but 512 x 512 x 2048 7.0 / 5.3 with
// only 4 steps each, and 300 x 3000 x 3000 20.2 / 18.3 with two blocks an SM.
// With 48 steps or more, and 64 or more for four splits, pairs split better than
// single blocks, as long as all of their clusters run at once (a GB300 holds 36
// of two pairs, 15 of four).  Pairs' split / otherwise: 1024 x 4096 x 1024 12.2 / 15.3,
// 256 x 8192 x 2048 15.2 / 20.5, 256 x 8192 x 1536 13.0 / 18.5, 512 x 8192 x 512
// 12.3 / 14.7; but 1024 x 2048 x 1024 9.6 / 9.4 with 32 steps, and 512 x 3712 x 2560
// 20.8 / 13.3 with 40 clusters.
template <int MODE, int SUMS>
cudaError_t launch_width(Product &p, const Mat &a, const Mat &b, int sms, cudaStream_t s) {
    const int64_t tm = ceil_div<int64_t>(p.rows, kBM), narrow = tm * ceil_div<int64_t>(p.cols, 64);
    const bool skinny = MODE != kWgrad && p.rows <= kSkinnyRows;
    const int64_t pairs = ceil_div<int64_t>(p.rows, 2 * kBM) * ceil_div<int64_t>(p.cols, 128);
    if (tm > 1 && pairs * 4 <= sms)
        for (int n = 4; n >= 2; n /= 2)
            if (p.k64 >= (n == 4 ? 64 : 48) && pairs <= clusters_at_once<MODE, 128, kPairSplit, SUMS>(2 * n))
                return launch_tiles<MODE, 128, kPairSplit, SUMS>(p, a, b, sms, s, n);
    int splits = 1;
    while (splits < 8) {
        const bool one_each = narrow * splits * 2 <= sms && p.k64 >= 16 * splits;
        const bool two_each = tm == 1 && narrow * splits <= sms && p.k64 >= (skinny ? 8 : 32) * splits;
        if (!one_each && !two_each) break;
        splits *= 2;
    }
    if constexpr (MODE != kWgrad)
        if (splits > 1 && skinny) return launch_tiles<MODE, 64, kSkinny, SUMS>(p, a, b, sms, s, splits);
    if (splits > 1) return launch_tiles<MODE, 64, kSplit, SUMS>(p, a, b, sms, s, splits);
    if (tm * ceil_div<int64_t>(p.cols, 128) <= sms / 2) return launch_tiles<MODE, 64, kSingle, SUMS>(p, a, b, sms, s);
    const bool few = tm * ceil_div<int64_t>(p.cols, 256) <= sms / 2;
    const bool one_wave = ceil_div<int64_t>(p.rows, 2 * kBM) * ceil_div<int64_t>(p.cols, 128) <= sms / 2;  // of pairs
    if (p.k64 <= 4 || (few && (tm == 1 || !one_wave))) return launch_tiles<MODE, 128, kSingle, SUMS>(p, a, b, sms, s);
    if (few) return launch_tiles<MODE, 128, kPair, SUMS>(p, a, b, sms, s);
    return launch_tiles<MODE, 256, kPair, SUMS>(p, a, b, sms, s);
}

// A single token's product: k among as many blocks as run at once, with a round
// or more each.  With less than a round in all, or with more than four a block (which
// waits for each round's reads before it asks for the next), the tensor cores' few rows do
// better.  This kernel / those, us (weights in L2; from memory where two are given):
// 2048 x 8192 6.4 / 9.5 (9.4 / 10.5), 8192 x 2048 6.5 / 9.2 (9.4 / 10.6), 2048 x
// 2048 4.3 / 6.2, 512 x 512 3.7 / 5.2, 2048 x 32000 27 / 35; but 8192 x 8192, eight rounds,
// 25.7 / 24.5, and 100 x 64 3.9 / 2.9.  Two rows at once were no better than there (11.4 / 9.5).
int token_splits(int64_t cols, int64_t k, int sms) {
    const int64_t tiles = ceil_div<int64_t>(cols, kTokenCols);
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= 2 * (int64_t)sms && k >= 2 * splits * kTokenRound) splits *= 2;
    return splits;
}
template <bool F32>
cudaError_t launch_token(const Token &p, int splits, cudaStream_t s) {
    const int64_t tiles = ceil_div<int64_t>(p.cols, kTokenCols);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * splits));
    cfg.blockDim = dim3(kTokenThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RA_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, token_kernel<F32>, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// out (rows x cols) = epilogue(A B); a and b as they lie in memory
template <int MODE>
cudaError_t launch_product(const Mat &a, const Mat &b, int64_t rows, int64_t cols, int64_t k, Epilogue ep, const Mat &out, const Mat &bias, const Mat &res,
                           Workspace *space, cudaStream_t s, float *db = nullptr, int db_add = 0) {
    Product p = {};
    p.ep = ep;
    if (out.aligned(32) && (res.empty() || res.aligned(32)))
        p.ep.rows_aligned = 32;
    else if (out.esz == 2 && res.empty() && out.aligned(16))
        p.ep.rows_aligned = 16;
    p.ep.bias_aligned = bias.aligned(32);
    p.ep.q_aligned = reinterpret_cast<uintptr_t>(ep.q) % 32 == 0;
    p.rows = rows;
    p.cols = cols;
    p.k64 = rows > 0 ? (int)ceil_div<int64_t>(k, kBK) : 0;
    p.db = db;
    p.dy = static_cast<const uint16_t *>(b.data);
    p.ld_dy = b.ld;
    p.dy_rows = k;
    p.db_add = db_add;
    int sms = 0;
    cudaError_t e = device_error_word(&p.err);
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t tm = ceil_div<int64_t>(rows, kBM), part_bytes = tail_bytes(rows, cols, k, sms);
    if (tm * ceil_div<int64_t>(cols, 64) >= kMaxExtent) return cudaErrorInvalidValue;
    if constexpr (MODE == kForward) {
        Token t{static_cast<const uint16_t *>(a.data), static_cast<const uint16_t *>(b.data), b.ld, cols, k, 0, p.ep};
        const int splits = token_splits(cols, k, sms);
        t.k_each = ceil_div<int64_t>(ceil_div<int64_t>(k, splits), kTokenRound) * kTokenRound;
        if (rows == 1 && k >= kTokenRound && t.k_each <= 4 * kTokenRound)
            return out.esz == 4 ? launch_token<true>(t, splits, s) : launch_token<false>(t, splits, s);
    }
    if (part_bytes > 0) p.partial = static_cast<float *>(space->take(part_bytes));  // without room: tiles whole
    if (out.esz == 4) return launch_width<MODE, kF32>(p, a, b, sms, s);
    return k > kLongSum ? launch_width<MODE, kBf16Long>(p, a, b, sms, s) : launch_width<MODE, kBf16>(p, a, b, sms, s);
}

// the checkpoint's two arrays as matrices
struct Kept {
    Mat q, e;
    bool ok;
};
Kept kept_mats(const int8_t *q, const uint8_t *e, int64_t rows, int64_t cols) {
    const int64_t groups = ceil_div<int64_t>(cols, kGroup);
    Kept k{{q, rows, groups * kGroup, groups * kGroup, 1}, {e, rows, groups, groups, 1}, true};
    k.ok = q != nullptr && e != nullptr && reinterpret_cast<uintptr_t>(q) % 16 == 0 && (k.q.empty() || k.q.pitch() <= kMaxSpan / rows);
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
    for (const Mat &a : {Mat{nullptr, m, k, k, 2}, Mat{nullptr, k, n, n, 2}, Mat{nullptr, m, n, n, 2}})
        if (!size_ok(a)) return 0;
    // at most two of the three matrices are laid out in one call
    const int64_t mk = laid_out_bytes(m, k), kn = laid_out_bytes(k, n), mn = laid_out_bytes(m, n);
    const int64_t least = mk < kn ? (mk < mn ? mk : mn) : (kn < mn ? kn : mn);
    return (size_t)(mk + kn + mn - least + kWorkspaceSlack);
}

size_t ra_linear_split_bytes(int64_t rows, int64_t cols, int64_t k) {
    if (rows < 0 || cols < 0 || k < 0 || rows >= kMaxExtent || cols >= kMaxExtent || k >= kMaxExtent) return 0;
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return 0;
    const int64_t bytes = tail_bytes(rows, cols, k, sms);
    return bytes > 0 ? (size_t)(bytes + kWorkspaceSlack) : 0;
}

ra_status ra_linear(const void *x, int64_t ld_x, const void *w, int64_t ld_w, int64_t m, int64_t k, int64_t n,
                    const void *bias, int bias_dtype, int act, const void *residual, int64_t ld_res, int res_dtype,
                    int8_t *save_q, uint8_t *save_e, void *y, int64_t ld_y, int y_dtype, void *ws, size_t ws_bytes,
                    void *stream) {
    const int ysz = esize(y_dtype);
    if (ysz == 0 || !act_ok(act)) return RA_ERR_INVALID_ARG;
    if ((bias && esize(bias_dtype) == 0) || (residual && esize(res_dtype) == 0)) return RA_ERR_INVALID_ARG;
    const Mat mx{x, m, k, ld_x, 2}, mw{w, k, n, ld_w, 2}, my{y, m, n, ld_y, ysz};
    const Mat mb{bias, bias ? 1 : 0, n, n, bias ? esize(bias_dtype) : 1};
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
    Workspace space(ws, ws_bytes);
    Mat a, b;
    if (!place(mx, &space, &a) || !place(mw, &space, &b)) return RA_ERR_INVALID_ARG;
    if (ws) {
        const Mat wm{ws, 1, (int64_t)ws_bytes, (int64_t)ws_bytes, 1};
        const Mat *all[] = {&mx, &mw, &my, &mb, &mr, &kept.q, &kept.e};
        for (int i = 0; i < (save_q ? 7 : 5); ++i)
            if (mats_overlap(wm, *all[i])) return RA_ERR_OVERLAP;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_layouts(Layouts{layout_of(mx, a), layout_of(mw, b)}, s);
    if (e != cudaSuccess) return cuda_status(e);
    const Epilogue ep{y, bias, residual, save_q, save_e, ld_y, ld_res, ceil_div<int64_t>(n, kGroup), bias_dtype == RA_F32,
                      res_dtype == RA_F32, act, 0};
    return cuda_status(launch_product<kForward>(a, b, m, n, k, ep, my, mb, mr, &space, s));
}

ra_status ra_linear_dgrad(const void *dy, int64_t ld_dy, const void *w, int64_t ld_w, int64_t m, int64_t k, int64_t n,
                          const int8_t *z_q, const uint8_t *z_e, int act, const void *residual, int64_t ld_res, int res_dtype,
                          void *dx, int64_t ld_dx, int dx_dtype, void *ws, size_t ws_bytes, void *stream) {
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
    Workspace space(ws, ws_bytes);
    Mat a, b;
    if (!place(md, &space, &a) || !place(mw, &space, &b)) return RA_ERR_INVALID_ARG;
    if (ws) {
        const Mat wm{ws, 1, (int64_t)ws_bytes, (int64_t)ws_bytes, 1};
        const Mat *all[] = {&md, &mw, &mx, &mr, &kept.q, &kept.e};
        for (int i = 0; i < (act != RA_ACT_NONE ? 6 : 4); ++i)
            if (mats_overlap(wm, *all[i])) return RA_ERR_OVERLAP;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_layouts(Layouts{layout_of(md, a), layout_of(mw, b)}, s);
    if (e != cudaSuccess) return cuda_status(e);
    const Epilogue ep{dx, nullptr, residual, act ? const_cast<int8_t *>(z_q) : nullptr, const_cast<uint8_t *>(z_e), ld_dx, ld_res,
                      ceil_div<int64_t>(k, kGroup), 0, res_dtype == RA_F32, act, 0};
    return cuda_status(launch_product<kDgrad>(a, b, m, k, n, ep, mx, Mat{nullptr, 0, 0, 0, 1}, mr, &space, s));
}

ra_status ra_linear_wgrad(const void *x, int64_t ld_x, const int8_t *z_q, const uint8_t *z_e, int act, const void *dy,
                          int64_t ld_dy, int64_t m, int64_t k, int64_t n, int accumulate, void *dw, int64_t ld_dw,
                          int dw_dtype, float *db, void *ws, size_t ws_bytes, void *stream) {
    const int wsz = esize(dw_dtype);
    // (an empty checkpoint's arrays may have no address)
    const bool from_kept = x == nullptr && (z_q != nullptr || z_e != nullptr || (act != RA_ACT_NONE && (m == 0 || k == 0)));
    if (wsz == 0 || !act_ok(act) || (!from_kept && act != RA_ACT_NONE)) return RA_ERR_INVALID_ARG;
    if (x != nullptr && (z_q != nullptr || z_e != nullptr)) return RA_ERR_INVALID_ARG;
    const Mat mx{x, from_kept ? 0 : m, k, from_kept ? k : ld_x, 2}, md{dy, m, n, ld_dy, 2}, mw{dw, k, n, ld_dw, wsz};
    const Mat mb{db, db ? 1 : 0, n, n, 4};
    if (!mat_ok(mx) || !mat_ok(md) || !mat_ok(mw) || !mat_ok(mb)) return RA_ERR_INVALID_ARG;
    if (m < 0 || m >= kMaxExtent) return RA_ERR_INVALID_ARG;
    const Kept kept = kept_mats(z_q, z_e, m, k);
    if (from_kept && !kept.q.empty() && !kept.ok) return RA_ERR_INVALID_ARG;
    const Mat *in[] = {&mx, &md, &kept.q, &kept.e};
    for (int i = 0; i < (from_kept ? 4 : 2); ++i)
        if (mats_overlap(mw, *in[i]) || mats_overlap(mb, *in[i])) return RA_ERR_OVERLAP;
    if (mats_overlap(mw, mb)) return RA_ERR_OVERLAP;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Workspace space(ws, ws_bytes);
    if (mw.empty() && mb.empty()) return RA_OK;
    Mat a, b;
    if (from_kept) {
        // the checkpoint's values (after the activation) as bf16 rows
        a = Mat{nullptr, m, k, laid_out_ld(k), 2};
        if (!a.empty() && (a.data = space.take(laid_out_bytes(m, k))) == nullptr) return RA_ERR_INVALID_ARG;
    } else if (!place(mx, &space, &a)) {
        return RA_ERR_INVALID_ARG;
    }
    if (!place(md, &space, &b)) return RA_ERR_INVALID_ARG;
    if (ws) {
        const Mat wm{ws, 1, (int64_t)ws_bytes, (int64_t)ws_bytes, 1};
        const Mat *all[] = {&mx, &md, &mw, &mb, &kept.q, &kept.e};
        for (int i = 0; i < (from_kept ? 6 : 4); ++i)
            if (mats_overlap(wm, *all[i])) return RA_ERR_OVERLAP;
    }
    const PackParams kept8{nullptr, const_cast<void *>(a.data), a.ld, const_cast<int8_t *>(z_q), const_cast<uint8_t *>(z_e), m, k, ceil_div<int64_t>(k, kGroup), act};
    const Layout lay_a = !from_kept ? layout_of(mx, a) : a.empty() ? Layout{} : layout_of(kept8);
    cudaError_t e = launch_layouts(Layouts{lay_a, layout_of(md, b)}, s);
    if (e != cudaSuccess) return cuda_status(e);
    if (db && m > kColumnRows) {
        e = launch_column_sum(b, accumulate, db, s);
        if (e != cudaSuccess || mw.empty()) return cuda_status(e);
        db = nullptr;
    }
    const Epilogue ep{dw, nullptr, accumulate ? dw : nullptr, nullptr, nullptr, ld_dw, ld_dw, 0, 0, dw_dtype == RA_F32, 0, 0};
    const Mat none{nullptr, 0, 0, 0, 1};
    return cuda_status(launch_product<kWgrad>(a, b, k, n, m, ep, mw, none, accumulate ? mw : none, &space, s, db, accumulate));
}

ra_status ra_selftest_linear_stall(int block, int timeout_us) {
    if (block < 0 || timeout_us < 1 || timeout_us > 10000000) return RA_ERR_INVALID_ARG;
    next_stall = {block, (uint64_t)timeout_us * 1000};
    return RA_OK;
}

}  // extern "C"
