// op_rows.cuh -- rows that a group of warps holds, and sums over them: what the
// norms and the log probabilities share.
#pragma once

#include "op_common.cuh"

namespace ra {
namespace op {

__device__ __forceinline__ uint32_t cluster_blocks() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_block() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a shared-memory place of another block of the cluster
__device__ __forceinline__ uint32_t place_in(const void *p, uint32_t block) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(block));
    return r;
}

constexpr int kMostBlocks = 8;  // of a cluster

// the threads of one group; `id` tells a block's groups apart
template <int WARPS>
__device__ __forceinline__ void group_meet(int id) {
    if constexpr (WARPS == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "n"(WARPS * 32) : "memory");
}

// Two sums over a row that WARPS warps hold, or the blocks of a cluster with WARPS
// warps each (CLUSTER).  Lanes are added by shuffles, then the warps' sums, which
// every warp writes to every block, by each thread in one order: a sum has one value
// in all of them.  Two sets of places take turns: whoever writes a set again has met
// the others after they read it.
template <int WARPS, bool CLUSTER>
struct RowSums {
    alignas(16) float warp[2][2][CLUSTER ? kMostBlocks : 1][WARPS];
};

template <int WARPS, bool CLUSTER>
__device__ __forceinline__ void row_sum(float (&v)[2], RowSums<WARPS, CLUSTER> &at, int id, int &turn) {
    // the half warps trade one sum for the other, and each half adds up its own
    const int lane = threadIdx.x & 31;
    const float give = lane < 16 ? v[1] : v[0];
    float own = (lane < 16 ? v[0] : v[1]) + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
    for (int o = 8; o > 0; o /= 2) own += __shfl_xor_sync(0xffffffffu, own, o);
    if constexpr (WARPS == 1) {
        v[0] = __shfl_sync(0xffffffffu, own, 0);
        v[1] = __shfl_sync(0xffffffffu, own, 16);
        return;
    }
    const int w = threadIdx.x % (WARPS * 32) / 32;
    uint32_t blocks = 1;
    if constexpr (CLUSTER) {
        blocks = cluster_blocks();
        if (lane % 16 < blocks)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(place_in(&at.warp[turn][lane / 16][cluster_block()][w], lane % 16)), "f"(own) : "memory");
        cluster_meet();
    } else {
        if (lane % 16 == 0) at.warp[turn][lane / 16][0][w] = own;
        group_meet<WARPS>(id);
    }
    constexpr int kEach = WARPS < 4 ? WARPS : 4;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float s[kEach] = {};
#pragma unroll 1
        for (uint32_t b = 0; b < blocks; ++b)
#pragma unroll
            for (int i = 0; i < WARPS; i += kEach) {
                const float *from = &at.warp[turn][k][CLUSTER ? b : 0][i];
                if constexpr (kEach == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(from);
                    s[0] += q.x;
                    s[1] += q.y;
                    s[2] += q.z;
                    s[3] += q.w;
                } else {
                    s[0] += from[0];
                    s[1] += from[1];
                }
            }
        v[k] = kEach == 4 ? (s[0] + s[1]) + (s[kEach - 2] + s[kEach - 1]) : s[0] + s[1];
    }
    turn ^= 1;
}

// Two binary32 values as one operand, and arithmetic on both at once with the
// result in registers of its own.
using Pair = uint64_t;
__device__ __forceinline__ Pair pair(float a, float b) {
    Pair v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ Pair both(float a) { return pair(a, a); }
__device__ __forceinline__ void apart(Pair v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ Pair pair_fma(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float pair_sum(Pair v) {
    float a, b;
    apart(v, a, b);
    return a + b;
}

// launch_pdl, in clusters of `cluster` blocks
template <class K, class... P>
static cudaError_t launch_clusters(K kern, int64_t grid, int cluster, int block, size_t smem, cudaStream_t s, const P &...params) {
    if (cluster == 1) return launch_pdl(kern, grid, block, smem, s, params...);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RA_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, params...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace op
}  // namespace ra
