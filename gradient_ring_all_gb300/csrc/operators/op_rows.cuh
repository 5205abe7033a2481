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

// Sums over a row that WARPS warps hold, or the blocks of a cluster with WARPS
// warps each (CLUSTER).  Lanes are added by shuffles, warps and blocks in their
// order, so a sum has one order and every thread the same result.  Two sets of
// places take turns: whoever writes a set again has met the others after they
// read it.
template <int K, int WARPS, bool CLUSTER>
struct RowSums {
    float warp[2][K][WARPS];
    float block[CLUSTER ? 2 : 1][K][CLUSTER ? kMostBlocks : 1];
};

template <int K, int WARPS, bool CLUSTER>
__device__ __forceinline__ void row_sum(float (&v)[K], RowSums<K, WARPS, CLUSTER> &at, int id, int &turn) {
    static_assert(K == 2, "two sums");
    // the half warps trade one sum for the other, and each half adds up its own
    const int lane = threadIdx.x & 31;
    const float give = lane < 16 ? v[1] : v[0];
    float own = (lane < 16 ? v[0] : v[1]) + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
    for (int o = 8; o > 0; o /= 2) own += __shfl_xor_sync(0xffffffffu, own, o);
    if constexpr (WARPS == 1) {
        v[0] = __shfl_sync(0xffffffffu, own, 0);
        v[1] = __shfl_sync(0xffffffffu, own, 16);
    }
    if constexpr (WARPS > 1) {
        if (lane % 16 == 0) at.warp[turn][lane / 16][threadIdx.x % (WARPS * 32) / 32] = own;
        group_meet<WARPS>(id);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = at.warp[turn][k][0];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) v[k] += at.warp[turn][k][w];
        }
    }
    if constexpr (CLUSTER) {
        const uint32_t blocks = cluster_blocks();
        if (threadIdx.x < blocks) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(place_in(&at.block[turn][k][cluster_block()], threadIdx.x)), "f"(v[k]) : "memory");
        }
        cluster_meet();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = at.block[turn][k][0];
            for (uint32_t b = 1; b < blocks; ++b) v[k] += at.block[turn][k][b];
        }
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
