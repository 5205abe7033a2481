// op_logprobs.cu -- log probabilities of given tokens with their distribution's
// entropy and its most likely alternatives, and the logits' gradient:
// ra_logprobs and ra_logprobs_grad.
#include "op_rows.cuh"

namespace ra {
namespace op {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = INFINITY;

// ---------------------------------------------------------------------------
// forward
//
// One pass over the logits: every thread keeps the sums of 2^y and y 2^y relative
// to one of its logits, and these shares are joined at the row's end (Growing, Share).
// WARPS warps take a row, in tiles of kSlots 16-byte vectors a thread.  A tile is read
// asynchronously into the thread's own places in shared memory; as a place is read
// from there, the same place of the next tile, of this row or the next, is on its
// way: no thread waits for another's loads.  Rows of any alignment: the few logits
// before the first and after the last whole vector are one more value of the first
// threads.
//
// Without alternatives memory bounds it: 8192 x 32000 bf16 84 us (6.2 TB/s), 5 us a row
// and block, three blocks an SM.  8 alternatives make it 142: their bound, the second
// look and the order are one after another in a row, in eight warps that meet, and
// shared memory has room for three rows an SM.

constexpr int kSlots = 16, kLogThreads = 256;

struct LogParams {
    const void *logits, *ids;
    float *logp, *lse, *entropy, *top_logp;
    int64_t *top_ids;
    int64_t ld, rows;
    int vocab, top, groups, id_bytes;  // groups: the next power of 2 to top
    float scale, scale2, reach, far;  // scale2: scale / ln 2; reach: 200 / scale2, beyond which 2^y is 0; far: kMostBits / scale2
};

// A logit and its index as a number that orders as the alternatives do: by
// value, among equals by falling index.  0 comes after every token that can be.
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);  // one zero
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }
__device__ __forceinline__ uint64_t rank_of(float z, uint32_t i) { return z == -kInf ? 0 : (uint64_t)key_of(z) << 32 | ~i; }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

// A share of a row: m one of its logits, s the sum of 2^y, w that of y 2^y, with
// y = (z - m) scale2 held to at least kLeast, where 2^y is 0 (the exponential
// flushes what is below 2^-126): so a token that cannot be, or is that far off,
// adds 0 and no 0 * infinity.  A NaN stays one.  m need not be the largest, but no
// logit is more than kMostBits above it: no sum can leave binary32, and a share whose
// m is so far below another's that its factor is 0 is worth less than 2^-60 of the
// other.  An empty share has m minus infinity and s = w = 0.
struct Share {
    float m, s, w;
};
constexpr float kLeast = -160.0f, kMostBits = 16.0f;
__device__ __forceinline__ float at_least(float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(kLeast));
    return r;
}
__device__ __forceinline__ float at_most_0(float y) {
    float r;
    asm("min.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(y));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN aside
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float base_of(float m) { return m == -kInf ? 0.0f : m; }
__device__ __forceinline__ void rebase(Share &a, float m, float scale2) {
    const float y = at_least((a.m - base_of(m)) * scale2), f = fast_exp2(y);
    a.w = f * fmaf(y, a.s, a.w);
    a.s = f * a.s;
    a.m = m;
}
// the warp's shares as one, in every lane
__device__ __forceinline__ Share join_lanes(Share a, float scale2) {
    rebase(a, value_of(__reduce_max_sync(0xffffffffu, key_of(a.m))), scale2);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
    return a;
}

// A 16-byte vector of logits as it lies in memory.
template <class T>
struct Vec {
    static constexpr int kEach = 16 / sizeof(T);
    uint32_t w[4];
    __device__ __forceinline__ void take(uint32_t shared) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(shared) : "memory");
    }
    __device__ __forceinline__ void load(const T *p) {
        const uint4 q = load_16(p);
        w[0] = q.x;
        w[1] = q.y;
        w[2] = q.z;
        w[3] = q.w;
    }
    __device__ __forceinline__ float at(int j) const {  // j not a constant
        const int k = sizeof(T) == 4 ? j : j / 2;
        const uint32_t v = k < 2 ? (k == 0 ? w[0] : w[1]) : (k == 2 ? w[2] : w[3]);
        return __uint_as_float(sizeof(T) == 4 ? v : j & 1 ? v & 0xffff0000u : v << 16);
    }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[j]);
        else
            return j & 1 ? __uint_as_float(w[j / 2] & 0xffff0000u) : __uint_as_float(w[j / 2] << 16);
    }
};
// the largest bf16 not above x, twice in a word
__device__ __forceinline__ uint32_t floor_bf16x2(float x) {
    const uint32_t b = __float_as_uint(x), h = (b & 0x80000000u ? b + 0xffffu : b) >> 16;
    return __byte_perm(h, h, 0x1010);
}
__device__ __forceinline__ uint32_t larger_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <class T>
__device__ __forceinline__ float largest(const Vec<T> &v) {
    float m = fmaxf(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < Vec<T>::kEach; j += 2) m = max3(m, v[j], v[j + 1]);
    return m;
}

// the largest of a batch, NaN aside (NaN if there is nothing else)
template <class T, int BATCH>
__device__ __forceinline__ float largest_of(const Vec<T> (&x)[BATCH]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t c[BATCH], m;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            c[i] = x[i].w[0];
#pragma unroll
            for (int k = 1; k < 4; ++k) asm("max.bf16x2 %0, %0, %1;" : "+r"(c[i]) : "r"(x[i].w[k]));
        }
        m = c[0];
#pragma unroll
        for (int i = 1; i < BATCH; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(c[i]));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
        float m = largest(x[0]);
#pragma unroll
        for (int i = 1; i < BATCH; ++i) m = max3(max3(m, x[i][0], x[i][1]), x[i][2], x[i][3]);
        return m;
    }
}

// A thread's share of a row as it grows: the logit m that its sums are relative to, and
// the tile's sums in pairs.  A batch with a logit above `above` first makes its largest
// the m (so does the first batch: m begins as minus infinity), which scales what has
// been summed.  So a finite mask costs little more than minus infinity: 8192 x 32000
// bf16 with the first half at the type's lowest value take 92 us, at minus infinity 84,
// unmasked 84.  (The warp's largest as the first m would take 84 and not 113 where 95 %
// at random are at -10^4, and ordinary rows 1 to 2 % more; to look at a batch's sums
// instead of its largest logit takes 87.)
//
// y = (z - m) scale2.  Where m allows it (near) two bf16 logits take one instruction
// less, and their bounds one less (84 us; 91 without; binary32 gains nothing by it):
// y = z scale2 - off, off the rounded m scale2, below 2^12, so that what the rounding
// left (`by`, at most 2^-13) goes out of the sums by its first-order factor, within
// 4e-9; and logits are held in pairs, before they are taken apart, to a least value
// whose exponential is 0 (low), which there is unless m is next to the type's lowest.
template <class T>
struct Growing {
    float m, above;
    Pair s2, w2, minus;
    uint32_t low;
    bool near;
    __device__ __forceinline__ explicit Growing(const LogParams &p) : s2(pair(0.0f, 0.0f)), w2(pair(0.0f, 0.0f)) { from(-kInf, p); }
    __device__ __forceinline__ void from(float logit, const LogParams &p) {
        m = logit;
        above = m == -kInf ? m : fminf(m + p.far, 3.402823466e38f);  // plus infinity is above any
        const float base = base_of(m), off = base * p.scale2;
        near = false;
        if constexpr (sizeof(T) == 2) {
            low = floor_bf16x2(base - p.reach);
            near = fabsf(off) < 4096.0f && low != 0xff80ff80u && (base - __uint_as_float(low & 0xffff0000u)) * p.scale2 >= -kLeast;
        }
        minus = both(near ? -off : -base);
    }
    __device__ __forceinline__ float by(const LogParams &p) const {
        float off, same;
        apart(minus, off, same);
        return near ? fmaf(base_of(m), p.scale2, off) : 0.0f;
    }
    // former: the sums of the tiles before, or null
    __device__ __forceinline__ void move(float logit, const LogParams &p, volatile float *former) {
        const float y = at_least(fmaf(m - logit, p.scale2, -by(p))), f = fast_exp2(y);
        w2 = pair_mul(both(f), pair_fma(both(y), s2, w2));
        s2 = pair_mul(both(f), s2);
        if (former != nullptr) {
            former[1] = f * fmaf(y, former[0], former[1]);
            former[0] = f * former[0];
        }
        from(logit, p);
    }
    template <bool NEAR, int BATCH>
    __device__ __forceinline__ void add(Vec<T> (&x)[BATCH], Pair scale2) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
#pragma unroll
            for (int j = 0; j < Vec<T>::kEach; j += 2) {
                if constexpr (NEAR) x[i].w[j / 2] = larger_nan(x[i].w[j / 2], low);
                const Pair z = pair(x[i][j], x[i][j + 1]);
                Pair y = NEAR ? pair_fma(z, scale2, minus) : pair_mul(pair_add(z, minus), scale2);
                float y0, y1;
                apart(y, y0, y1);
                if constexpr (!NEAR) {
                    y0 = at_least(y0);
                    y1 = at_least(y1);
                    y = pair(y0, y1);
                }
                const Pair e = pair(fast_exp2(y0), fast_exp2(y1));
                s2 = pair_add(s2, e);
                w2 = pair_fma(e, y, w2);
            }
        }
    }
    // with the sums in whole
    __device__ __forceinline__ Share share(const LogParams &p, float s, float w) const {
        const float left = by(p), f = fmaf(left, -kLn2, 1.0f);
        return Share{m, s * f, fmaf(-left, s, w) * f};
    }
};

constexpr int kMostTop = RA_LOGPROBS_MAX_TOP;

// What a row's group has in shared memory beside the landing places.  list: the
// best so far, then candidates, of this tile and the last one; far_*: what the
// other blocks of a cluster send to the first.
template <int WARPS, bool TOP, bool CLUSTER>
struct RowRoom {
    static constexpr int kList = !TOP ? 1 : WARPS == 8 ? 224 : 288;  // what three blocks an SM leave room for
    uint64_t list[WARPS == 8 ? 2 : 1][TOP ? kMostTop + kList : 1];  // rows of fewer warps are one tile
    uint64_t far_list[TOP && CLUSTER ? kMostBlocks * kMostTop : 1];
    uint64_t round[WARPS];
    Share shares[2][WARPS];
    Share far_share[CLUSTER ? kMostBlocks : 1];
    uint32_t keys[64];
    int64_t token[2];  // this row's id and the next one's, as they lie in memory
    int count[2];
};

// The `top` highest of list[0 .. n), by one warp: lane j gets the j-th.
__device__ __forceinline__ uint64_t pick(const uint64_t *list, int n, int top, int lane) {
    uint64_t last = ~0ull, mine = 0, best = 0;
    bool look = true;
    for (int k = 0; k < top; ++k) {
        if (look) {
            best = 0;
            for (int i = lane; i < n; i += 32) {
                const uint64_t v = list[i];
                if (v < last && v > best) best = v;
            }
        }
        __syncwarp();
        last = warp_max(best);
        look = best == last;
        if (lane == k) mine = last;
    }
    return mine;
}

// how many of list[0 .. n) are above v
__device__ __forceinline__ int above(const uint64_t *list, int n, uint64_t v) {
    int k = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) k += list[i] > v;
    return k;
}

// one more candidate, as long as the list has room
__device__ __forceinline__ void push(float z, uint32_t i, uint64_t *list, int room, int *count) {
    if (*(volatile int *)count <= room) {
        const int at = atomicAdd(count, 1);
        if (at < room) list[at] = rank_of(z, i);
    }
}
__device__ __forceinline__ float height_at(uint32_t shared) {
    float h;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(h) : "r"(shared) : "memory");
    return h;
}
// The logits from `least` on of a thread's vectors, BATCH a batch and THREADS apart,
// of the `left` that are left of the row from `from` on (index: the first one's).
// The batches that have some (heights: each one's largest, in shared memory) are
// read again from L2.
template <class T, int THREADS, int BATCH>
__device__ __forceinline__ void collect(const T *from, int left, uint32_t index, int slots, uint32_t heights, float least, uint64_t *list, int room, int *count) {
    constexpr int kEach = Vec<T>::kEach;
    uint32_t which = 0;  // batches
#pragma unroll
    for (int i = 0; i < kSlots / BATCH; ++i) which |= i * BATCH < slots && height_at(heights + i * 4) >= least ? 1u << i : 0u;
#pragma unroll 1
    for (; which != 0; which &= which - 1) {
        const int first = (__ffs(which) - 1) * (BATCH * THREADS);
        Vec<T> q[BATCH];
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (left > first + i * THREADS) q[i].load(from + (first + i * THREADS) * kEach);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) hits |= left > first + i * THREADS && largest(q[i]) >= least ? 1u << i : 0u;
#pragma unroll 1
        for (; hits != 0; hits &= hits - 1) {
            const int i = __ffs(hits) - 1;
            Vec<T> x = q[0];
#pragma unroll
            for (int k = 1; k < BATCH; ++k)
                if (k == i) x = q[k];
            uint32_t these = 0;
#pragma unroll
            for (int j = 0; j < kEach; ++j) these |= x[j] >= least ? 1u << j : 0u;
#pragma unroll 1
            for (; these != 0; these &= these - 1) {
                const int j = __ffs(these) - 1;
                push(x.at(j), index + (uint32_t)((first + i * THREADS) * kEach + j), list, room, count);
            }
        }
    }
}

// places worked on at a time; rows of few vectors are not to fill four
template <int WARPS>
constexpr int batch_of() {
    return WARPS == 1 ? 2 : 4;
}
constexpr int kLogBlocks = 3;  // resident on an SM, as far as registers go
// shared memory: the rooms, the batches' largest logits, and a row's `slots` places,
// which begin where a line does
template <int WARPS, bool TOP, bool CLUSTER>
constexpr int log_fixed() {
    return kLogThreads / (WARPS * 32) * (int)sizeof(RowRoom<WARPS, TOP, CLUSTER>) + (TOP ? kLogThreads * kSlots / batch_of<WARPS>() * 4 : 0);
}
template <int WARPS, bool TOP, bool CLUSTER>
constexpr int log_smem(int slots) {
    return ceil_div(log_fixed<WARPS, TOP, CLUSTER>(), 128) * 128 + kLogThreads * slots * 16;
}

template <class T, int WARPS, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(kLogThreads, kLogBlocks) logprobs_kernel(const LogParams p) {
    using Room = RowRoom<WARPS, TOP, CLUSTER>;
    constexpr int kThreads = WARPS * 32, kGroups = kLogThreads / kThreads, kEach = Vec<T>::kEach, kTile = kThreads * kSlots;  // vectors
    constexpr int kBatch = batch_of<WARPS>();
    extern __shared__ __align__(128) unsigned char smem[];
    const int t = threadIdx.x % kThreads, lane = threadIdx.x & 31, warp = t / 32, id = threadIdx.x / kThreads;
    Room &room = reinterpret_cast<Room *>(smem)[id];
    const uint32_t heights = smem_addr(smem) + kGroups * (int)sizeof(Room) + threadIdx.x * (kSlots / kBatch * 4);  // the largest logit of each batch
    const uint32_t land = smem_addr(smem) + log_smem<WARPS, TOP, CLUSTER>(0) + threadIdx.x * 16;  // the thread's places, kPitch apart
    constexpr int kPitch = kLogThreads * 16;
    if (t < 2) room.count[t] = 0;
    group_meet<WARPS>(id);
    pdl_enter();
    const int parts = CLUSTER ? (int)cluster_blocks() : 1, part = CLUSTER ? (int)cluster_block() : 0;
    if constexpr (CLUSTER) cluster_meet();
    // (below 2^31 rows: no sum of these wraps)
    const uint32_t first = CLUSTER ? blockIdx.x / parts : blockIdx.x * kGroups + id, stride = CLUSTER ? gridDim.x / parts : gridDim.x * kGroups, last_row = (uint32_t)p.rows;

    struct Row {  // where a row's whole vectors begin, how many logits are before them, how many vectors there are
        const T *begin;
        int head, vecs;
        // the index of the logit outside the whole vectors that thread t has, or -1
        __device__ __forceinline__ int odd_place(int t, int vocab) const {
            const int i = t < 8 ? t : head + vecs * kEach + t - 8;
            return t < 16 && i < (t < 8 ? head : vocab) ? i : -1;
        }
    };
    auto row_at = [&](uint32_t r) {
        const T *from = static_cast<const T *>(p.logits) + (int64_t)r * p.ld;
        const int head = min((int)(-(reinterpret_cast<intptr_t>(from) / (int)sizeof(T)) & (kEach - 1)), p.vocab);
        return Row{from + head, head, (p.vocab - head) / kEach};
    };
    // the loads of a tile into places i0 .. i0 + 3; `left` vectors are left of the
    // row from `from` on, this thread's first
    auto fetch = [&](int i0, const T *from, int left) {
        const uint32_t to = land + i0 * kPitch;
        from += i0 * kThreads * kEach;
        left -= i0 * kThreads;
        if (left + t >= kBatch * kThreads) {  // all of the group's
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * kPitch), "l"(from + i * kThreads * kEach) : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (left > i * kThreads)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * kPitch), "l"(from + i * kThreads * kEach) : "memory");
                else
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to + i * kPitch), "r"(sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u) : "memory");
            }
        }
    };

    int turn = 0, side = 0;
    const Pair scale2 = both(p.scale2);
    const bool finishes = part == 0 && t == 0 && p.logp != nullptr;  // looks after the given token
    auto fetch_token = [&](uint32_t r) {
        if (!finishes) return;
        const uint32_t to = smem_addr(&room.token[turn]);
        if (p.id_bytes == 8)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(static_cast<const int64_t *>(p.ids) + r) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(static_cast<const int32_t *>(p.ids) + r) : "memory");
    };

    if (first < last_row) {
        const Row row = row_at(first);
        const int v0 = part * kTile + t;
        for (int i0 = 0; i0 < kSlots && i0 * kThreads < row.vecs - v0 + t; i0 += kBatch) fetch(i0, row.begin + (int64_t)v0 * kEach, row.vecs - v0);
        fetch_token(first);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (uint32_t r = first; r < last_row; r += stride) {
        const Row row = row_at(r);
        const int steps = max(1, ceil_div(row.vecs, kTile * parts));
        Share a;
        Growing<T> sums(p);
        volatile float former[2];  // sums of the tiles before, not in registers (there they make 142 us 154, with 8 alternatives)
        // one of the logits outside the whole vectors, for the first 16 threads
        Raw<T, 1> odd_raw, given;
        const int odd_at = row.odd_place(t, p.vocab);
        const bool has_odd = part == 0 && odd_at >= 0;
        if (has_odd) odd_raw.load(row.begin - row.head + odd_at);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        bool inside = false;
        if (finishes) {
            const int64_t i = p.id_bytes == 8 ? *(volatile int64_t *)&room.token[turn] : *(volatile int32_t *)&room.token[turn];
            inside = i >= 0 && i < p.vocab;
            if (inside) given.load(row.begin - row.head + i);
        }
        turn ^= 1;
        int have = 0;  // of the best
        for (int step = 0; step < steps; ++step) {
            const int v0 = (step * parts + part) * kTile + t;
            const int g0 = v0 - t, slots = min(kSlots, ceil_div(row.vecs - g0, kThreads));  // the same for the whole group
            const bool last_step = step + 1 == steps;
            // where the next tile's loads are: this row's, the next row's, or none
            const T *ahead = row.begin + (int64_t)(v0 + kTile * parts) * kEach;
            int ahead_left = row.vecs - (v0 + kTile * parts);
            if (last_step) {
                ahead_left = 0;
                if (r + stride < last_row) {
                    const Row next = row_at(r + stride);
                    ahead = next.begin + (int64_t)(part * kTile + t) * kEach;
                    ahead_left = next.vecs - (part * kTile + t);
                }
            }
            float most = -kInf;  // the largest
            const int ahead_slots = min(kSlots, ceil_div(ahead_left + t, kThreads)), most_slots = max(slots, ahead_slots);
            if (step > 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
            for (int i0 = 0; i0 < most_slots; i0 += kBatch) {
                Vec<T> x[kBatch];
                // places that no vector went to hold minus infinity
#pragma unroll
                for (int i = 0; i < kBatch; ++i) x[i].take(land + (i0 + i) * kPitch);
                if (i0 < ahead_slots) fetch(i0, ahead, ahead_left);  // what these places held has been read
                if (i0 >= slots) continue;
                const float here = largest_of(x);
                if (here > sums.above) sums.move(here, p, WARPS == 8 && step > 0 ? former : nullptr);
                if constexpr (sizeof(T) == 2) {
                    if (sums.near)
                        sums.template add<true>(x, scale2);
                    else
                        sums.template add<false>(x, scale2);
                } else {
                    sums.template add<false>(x, scale2);
                }
                if constexpr (TOP) {
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(heights + i0 / kBatch * 4), "f"(here) : "memory");
                    most = fmaxf(most, here);
                }
            }
            if (last_step && r + stride < last_row) fetch_token(r + stride);
            asm volatile("cp.async.commit_group;" ::: "memory");
            const float odd = has_odd && step == 0 ? odd_raw[0] : -kInf;
            if (WARPS == 8 && !last_step) {  // a tile's sums are added up by themselves
                former[0] = (step > 0 ? former[0] : 0.0f) + pair_sum(sums.s2);
                former[1] = (step > 0 ? former[1] : 0.0f) + pair_sum(sums.w2);
                sums.s2 = sums.w2 = both(0.0f);
            }
            if (last_step) {
                const bool more = WARPS == 8 && step > 0;
                a = sums.share(p, pair_sum(sums.s2) + (more ? former[0] : 0.0f), pair_sum(sums.w2) + (more ? former[1] : 0.0f));
                if (has_odd) {
                    const float z = odd_raw[0];
                    if (z > a.m) rebase(a, z, p.scale2);
                    const float y = at_least((z - base_of(a.m)) * p.scale2), e = fast_exp2(y);
                    a.s += e;
                    a.w = fmaf(e, y, a.w);
                }
                a = join_lanes(a, p.scale2);
                if (WARPS > 1 && lane == 0) room.shares[turn][warp] = a;
            }

            if constexpr (TOP) {
                // A bound that `top` logits reach: of the largest logits of groups of
                // threads the top-th.  The logits that reach it are the candidates.  Up
                // to 8: as many groups as the next power of 2, the least of them; up to
                // 20: 32 groups, each place found by counting; else 64 groups, one by
                // one.  (22 candidates for 8, 31 for 20, 44 for 32, where logits lie at
                // random; more groups cost more than fewer candidates save.)
                constexpr int kEachWarp = 32 / WARPS;  // groups
                const int fine = p.top > 20 ? 2 : 1;   // times as many
                uint32_t key = key_of(fmaxf(most, odd)), other = 0;
                if (WARPS == 1 && fine == 2) {  // a lane's batches are two groups
                    float h[2] = {odd, -kInf};
                    for (int i = 0; i * kBatch < slots; ++i) h[i & 1] = fmaxf(h[i & 1], height_at(heights + i * 4));
                    key = key_of(h[0]);
                    other = key_of(h[1]);
                    room.keys[32 + lane] = other;
                }
                const int lanes = WARPS == 1 ? 1 : 32 / (kEachWarp * fine);  // of a group
                for (int o = lanes / 2; o > 0; o /= 2) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
                if (lane % lanes == 0) room.keys[(warp * 32 + lane) / lanes] = key;
                group_meet<WARPS>(id);
                key = room.keys[lane];
                if (p.top <= 8) {
                    for (int o = p.groups; o < 32; o *= 2) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
                    key = __reduce_min_sync(0xffffffffu, key);
                } else if (fine == 1) {
                    int before = 0;
#pragma unroll 8
                    for (int i = 0; i < 32; ++i) {
                        const uint32_t o = room.keys[i];
                        before += o > key || (o == key && i < lane);
                    }
                    key = __shfl_sync(0xffffffffu, key, __ffs(__ballot_sync(0xffffffffu, before == p.top - 1)) - 1);
                } else {
                    other = room.keys[32 + lane];
                    uint32_t low = 0;
#pragma unroll 1
                    for (int k = 0; k < p.top; ++k) {
                        low = __reduce_max_sync(0xffffffffu, max(key, other));
                        if (lane == __ffs(__ballot_sync(0xffffffffu, max(key, other) == low)) - 1) (key == low ? key : other) = 0;
                    }
                    key = low;
                }
                uint64_t *const list = room.list[WARPS == 8 ? side : 0];
                if (have == p.top) key = max(key, (uint32_t)(list[p.top - 1] >> 32));  // of the best so far
                const float least = fmaxf(value_of(key), -3.402823466e38f);
                int *const count = &room.count[side];
                if (odd >= least) push(odd, odd_at, list + have, Room::kList, count);
                if (most >= least)
                    collect<T, kThreads, kBatch>(row.begin + (int64_t)v0 * kEach, row.vecs - v0, (uint32_t)row.head + (uint32_t)v0 * kEach, slots, heights, least,
                                                 list + have, Room::kList, count);
                group_meet<WARPS>(id);
                int n = *(volatile int *)count;
                if (n > Room::kList) {
                    // too many reach the bound (equal logits): the best one by one
                    uint64_t last = ~0ull;
#pragma unroll 1
                    for (int k = 0; k < p.top; ++k) {
                        uint64_t best = 0;
                        auto look = [&](float z, uint32_t i) {
                            const uint64_t v = rank_of(z, i);
                            if (v < last && v > best) best = v;
                        };
                        const int end = min(row.vecs, g0 + kTile) * kEach;
                        for (int c = v0 * kEach; c < end; c += kThreads * kEach)
                            for (int j = 0; j < kEach; ++j) look(to_f32<T>(row.begin[c + j]), row.head + c + j);
                        look(odd, odd_at);
                        best = warp_max(best);
                        if constexpr (WARPS > 1) {
                            if (lane == 0) room.round[warp] = best;
                            group_meet<WARPS>(id);
#pragma unroll
                            for (int w = 0; w < WARPS; ++w) best = room.round[w] > best ? room.round[w] : best;
                        }
                        last = best;
                        if (t == 0) list[have + k] = best;
                        group_meet<WARPS>(id);
                    }
                    n = p.top;
                }
                n += have;
                // The best of them, in order.  (The other list and count are free: all
                // threads have met twice since they were looked at.)
                if (t == 0) room.count[side ^ 1] = 0;
                have = min(n, p.top);
                side ^= 1;
                const bool few = n <= 64;
                if (warp == 0 || (few && warp * 32 < n)) {
                    const bool out = !CLUSTER && last_step;
                    if (WARPS > 1 && out) a = join_lanes(lane < WARPS ? room.shares[turn][lane] : Share{-kInf, 0.0f, 0.0f}, p.scale2);
                    const bool odd_row = a.s != a.s;
                    const float base = base_of(a.m), log_s = logf(a.s);
                    auto emit = [&](int k, uint64_t v) {
                        if (out) {
                            p.top_ids[(int64_t)r * p.top + k] = odd_row || v == 0 ? -1 : (int64_t)(uint32_t)~(uint32_t)v;
                            p.top_logp[(int64_t)r * p.top + k] = odd_row ? a.s : v == 0 ? -kInf : (value_of((uint32_t)(v >> 32)) - base) * p.scale - log_s;
                        } else {
                            room.list[WARPS == 8 ? side : 0][k] = v;  // (never with fewer warps)
                        }
                    };
                    if (few) {  // each finds its place by counting those above it
                        for (int i = t; i < n; i += kThreads) {
                            const uint64_t v = list[i];
                            const int k = above(list, n, v);
                            if (k < p.top) emit(k, v);
                        }
                        if (t >= have && t < p.top) emit(t, 0);
                    } else {  // one by one, by one warp
                        const uint64_t mine = pick(list, n, p.top, lane);
                        if (lane < p.top) emit(lane, mine);
                    }
                }
            }
        }

        if constexpr (WARPS > 1) {
            if (!TOP || CLUSTER) {
                group_meet<WARPS>(id);
                if (warp == 0) a = join_lanes(lane < WARPS ? room.shares[turn][lane] : Share{-kInf, 0.0f, 0.0f}, p.scale2);
            }
        }
        if constexpr (CLUSTER) {
            if (warp == 0) {
                if (lane == 0) {
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(place_in(&room.far_share[part].m, 0)), "f"(a.m) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(place_in(&room.far_share[part].s, 0)), "f"(a.s) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(place_in(&room.far_share[part].w, 0)), "f"(a.w) : "memory");
                }
                if constexpr (TOP) {
                    const uint64_t v = lane < have ? room.list[side][lane] : 0;
                    if (lane < p.top) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(place_in(&room.far_list[part * p.top + lane], 0)), "l"(v) : "memory");
                }
            }
            cluster_meet();
            if (part == 0 && (TOP || warp == 0)) {
                a = join_lanes(lane < parts ? room.far_share[lane] : Share{-kInf, 0.0f, 0.0f}, p.scale2);
                if constexpr (TOP) {
                    const bool odd_row = a.s != a.s;
                    const float base = base_of(a.m), log_s = logf(a.s);
                    int there = 0;
                    for (int i = t; i < parts * p.top; i += kThreads) {
                        const uint64_t v = room.far_list[i];
                        const int k = v ? above(room.far_list, parts * p.top, v) : kMostTop;
                        if (k < p.top) {
                            p.top_ids[(int64_t)r * p.top + k] = odd_row ? -1 : (int64_t)(uint32_t)~(uint32_t)v;
                            p.top_logp[(int64_t)r * p.top + k] = odd_row ? a.s : (value_of((uint32_t)(v >> 32)) - base) * p.scale - log_s;
                        }
                    }
                    if (warp == 0) {
                        there = above(room.far_list, parts * p.top, 0);
                        if (lane >= there && lane < p.top) {
                            p.top_ids[(int64_t)r * p.top + lane] = -1;
                            p.top_logp[(int64_t)r * p.top + lane] = odd_row ? a.s : -kInf;
                        }
                    }
                }
            }
        }
        if (part == 0 && t == 0) {
            const bool none = a.m == -kInf && a.s == 0.0f;
            const float base = base_of(a.m), log_s = logf(a.s);
            p.lse[r] = none ? -kInf : fmaf(base, p.scale, log_s);
            if (p.entropy != nullptr) {
                const float h = none ? 0.0f : log_s - a.w / a.s * kLn2;
                p.entropy[r] = h < 0.0f ? 0.0f : h;  // by the roundings of a certain token's row
            }
            if (p.logp != nullptr) p.logp[r] = !inside ? 0.0f : none ? -kInf : (given[0] - base) * p.scale - log_s;
        }
        if constexpr (CLUSTER) cluster_meet();  // the first block has read what the others sent
    }
}

template <class T, int WARPS, bool TOP, bool CLUSTER>
cudaError_t launch_logprobs(const LogParams &p, int cluster, cudaStream_t s) {
    // a row of one tile has only the places that it needs
    const int batch = batch_of<WARPS>(), vecs = ceil_div(p.vocab, Vec<T>::kEach), used = ceil_div(ceil_div(vecs, WARPS * 32), batch) * batch;
    const int bytes = log_smem<WARPS, TOP, CLUSTER>(used < kSlots ? used > batch ? used : batch : kSlots);
    const cudaError_t e = opt_in_smem<logprobs_kernel<T, WARPS, TOP, CLUSTER>>(log_smem<WARPS, TOP, CLUSTER>(kSlots));
    if (e != cudaSuccess) return e;
    const int room = (228 << 10) / (bytes + 1024), resident = room < kLogBlocks ? room : kLogBlocks;
    const int64_t blocks = ceil_div<int64_t>(p.rows, kLogThreads / (WARPS * 32)), most = 152 * resident / cluster;
    return launch_clusters(logprobs_kernel<T, WARPS, TOP, CLUSTER>, (blocks < most ? blocks : most) * cluster, cluster, kLogThreads, bytes, s, p);
}

template <class T, bool TOP>
cudaError_t launch_logprobs(const LogParams &p, cudaStream_t s) {
    // As few warps as hold the row in one tile: more rows are under way at once, and fewer
    // warps meet (65536 x 1000 bf16: one warp 46 us, two 94, eight 351; 16384 x 4000 27,
    // 34, 90; 8192 x 8000 two 27, eight 47; 8192 x 8300 four 38, eight 59; x 16000 46, 59;
    // with 8 alternatives 81, 119).  A few rows lose up to 2 us by it.
    const int vecs = ceil_div(p.vocab, Vec<T>::kEach);
    if (vecs <= 32 * kSlots) return launch_logprobs<T, 1, TOP, false>(p, 1, s);
    if (vecs <= 64 * kSlots) return launch_logprobs<T, 2, TOP, false>(p, 1, s);
    if (vecs <= 128 * kSlots) return launch_logprobs<T, 4, TOP, false>(p, 1, s);
    // few long rows: clusters share a row, while all blocks run at once (16 x 131071
    // binary32 6.5 us, 12.4 a block a row; with 8 alternatives 12 and 28)
    const int64_t tiles = ceil_div(vecs, kLogThreads * kSlots);
    int cluster = 1;
    while (cluster < kMostBlocks && cluster < tiles && p.rows * cluster * 2 <= 152 * 2) cluster *= 2;
    return cluster == 1 ? launch_logprobs<T, 8, TOP, false>(p, 1, s) : launch_logprobs<T, 8, TOP, true>(p, cluster, s);
}

// ---------------------------------------------------------------------------
// backward
//
// d = q (c0 + c1 y) for y = log2 p, q = 2^y, and scale g more at the given token:
// c0 = -scale (g + e H), c1 = -scale e ln 2.  y = (z scale - lse) log2 e, the difference
// by one rounding: what is left is lse's own, which is not to make a p above 1.
//
// LANES lanes take a stretch of a row, kFlight vectors of 8 logits a lane: a warp, or
// for short rows a quarter of one, so that four rows' few numbers and logits are under
// way at once (65536 x 100 bf16 20 us a warp a row, 7 so; x 257 25 and 13; x 512 29 and
// 24; from 600 on the same).  Memory bounds the long rows: 8192 x 32000 bf16 150 us,
// 7.0 TB/s (152 without arithmetic on pairs).

constexpr int kGradThreads = 256, kFlight = 4;

struct LogGradParams {
    const void *logits, *ids;
    const float *lse, *entropy, *g, *ge;
    void *out;
    int64_t ld, ld_out, rows, stretches;  // of a row
    int vocab, id_bytes;
    float scale;
};

template <class T, class TO, bool ENTROPY, int LANES>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const LogGradParams p) {
    pdl_enter();
    constexpr int kStretch = LANES * kFlight, kAtOnce = kGradThreads / LANES;  // vectors, stretches
    const int lane = threadIdx.x % LANES;
    const int64_t total = p.rows * p.stretches;
    for (int64_t u = (int64_t)blockIdx.x * kAtOnce + threadIdx.x / LANES; u < total; u += (int64_t)gridDim.x * kAtOnce) {
        int64_t r, k;
        row_of(u, p.stretches, total, &r, &k);
        const T *row = static_cast<const T *>(p.logits) + r * p.ld;
        TO *out = static_cast<TO *>(p.out) + r * p.ld_out;
        // whole vectors of 8 begin where the narrower type's do; rows whose two
        // sides disagree there are done value by value
        constexpr int kMask = sizeof(T) == 4 && sizeof(TO) == 4 ? 3 : 7;
        const intptr_t narrow = sizeof(T) <= sizeof(TO) ? reinterpret_cast<intptr_t>(row) / (int)sizeof(T) : reinterpret_cast<intptr_t>(out) / (int)sizeof(TO);
        int head = min((int)(-narrow & kMask), p.vocab), vecs = (p.vocab - head) / 8;
        if (((reinterpret_cast<uintptr_t>(row + head) | reinterpret_cast<uintptr_t>(out + head)) & 15) != 0) vecs = 0;
        Raw<T, 8> x[kFlight];
        const int v0 = (int)k * kStretch + lane;
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (v0 + LANES * i < vecs) x[i].load(row + head + (int64_t)(v0 + LANES * i) * 8);
        const int64_t id = p.g == nullptr ? -1 : p.id_bytes == 8 ? static_cast<const int64_t *>(p.ids)[r] : static_cast<const int32_t *>(p.ids)[r];
        const float lse = p.lse[r], given = p.g == nullptr ? 0.0f : p.g[r];
        const float ge = ENTROPY ? p.ge[r] : 0.0f, h = ENTROPY ? p.entropy[r] : 0.0f;
        // none: no token can be, or lse is so low that its rounding leaves p no digit: zeros
        const bool none = lse < -16777216.0f, inside = id >= 0 && id < p.vocab;
        const int at = none || !inside ? -1 : (int)id;
        const float g = inside ? given : 0.0f, off = none ? 0.0f : -lse, hot = p.scale * g;
        const float c0 = none ? 0.0f : ENTROPY ? -p.scale * fmaf(ge, h, g) : -hot, c1 = none ? 0.0f : -p.scale * kLn2 * ge;
        const Pair scale = both(p.scale), offs = both(off);
        auto slopes = [&](float z0, float z1, float &d0, float &d1) {
            float y0, y1;
            apart(pair_fma(pair(z0, z1), scale, offs), y0, y1);
            apart(pair_mul(pair(at_most_0(y0), at_most_0(y1)), both(kLog2e)), y0, y1);
            if constexpr (ENTROPY) {
                y0 = at_least(y0);
                y1 = at_least(y1);
                d0 = fast_exp2(y0) * fmaf(c1, y0, c0);
                d1 = fast_exp2(y1) * fmaf(c1, y1, c0);
            } else {
                d0 = fast_exp2(y0) * c0;
                d1 = fast_exp2(y1) * c0;
            }
        };
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            if (v0 + LANES * i >= vecs) break;
            const int c = head + (v0 + LANES * i) * 8;
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) slopes(x[i][j], x[i][j + 1], d[j], d[j + 1]);
            if ((unsigned)(at - c) < 8u) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at - c == j) d[j] += hot;
            }
            store_w<TO, 8>(out + c, d);
        }
        auto one = [&](int64_t c) {
            float d, same;
            slopes(to_f32<T>(row[c]), 0.0f, d, same);
            if (c == at) d += hot;
            out[c] = from_f32<TO>(d);
        };
        if (vecs == 0) {
            const int64_t end = k + 1 < p.stretches ? (k + 1) * kStretch * 8 : p.vocab;
            for (int64_t c = k * kStretch * 8 + lane; c < end; c += LANES) one(c);
        } else if (k == 0) {  // the values outside the whole vectors
#pragma unroll
            for (int i = lane; i < 16; i += LANES) {
                const int c = i < 8 ? i : head + vecs * 8 + i - 8;
                if (c < (i < 8 ? head : p.vocab)) one(c);
            }
        }
    }
}

template <class T, class TO, int LANES>
cudaError_t launch_logprobs_grad(LogGradParams p, cudaStream_t s) {
    p.stretches = p.vocab < 8 ? 1 : ceil_div<int64_t>(p.vocab / 8, LANES * kFlight);
    const int64_t blocks = ceil_div<int64_t>(p.rows * p.stretches, kGradThreads / LANES), grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    return launch_pdl(p.ge ? logprobs_grad_kernel<T, TO, true, LANES> : logprobs_grad_kernel<T, TO, false, LANES>, grid, kGradThreads, 0, s, p);
}
template <class T, class TO>
cudaError_t launch_logprobs_grad(const LogGradParams &p, cudaStream_t s) {
    return p.vocab <= 520 ? launch_logprobs_grad<T, TO, 8>(p, s) : launch_logprobs_grad<T, TO, 32>(p, s);
}

bool ids_ok(const void *ids, int id_bytes, int64_t rows) {
    return (id_bytes == 4 || id_bytes == 8) && (rows == 0 || (ids != nullptr && reinterpret_cast<uintptr_t>(ids) % id_bytes == 0));
}
bool scale_ok(float scale) { return scale > 0.0f && scale * kLog2e < kInf; }
bool floats_ok(const void *v) { return reinterpret_cast<uintptr_t>(v) % 4 == 0; }
Mat line(const void *v, int64_t n, int esz) { return Mat{v, v ? 1 : 0, n, n, esz}; }

}  // namespace
}  // namespace op
}  // namespace ra

extern "C" {

ra_status ra_logprobs(const void *logits, int64_t ld, int dtype, int64_t rows, int64_t vocab, const void *ids, int id_bytes,
                      float scale, float *logp, float *lse, float *entropy, int top, int64_t *top_ids, float *top_logp,
                      void *stream) {
    using namespace ra;
    using namespace ra::op;
    const int esz = esize(dtype);
    if (esz == 0 || !scale_ok(scale) || top < 0 || top > RA_LOGPROBS_MAX_TOP) return RA_ERR_INVALID_ARG;
    const Mat a{logits, rows, vocab, ld, esz};
    if (!mat_ok(a)) return RA_ERR_INVALID_ARG;
    if (vocab > RA_LOGPROBS_MAX_VOCAB) return RA_ERR_UNSUPPORTED;
    if (rows == 0) return RA_OK;
    if (lse == nullptr || !floats_ok(lse) || !floats_ok(logp) || !floats_ok(entropy) || (logp != nullptr && !ids_ok(ids, id_bytes, rows))) return RA_ERR_INVALID_ARG;
    if (top > 0 && (top_ids == nullptr || top_logp == nullptr || !floats_ok(top_logp) || reinterpret_cast<uintptr_t>(top_ids) % 8 != 0)) return RA_ERR_INVALID_ARG;
    const Mat i = line(logp ? ids : nullptr, rows, id_bytes);
    const Mat out[] = {line(logp, rows, 4), line(lse, rows, 4), line(entropy, rows, 4), line(top ? top_ids : nullptr, rows * top, 8),
                       line(top ? top_logp : nullptr, rows * top, 4)};
    for (int o = 0; o < 5; ++o) {
        if (mats_overlap(out[o], a) || mats_overlap(out[o], i)) return RA_ERR_OVERLAP;
        for (int q = 0; q < o; ++q)
            if (mats_overlap(out[o], out[q])) return RA_ERR_OVERLAP;
    }
    int groups = 1;
    while (groups < top) groups *= 2;
    const LogParams p{logits, ids, logp, lse, entropy, top_logp, top_ids, ld, rows, (int)vocab, top, groups, id_bytes, scale, scale * kLog2e, 200.0f / (scale * kLog2e), kMostBits / (scale * kLog2e)};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == RA_F32) return cuda_status(top > 0 ? launch_logprobs<float, true>(p, s) : launch_logprobs<float, false>(p, s));
    return cuda_status(top > 0 ? launch_logprobs<uint16_t, true>(p, s) : launch_logprobs<uint16_t, false>(p, s));
}

ra_status ra_logprobs_grad(const void *logits, int64_t ld, int dtype, int64_t rows, int64_t vocab, const void *ids,
                           int id_bytes, float scale, const float *lse, const float *entropy, const float *grad_logp,
                           const float *grad_entropy, void *out, int64_t ld_out, int out_dtype, void *stream) {
    using namespace ra;
    using namespace ra::op;
    const int esz = esize(dtype), eso = esize(out_dtype);
    if (esz == 0 || eso == 0 || !scale_ok(scale)) return RA_ERR_INVALID_ARG;
    const Mat a{logits, rows, vocab, ld, esz}, b{out, rows, vocab, ld_out, eso};
    if (!mat_ok(a) || !mat_ok(b)) return RA_ERR_INVALID_ARG;
    if (vocab > RA_LOGPROBS_MAX_VOCAB) return RA_ERR_UNSUPPORTED;
    if (a.empty()) return RA_OK;
    if (lse == nullptr || !floats_ok(lse) || !floats_ok(entropy) || !floats_ok(grad_logp) || !floats_ok(grad_entropy) ||
        (grad_logp != nullptr && !ids_ok(ids, id_bytes, rows)))
        return RA_ERR_INVALID_ARG;
    if (grad_entropy != nullptr && entropy == nullptr) return RA_ERR_INVALID_ARG;
    const Mat in[] = {line(grad_logp ? ids : nullptr, rows, id_bytes), line(lse, rows, 4), line(grad_entropy ? entropy : nullptr, rows, 4), line(grad_logp, rows, 4),
                      line(grad_entropy, rows, 4)};
    for (const Mat &m : in)
        if (mats_overlap(b, m)) return RA_ERR_OVERLAP;
    if (mats_overlap(a, b) && !same_mat(a, b)) return RA_ERR_OVERLAP;
    const LogGradParams p{logits, ids, lse, entropy, grad_logp, grad_entropy, out, ld, ld_out, rows, 1, (int)vocab, id_bytes, scale};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == RA_F32) return cuda_status(out_dtype == RA_F32 ? launch_logprobs_grad<float, float>(p, s) : launch_logprobs_grad<float, uint16_t>(p, s));
    return cuda_status(out_dtype == RA_F32 ? launch_logprobs_grad<uint16_t, float>(p, s) : launch_logprobs_grad<uint16_t, uint16_t>(p, s));
}

}  // extern "C"
