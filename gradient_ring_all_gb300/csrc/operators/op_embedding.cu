// op_embedding.cu -- rows of an embedding table and the table's gradient:
// ra_embedding_lookup and ra_embedding_grad.
#include "op_common.cuh"

namespace ra {
namespace op {
namespace {

// ---------------------------------------------------------------------------
// lookup: out[t] = scale * table[id_t], zeros for an id outside the table.
// A warp a token; each lane takes W neighbouring columns at a time, 8 such in
// flight.  Bound by the rows' way in and out: 16384 tokens x 2048 bf16 15.7 us,
// 8.6 TB/s counting every row (the frequent ones come from L2); with 4 in
// flight 21.9 us.

constexpr int kLookupThreads = 256, kLookupFlight = 8;

struct LookupParams {
    const void *table;
    const void *ids;
    void *out;
    int64_t ldt, ldo, tokens, vocab, d;
    float scale;
};

template <class I>
__device__ __forceinline__ int64_t load_id(const void *ids, int64_t t, int64_t vocab) {
    const int64_t v = (int64_t) static_cast<const I *>(ids)[t];
    return v >= 0 && v < vocab ? v : -1;
}

template <class T, class I, int W>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const LookupParams p) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kLookupThreads / 32);
    for (int64_t t = (int64_t)blockIdx.x * (kLookupThreads / 32) + threadIdx.x / 32; t < p.tokens; t += step) {
        const int64_t id = load_id<I>(p.ids, t, p.vocab);
        const T *src = static_cast<const T *>(p.table) + (id < 0 ? 0 : id) * p.ldt;
        T *dst = static_cast<T *>(p.out) + t * p.ldo;
        for (int64_t c0 = lane * W; c0 < p.d; c0 += 32 * W * kLookupFlight) {
            Raw<T, W> x[kLookupFlight];
#pragma unroll
            for (int k = 0; k < kLookupFlight; ++k) {
                const int64_t c = c0 + k * 32 * W;
                if (c < p.d && id >= 0) x[k].load(src + c);
            }
#pragma unroll
            for (int k = 0; k < kLookupFlight; ++k) {
                const int64_t c = c0 + k * 32 * W;
                if (c >= p.d) break;
                float y[W];
#pragma unroll
                for (int j = 0; j < W; ++j) y[j] = id >= 0 ? __fmul_rn(x[k][j], p.scale) : 0.0f;
                store_w<T, W>(dst + c, y);
            }
        }
    }
}

// columns a lane takes at once: the widest that every row of all the given
// matrices and the width d allow
int common_width(const Mat &a, const Mat &b, int64_t d, int widest) {
    for (int w = widest; w > 1; w /= 2) {
        const int ba = w * a.esz < 16 ? w * a.esz : 16, bb = w * b.esz < 16 ? w * b.esz : 16;
        if (d % w == 0 && a.aligned(ba) && b.aligned(bb)) return w;
    }
    return 1;
}

template <class T, class I>
cudaError_t launch_lookup(const LookupParams &p, int width, cudaStream_t s) {
    const int64_t blocks = ceil_div<int64_t>(p.tokens, kLookupThreads / 32);
    const int64_t grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    if (width == 8) {
        if constexpr (sizeof(T) == 2) return launch_pdl(lookup_kernel<T, I, 8>, grid, kLookupThreads, 0, s, p);
    }
    if (width == 4) return launch_pdl(lookup_kernel<T, I, 4>, grid, kLookupThreads, 0, s, p);
    if (width == 2) return launch_pdl(lookup_kernel<T, I, 2>, grid, kLookupThreads, 0, s, p);
    return launch_pdl(lookup_kernel<T, I, 1>, grid, kLookupThreads, 0, s, p);
}

// ---------------------------------------------------------------------------
// gradient: out[v] = scale * the sum of grad[t] over the tokens t with
// id_t = v, in binary32 and in the tokens' order.
//
// 1. The token positions are sorted by id, stably: least-significant-digit
//    radix passes of kDigitBits over the ids (an id outside the table counts as
//    `vocab` and sorts behind the rest).  A pass is a histogram of each tile
//    of kSortTile tokens, one scan over all (digit, tile) counts, and a
//    scatter in which each warp ranks its own run of tokens.
// 2. The sorted positions are cut into pieces of 8 to 32 tokens.  A block sums
//    one piece, so an id with very many tokens is spread over many blocks.
//    A run of one id inside a piece is finished there; of a run that crosses
//    a piece's edge the piece keeps a partial sum, and a second kernel joins
//    these in order.  Which values are added in which order is fixed by the
//    ids alone, so results do not change from call to call.
// 3. The table's gradient is set to zero first (unless it is added to), by
//    further blocks of the sorting launches: these few small blocks wait on
//    latency, while the zeros need only the memory's write rate, so the sort
//    costs next to nothing beside them.  Rows that tokens name are written
//    twice; telling them apart first would put the zeros behind the sort.
//
// 8192 tokens into 32000 x 2048 binary32: 39 us sort and zeros (6.7 TB/s), 15 us
// sums, 8 us joins.  65521 tokens of 257 ids, 1022 wide: 22 us sort, 33 us sums
// (4 TB/s, 4-byte accesses), 10 us joins.

constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 4;                         // tokens a thread holds
constexpr int kSortTile = kSortThreads * kSortRounds;  // 1024
constexpr int kPieceMost = 32;

// A share of the table gradient's rows that a launch sets to zero.
struct ZeroShare {
    char *out;
    int64_t pitch, row_bytes, row0, rows;
};
// `bytes` (an even number) from `a` (an even address) on, by threads
// first, first + step, ..: together they write one window that moves through
// the range (stretches of 64 KB a block were a fifth slower)
__device__ __forceinline__ void zero_range(char *a, int64_t bytes, int64_t first, int64_t step) {
    const int64_t head = min((int64_t)(-reinterpret_cast<intptr_t>(a) & 15), bytes), words = (bytes - head) / 16, tail = bytes - head - words * 16;
    if (first < head / 2) reinterpret_cast<uint16_t *>(a)[first] = 0;
    for (int64_t i = first; i < words; i += step) reinterpret_cast<uint4 *>(a + head)[i] = make_uint4(0, 0, 0, 0);
    if (first < tail / 2) reinterpret_cast<uint16_t *>(a + head + words * 16)[first] = 0;
}

// At least 32 KB a block, and 8 blocks an SM at most (one an SM, each looping
// longer, took 76 us for table_grad_step instead of 64).
constexpr int64_t kMaxZeroBlocks = 152 * 8;
inline int64_t zero_blocks(const ZeroShare &z, int64_t most) {
    const int64_t blocks = ceil_div<int64_t>(z.rows * z.row_bytes, 1 << 15);
    return blocks < most ? blocks : most;
}

// the work of block `at` of `blocks`
template <int THREADS>
__device__ __forceinline__ void zero_share(const ZeroShare &z, int64_t at, int64_t blocks) {
    char *base = z.out + z.row0 * z.pitch;
    if (z.row_bytes == z.pitch) {
        zero_range(base, z.rows * z.pitch, at * THREADS + threadIdx.x, blocks * THREADS);
    } else {
        for (int64_t r = at; r < z.rows; r += blocks) zero_range(base + r * z.pitch, z.row_bytes, threadIdx.x, THREADS);
    }
}

struct SortParams {
    ZeroShare zero;
    const void *ids;  // first pass
    const uint32_t *key_in, *pos_in;
    uint32_t *key_out, *pos_out;
    uint32_t *hist;   // [kDigits][tiles]
    uint32_t *joins;  // set to zero by the first launch
    int64_t tokens, vocab;
    int tiles, shift;  // blocks from `tiles` on set zeros
    int passes;
};

template <class I, bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const SortParams &p, int64_t t) {
    if constexpr (FIRST) {
        const int64_t v = load_id<I>(p.ids, t, p.vocab);
        return v < 0 ? (uint32_t)p.vocab : (uint32_t)v;
    } else {
        return p.key_in[t];
    }
}

template <class I, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortParams p) {
    __shared__ uint32_t count[kDigits];
    pdl_enter();
    if (blockIdx.x >= p.tiles) {
        zero_share<kSortThreads>(p.zero, blockIdx.x - p.tiles, gridDim.x - p.tiles);
        return;
    }
    if (FIRST && blockIdx.x == 0 && threadIdx.x == 0) *p.joins = 0;
    for (int k = threadIdx.x; k < kDigits; k += kSortThreads) count[k] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kSortTile;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t t = base + r * kSortThreads + threadIdx.x;
        if (t < p.tokens) atomicAdd(&count[(sort_key<I, FIRST>(p, t) >> p.shift) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < kDigits; k += kSortThreads) p.hist[(int64_t)k * p.tiles + blockIdx.x] = count[k];
}

// exclusive prefix sums over the digits' counts, in place, by one block; a
// thread takes kScanEach neighbours (the array has room for whole ones)
constexpr int kScanThreads = 1024, kScanEach = 16;
__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(const SortParams p) {
    __shared__ uint32_t warp_sum[32];
    pdl_enter();
    if (blockIdx.x >= 1) {
        zero_share<kScanThreads>(p.zero, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    const int64_t n = (int64_t)kDigits * p.tiles;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    uint32_t carry = 0;
    for (int64_t base = 0; base < n; base += kScanThreads * kScanEach) {
        const int64_t i = base + threadIdx.x * kScanEach;
        uint4 *h = reinterpret_cast<uint4 *>(p.hist + i);
        uint32_t v[kScanEach], total = 0;
#pragma unroll
        for (int g = 0; g < kScanEach / 4; ++g) {
            const uint4 x = i < n ? h[g] : make_uint4(0, 0, 0, 0);
            v[4 * g] = x.x;
            v[4 * g + 1] = x.y;
            v[4 * g + 2] = x.z;
            v[4 * g + 3] = x.w;
        }
#pragma unroll
        for (int k = 0; k < kScanEach; ++k) {  // each value becomes the sum of those before it in the thread
            const uint32_t x = v[k];
            v[k] = total;
            total += x;
        }
        uint32_t s = total;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += o;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        if (warp == 0) {
            uint32_t w = warp_sum[lane];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, w, d);
                if (lane >= d) w += o;
            }
            warp_sum[lane] = w;
        }
        __syncthreads();
        const uint32_t before = carry + (warp ? warp_sum[warp - 1] : 0) + s - total;
        if (i < n) {
#pragma unroll
            for (int g = 0; g < kScanEach / 4; ++g)
                h[g] = make_uint4(before + v[4 * g], before + v[4 * g + 1], before + v[4 * g + 2], before + v[4 * g + 3]);
        }
        carry += warp_sum[31];
        __syncthreads();
    }
}

// A warp's ranks of R * 32 keys by one digit: lanes with one digit find each
// other with a match, the digit's count so far (in the warp's own counters)
// gives the rank of the first of them.  A digit of kDigits is no key.
template <int R, class C>
__device__ __forceinline__ void rank_by_digit(C *count, const uint32_t (&digit)[R], uint32_t (&rank)[R]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t peers = __match_any_sync(0xffffffffu, digit[r]);
        const uint32_t below = __popc(peers & ((1u << lane) - 1));
        const bool in = digit[r] < kDigits;
        uint32_t before = 0;
        if (in) before = count[digit[r]];
        __syncwarp();
        if (in && below == 0) count[digit[r]] = (C)(before + __popc(peers));
        __syncwarp();
        rank[r] = before + below;
    }
}

// Each warp owns kSortRounds * 32 consecutive tokens; its counters become
// offsets by a prefix over the warps.
template <class I, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const SortParams p) {
    __shared__ uint32_t count[kSortWarps][kDigits];
    pdl_enter();
    if (blockIdx.x >= p.tiles) {
        zero_share<kSortThreads>(p.zero, blockIdx.x - p.tiles, gridDim.x - p.tiles);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    for (int k = threadIdx.x; k < kSortWarps * kDigits; k += kSortThreads) (&count[0][0])[k] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * kSortTile + warp * (kSortRounds * 32);
    uint32_t key[kSortRounds], pos[kSortRounds], digit[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t t = base + r * 32 + lane;
        const bool in = t < p.tokens;
        key[r] = in ? sort_key<I, FIRST>(p, t) : 0;
        pos[r] = in ? (FIRST ? (uint32_t)t : p.pos_in[t]) : 0;
        digit[r] = in ? (key[r] >> p.shift) & (kDigits - 1) : kDigits;
    }
    rank_by_digit<kSortRounds>(count[warp], digit, rank);
    __syncthreads();
    for (int k = threadIdx.x; k < kDigits; k += kSortThreads) {
        uint32_t at = p.hist[(int64_t)k * p.tiles + blockIdx.x];
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = count[w][k];
            count[w][k] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        if (base + r * 32 + lane >= p.tokens) break;
        const uint32_t at = count[warp][(key[r] >> p.shift) & (kDigits - 1)] + rank[r];
        p.key_out[at] = key[r];
        p.pos_out[at] = pos[r];
    }
}

// Up to 1024 * R tokens: one block sorts them through shared memory, all
// passes in one launch, and the others set zeros.
constexpr int kBlockSortThreads = 1024, kBlockSortWarps = 32;
constexpr int block_sort_smem(int r) { return kBlockSortThreads * r * 8 + kBlockSortWarps * kDigits * 2 + 32 * 4; }
template <class I, int R>
__global__ void __launch_bounds__(kBlockSortThreads) sort_block_kernel(const SortParams p) {
    extern __shared__ uint32_t sorted[];  // keys and positions, then the warps' counters
    pdl_enter();
    if (blockIdx.x >= 1) {
        zero_share<kBlockSortThreads>(p.zero, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    uint32_t *skey = sorted, *spos = sorted + kBlockSortThreads * R;
    uint16_t(*count)[kDigits] = reinterpret_cast<uint16_t(*)[kDigits]>(sorted + 2 * kBlockSortThreads * R);
    uint32_t *warp_sum = reinterpret_cast<uint32_t *>(count + kBlockSortWarps);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, base = warp * (R * 32) + lane, n = (int)p.tokens;
    if (threadIdx.x == 0) *p.joins = 0;
    uint32_t key[R], pos[R], digit[R], rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int t = base + r * 32;
        key[r] = t < n ? sort_key<I, true>(p, t) : 0;
        pos[r] = t;
    }
    for (int pass = 0; pass < p.passes; ++pass) {
#pragma unroll
        for (int r = 0; r < R; ++r) digit[r] = base + r * 32 < n ? (key[r] >> (pass * kDigitBits)) & (kDigits - 1) : kDigits;
        for (int k = lane; k < kDigits; k += 32) count[warp][k] = 0;
        __syncwarp();
        rank_by_digit<R>(count[warp], digit, rank);
        __syncthreads();
        // each digit's total, then its start: a prefix over the digits; the
        // warps' counts become offsets within the digit
        uint32_t total = 0;
        if (threadIdx.x < kDigits) {
            for (int w = 0; w < kBlockSortWarps; ++w) {
                const uint32_t c = count[w][threadIdx.x];
                count[w][threadIdx.x] = (uint16_t)total;
                total += c;
            }
        }
        uint32_t sum = total;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        if (threadIdx.x < kDigits) {
            for (int w = 0; w < warp; ++w) sum += warp_sum[w];
            skey[threadIdx.x] = sum - total;  // the digit's start, read below before the keys move in
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (digit[r] < kDigits) rank[r] += skey[digit[r]] + count[warp][digit[r]];
        __syncthreads();
        const bool last = pass + 1 == p.passes;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (digit[r] == kDigits) continue;
            if (last) {
                p.key_out[rank[r]] = key[r];
                p.pos_out[rank[r]] = pos[r];
            } else {
                skey[rank[r]] = key[r];
                spos[rank[r]] = pos[r];
            }
        }
        if (last) return;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = base + r * 32;
            if (t < n) {
                key[r] = skey[t];
                pos[r] = spos[t];
            }
        }
        __syncthreads();
    }
}

// A run of one id that crosses pieces: the piece it begins in, how many
// pieces after that begin with it, and the id.
struct alignas(16) Join {
    uint32_t first, count, id;
};

struct GradParams {
    const void *grad;
    void *out;
    const uint32_t *key, *pos;
    float *part;      // [2 * pieces][ldp]: the sums of a piece's first and last run
    Join *joins;      // their count (in `first`), then the runs that cross pieces, in any order
    int64_t ldg, ldo, ldp, tokens, vocab, d;
    int64_t pieces;
    int piece;  // tokens a piece
    float scale;
    int accumulate;
    int list;  // whether the runs that cross pieces are to be listed
};

// the first index with key[index] >= v, by a warp (33-way search)
__device__ __forceinline__ int64_t lower_bound_warp(const uint32_t *key, int64_t n, uint32_t v) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = n;  // the answer is in [lo, hi]
    while (hi > lo) {
        const int64_t step = ceil_div<int64_t>(hi - lo, 32);
        const int64_t at = lo + lane * step;
        const uint32_t less = __ballot_sync(0xffffffffu, at < hi && key[at] < v);
        const int k = __popc(less);  // probes 0 .. k-1 are below v
        const int64_t nlo = k ? lo + (k - 1) * step + 1 : lo;
        const int64_t nhi = k < 32 && lo + k * step < hi ? lo + k * step : hi;
        lo = nlo;
        hi = nhi;
    }
    return lo;
}

constexpr int kGradThreads = 128;

// A thread takes kRowBytes of a row, 8 bf16 or 4 binary32 columns, as N
// accesses of W columns, W the widest that the rows' places allow; the
// accesses of a warp are neighbours, so any W is coalesced, and the work per
// token (which run, where it ends) is shared by all N.
constexpr int kRowBytes = 16;

template <class TO, int W>
__device__ __forceinline__ void finish_row(const GradParams &p, uint32_t v, int64_t c, float (&sum)[W]) {
    TO *o = static_cast<TO *>(p.out) + (int64_t)v * p.ldo + c;
    float old[W];
    if (p.accumulate) load_w<TO, W>(o, old);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        sum[j] = __fmul_rn(sum[j], p.scale);
        if (p.accumulate) sum[j] = __fadd_rn(old[j], sum[j]);
    }
    store_w<TO, W>(o, sum);
}

template <class TI, class TO, int W>
__global__ void __launch_bounds__(kGradThreads) grad_pieces_kernel(const GradParams p) {
    constexpr int N = kRowBytes / (W * (int)sizeof(TI)), kFlight = 8;
    __shared__ uint32_t key[kPieceMost + 2], pos[kPieceMost];
    pdl_enter();
    const int64_t i0 = (int64_t)blockIdx.x * p.piece;
    const int count = (int)(p.tokens - i0 < p.piece ? p.tokens - i0 : p.piece);
    constexpr uint32_t kNone = 0xffffffffu;
    if (threadIdx.x < count + 2) {
        const int64_t i = i0 - 1 + threadIdx.x;
        key[threadIdx.x] = i >= 0 && i < p.tokens ? p.key[i] : kNone;
    }
    if (threadIdx.x < count) pos[threadIdx.x] = p.pos[i0 + threadIdx.x];
    __syncthreads();
    const int64_t c = ((int64_t)blockIdx.y * kGradThreads * N + threadIdx.x) * W;  // and every kGradThreads * W on
    if (p.list && blockIdx.y == 0 && threadIdx.x >= kGradThreads - 32) {
        const uint32_t v = key[count];
        if (v < p.vocab && key[count + 1] == v && !(key[1] == v && key[0] == v)) {
            // a run begins here that later pieces go on with: how many of them, to its end
            const int64_t i1 = i0 + count, end = i1 + lower_bound_warp(p.key + i1, p.tokens - i1, v + 1);
            if (threadIdx.x == kGradThreads - 1) {
                Join j;
                j.first = blockIdx.x;
                j.count = (uint32_t)ceil_div<int64_t>(end - i1, p.piece);
                j.id = v;
                p.joins[1 + atomicAdd(&p.joins[0].first, 1u)] = j;
            }
        }
    }
    const TI *grad = static_cast<const TI *>(p.grad) + c;
    float sum[N][W];
    int begin = 0;  // of the open run
    for (int k0 = 0; k0 < count; k0 += kFlight) {
        Raw<TI, W> x[kFlight][N];
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (k0 + f < count && key[k0 + f + 1] < p.vocab && c + n * kGradThreads * W < p.d)
                    x[f][n].load(grad + (int64_t)pos[k0 + f] * p.ldg + n * kGradThreads * W);
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int k = k0 + f;
            if (k >= count || key[k + 1] >= p.vocab) break;
            const uint32_t v = key[k + 1];
            if (k == 0 || key[k] != v) {
                begin = k;
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int j = 0; j < W; ++j) sum[n][j] = x[f][n][j];
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int j = 0; j < W; ++j) sum[n][j] = __fadd_rn(sum[n][j], x[f][n][j]);
            }
            if (k + 1 < count && key[k + 2] == v) continue;
            // the run ends here, or at the piece's end
            const bool from_before = begin == 0 && key[0] == v;
            const bool goes_on = k + 1 == count && key[k + 2] == v;
            float *part = p.part + (2 * (int64_t)blockIdx.x + (from_before ? 0 : 1)) * p.ldp;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int64_t at = c + n * kGradThreads * W;
                if (at >= p.d) break;
                if (from_before || goes_on)
                    store_w<float, W>(part + at, sum[n]);
                else
                    finish_row<TO, W>(p, v, at, sum[n]);
            }
        }
    }
}

// The runs that cross pieces, from the list: the sum of the piece in which one
// begins and those of the pieces after it.  The block's warps take consecutive
// shares of these pieces, which are then added in order; the list's own order
// decides nothing.
constexpr int kJoinWarps = 8, kJoinBlocks = 152, kJoinCols = 4;  // columns a lane takes; stored W at a time
template <class TO, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) grad_join_kernel(const GradParams p) {
    __shared__ float part[kJoinWarps][kJoinCols][32];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = ((int64_t)blockIdx.y * 32 + lane) * kJoinCols;
    const uint32_t runs = p.joins[0].first;
    for (uint32_t run = blockIdx.x; run < runs; run += gridDim.x) {
        const Join join = p.joins[1 + run];
        const int64_t first = join.first, count = join.count;
        const int64_t k0 = count * warp / kJoinWarps, k1 = count * (warp + 1) / kJoinWarps;
        float sum[kJoinCols] = {};
        if (c < p.d) {  // a partial sum's row has room for whole fours
            if (warp == 0) load_w<float, kJoinCols>(p.part + (2 * first + 1) * p.ldp + c, sum);
            const float *from = p.part + 2 * (first + 1) * p.ldp + c;
            constexpr int kFlight = 8;
            for (int64_t k = k0; k < k1; k += kFlight) {
                Raw<float, kJoinCols> x[kFlight];
#pragma unroll
                for (int f = 0; f < kFlight; ++f)
                    if (k + f < k1) x[f].load(from + 2 * (k + f) * p.ldp);
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    if (k + f >= k1) break;
#pragma unroll
                    for (int j = 0; j < kJoinCols; ++j) sum[j] = __fadd_rn(sum[j], x[f][j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kJoinCols; ++j) part[warp][j][lane] = sum[j];
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
                for (int j = 0; j < kJoinCols; ++j) sum[j] = __fadd_rn(sum[j], part[w][j][lane]);
#pragma unroll
            for (int j = 0; j < kJoinCols; j += W) {
                float some[W];
#pragma unroll
                for (int i = 0; i < W; ++i) some[i] = sum[j + i];
                if (c + j < p.d) finish_row<TO, W>(p, join.id, c + j, some);
            }
        }
        __syncthreads();
    }
}

struct GradPlan {
    int64_t key[2], pos[2], hist, joins, part, bytes;  // offsets into the workspace
    int64_t pieces, ldp;
    int tiles, passes, piece;
};

GradPlan plan_grad(int64_t tokens, int64_t vocab, int64_t d) {
    GradPlan g = {};
    auto take = [&](int64_t bytes) {
        const int64_t at = g.bytes;
        g.bytes += ceil_div<int64_t>(bytes, 256) * 256;
        return at;
    };
    g.tiles = (int)ceil_div<int64_t>(tokens, kSortTile);
    // few tokens: short pieces, so that there are enough blocks
    g.piece = tokens <= 4096 ? 8 : kPieceMost;
    g.pieces = ceil_div<int64_t>(tokens, g.piece);
    g.ldp = ceil_div<int64_t>(d, 8) * 8;
    g.passes = 1;
    while (vocab >> (kDigitBits * g.passes)) ++g.passes;  // the key `vocab` itself has to fit
    for (int k = 0; k < 2; ++k) {
        g.key[k] = take(tokens * 4);
        g.pos[k] = take(tokens * 4);
    }
    g.hist = take((int64_t)kDigits * g.tiles * 4 + kScanEach * 4);
    g.joins = take((1 + g.pieces) * (int64_t)sizeof(Join));
    g.part = take(2 * g.pieces * g.ldp * 4);
    return g;
}

__global__ void __launch_bounds__(kSortThreads) zero_kernel(const ZeroShare z) {
    pdl_enter();
    zero_share<kSortThreads>(z, blockIdx.x, gridDim.x);
}

template <class I, int R>
cudaError_t launch_sort_block(const SortParams &p, cudaStream_t s) {
    constexpr int smem = block_sort_smem(R);
    if (smem > 48 * 1024) {
        const cudaError_t e = opt_in_smem<sort_block_kernel<I, R>>(smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(sort_block_kernel<I, R>, 1 + zero_blocks(p.zero, kMaxZeroBlocks), kBlockSortThreads, smem, s, p);
}

// The sort, to the places plan_grad gives the last pass: one launch for up to
// kBlockSortMost tokens, else 3 launches a pass.  Each launch also sets its
// share of `zero` to zero.
constexpr int kBlockSortMost = 16 * kBlockSortThreads;
template <class I>
cudaError_t launch_sort(const GradPlan &g, char *ws, const void *ids, int64_t tokens, int64_t vocab, const ZeroShare &zero, cudaStream_t s) {
    SortParams p = {};
    p.ids = ids;
    p.hist = reinterpret_cast<uint32_t *>(ws + g.hist);
    p.joins = reinterpret_cast<uint32_t *>(ws + g.joins);
    p.tokens = tokens;
    p.vocab = vocab;
    p.tiles = g.tiles;
    p.passes = g.passes;
    auto places = [&](int pass) {
        const int from = (pass + 1) & 1, to = pass & 1;
        p.key_in = reinterpret_cast<uint32_t *>(ws + g.key[from]);
        p.pos_in = reinterpret_cast<uint32_t *>(ws + g.pos[from]);
        p.key_out = reinterpret_cast<uint32_t *>(ws + g.key[to]);
        p.pos_out = reinterpret_cast<uint32_t *>(ws + g.pos[to]);
        p.shift = pass * kDigitBits;
    };
    if (tokens <= kBlockSortMost) {
        places(g.passes - 1);
        p.zero = zero;
        if (tokens <= kBlockSortThreads) return launch_sort_block<I, 1>(p, s);
        if (tokens <= 4 * kBlockSortThreads) return launch_sort_block<I, 4>(p, s);
        return launch_sort_block<I, 16>(p, s);
    }
    const int launches = 3 * g.passes;
    int launch = 0;
    auto share = [&]() {  // the next launch's share of the zeros; the blocks it takes
        p.zero = zero;
        p.zero.row0 = zero.rows * launch / launches;
        p.zero.rows = zero.rows * (launch + 1) / launches - p.zero.row0;
        ++launch;
        return zero_blocks(p.zero, kMaxZeroBlocks);
    };
    for (int pass = 0; pass < g.passes; ++pass) {
        places(pass);
        int64_t extra = share();
        cudaError_t e = launch_pdl(pass == 0 ? sort_count_kernel<I, true> : sort_count_kernel<I, false>, g.tiles + extra, kSortThreads, 0, s, p);
        if (e != cudaSuccess) return e;
        extra = share();
        e = launch_pdl(sort_scan_kernel, 1 + extra, kScanThreads, 0, s, p);
        if (e != cudaSuccess) return e;
        extra = share();
        e = launch_pdl(pass == 0 ? sort_scatter_kernel<I, true> : sort_scatter_kernel<I, false>, g.tiles + extra, kSortThreads, 0, s, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <class K, class P>
cudaError_t launch_2d(K kern, int64_t gx, int64_t gy, int threads, cudaStream_t s, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)gx, (unsigned)gy);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RA_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// Columns that a launch takes: the second grid extent, 32 * kJoinCols or more of
// them a block, stays below 2^16.
constexpr int64_t kLaunchCols = (int64_t)1 << 22;
template <class TI, class TO, int W>
cudaError_t launch_sums(const GradParams &whole, cudaStream_t s) {
    for (int64_t c0 = 0; c0 < whole.d; c0 += kLaunchCols) {
        GradParams p = whole;
        p.grad = static_cast<const TI *>(whole.grad) + c0;
        p.out = static_cast<TO *>(whole.out) + c0;
        p.part = whole.part + c0;
        p.d = whole.d - c0 < kLaunchCols ? whole.d - c0 : kLaunchCols;
        p.list = c0 == 0;  // the runs are the same for all columns
        cudaError_t e = launch_2d(grad_pieces_kernel<TI, TO, W>, p.pieces, ceil_div<int64_t>(p.d * (int64_t)sizeof(TI), kGradThreads * kRowBytes), kGradThreads, s, p);
        if (e == cudaSuccess && p.pieces > 1)
            e = launch_2d(grad_join_kernel<TO, (W < kJoinCols ? W : kJoinCols)>, p.pieces - 1 < kJoinBlocks ? p.pieces - 1 : kJoinBlocks,
                          ceil_div<int64_t>(p.d, 32 * kJoinCols), kJoinWarps * 32, s, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <class TI, class TO>
cudaError_t launch_grad(const GradParams &p, int width, cudaStream_t s) {
    if constexpr (sizeof(TI) == 2)
        if (width == 8) return launch_sums<TI, TO, 8>(p, s);
    if (width == 4) return launch_sums<TI, TO, 4>(p, s);
    if (width == 2) return launch_sums<TI, TO, 2>(p, s);
    return launch_sums<TI, TO, 1>(p, s);
}

}  // namespace
}  // namespace op
}  // namespace ra

using namespace ra;
using namespace ra::op;

extern "C" {

ra_status ra_embedding_lookup(const void *table, int64_t ld_table, int dtype, int64_t vocab, int64_t d, const void *ids,
                              int id_bytes, int64_t tokens, float scale, void *out, int64_t ld_out, void *stream) {
    const int esz = esize(dtype);
    if (esz == 0 || (id_bytes != 4 && id_bytes != 8)) return RA_ERR_INVALID_ARG;
    const Mat t{table, vocab, d, ld_table, esz}, o{out, tokens, d, ld_out, esz}, i{ids, tokens, 1, 1, id_bytes};
    if (!mat_ok(t) || !mat_ok(o)) return RA_ERR_INVALID_ARG;
    if (o.empty()) return RA_OK;
    if (!mat_ok(i)) return RA_ERR_INVALID_ARG;
    if (mats_overlap(t, o) || mats_overlap(i, o)) return RA_ERR_OVERLAP;
    const LookupParams p{table, ids, out, ld_table, ld_out, tokens, vocab, d, scale};
    const int width = common_width(t, o, d, 16 / esz);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == RA_F32)
        return cuda_status(id_bytes == 4 ? launch_lookup<float, int32_t>(p, width, s) : launch_lookup<float, int64_t>(p, width, s));
    return cuda_status(id_bytes == 4 ? launch_lookup<uint16_t, int32_t>(p, width, s) : launch_lookup<uint16_t, int64_t>(p, width, s));
}

size_t ra_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t d) {
    if (tokens <= 0 || vocab < 0 || d <= 0 || tokens >= kMaxExtent || vocab >= kMaxExtent || d >= kMaxExtent) return 0;
    return (size_t)plan_grad(tokens, vocab, d).bytes;
}

ra_status ra_embedding_grad(const void *grad, int64_t ld_grad, int grad_dtype, const void *ids, int id_bytes, int64_t tokens,
                            float scale, int accumulate, void *out, int64_t ld_out, int out_dtype, int64_t vocab, int64_t d,
                            void *ws, size_t ws_bytes, void *stream) {
    const int gsz = esize(grad_dtype), osz = esize(out_dtype);
    if (gsz == 0 || osz == 0 || (id_bytes != 4 && id_bytes != 8)) return RA_ERR_INVALID_ARG;
    const Mat g{grad, tokens, d, ld_grad, gsz}, o{out, vocab, d, ld_out, osz}, i{ids, tokens, 1, 1, id_bytes};
    if (!mat_ok(g) || !mat_ok(o)) return RA_ERR_INVALID_ARG;
    if (o.empty()) return RA_OK;
    if (!mat_ok(i)) return RA_ERR_INVALID_ARG;
    const GradPlan plan = plan_grad(tokens, vocab, d);
    const Mat w{ws, 1, plan.bytes, plan.bytes, 1};
    if (tokens > 0) {
        if (ws == nullptr || reinterpret_cast<uintptr_t>(ws) % 16 != 0 || ws_bytes < (size_t)plan.bytes) return RA_ERR_INVALID_ARG;
        if (mats_overlap(w, g) || mats_overlap(w, o) || mats_overlap(w, i)) return RA_ERR_OVERLAP;
    }
    if (mats_overlap(g, o) || mats_overlap(i, o)) return RA_ERR_OVERLAP;
    if (tokens == 0 && accumulate) return RA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *base = static_cast<char *>(ws);
    const ZeroShare zero{static_cast<char *>(out), vocab > 1 ? o.pitch() : o.row_bytes(), o.row_bytes(), 0, accumulate ? 0 : vocab};
    if (tokens == 0) return cuda_status(launch_pdl(zero_kernel, zero_blocks(zero, kMaxZeroBlocks), kSortThreads, 0, s, zero));
    cudaError_t e = id_bytes == 4 ? launch_sort<int32_t>(plan, base, ids, tokens, vocab, zero, s)
                                  : launch_sort<int64_t>(plan, base, ids, tokens, vocab, zero, s);
    if (e != cudaSuccess) return cuda_status(e);
    const int sorted = (plan.passes + 1) & 1;
    const GradParams p{grad, out,
                       reinterpret_cast<const uint32_t *>(base + plan.key[sorted]),
                       reinterpret_cast<const uint32_t *>(base + plan.pos[sorted]),
                       reinterpret_cast<float *>(base + plan.part), reinterpret_cast<Join *>(base + plan.joins),
                       ld_grad, ld_out, plan.ldp, tokens, vocab, d, plan.pieces, plan.piece, scale, accumulate, 1};
    const int width = common_width(g, o, d, 16 / gsz);
    if (gsz == 4) return cuda_status(osz == 4 ? launch_grad<float, float>(p, width, s) : launch_grad<float, uint16_t>(p, width, s));
    return cuda_status(osz == 4 ? launch_grad<uint16_t, float>(p, width, s) : launch_grad<uint16_t, uint16_t>(p, width, s));
}

}  // extern "C"
