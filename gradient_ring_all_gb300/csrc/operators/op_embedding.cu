// op_embedding.cu -- rows of an embedding table and the table's gradient:
// ra_embedding_lookup and ra_embedding_grad.
#include "op_common.cuh"

namespace ra {
namespace op {
namespace {

// ---------------------------------------------------------------------------
// lookup: out[t] = scale * table[id_t], zeros for an id outside the table.
// A warp a token; each lane takes W neighbouring columns at a time, 4 of them
// in flight.

constexpr int kLookupThreads = 256;

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
        constexpr int kFlight = 4;
        for (int64_t c0 = lane * W; c0 < p.d; c0 += 32 * W * kFlight) {
            float x[kFlight][W];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const int64_t c = c0 + k * 32 * W;
                if (c < p.d && id >= 0) {
                    load_w<T, W>(src + c, x[k]);
                } else {
#pragma unroll
                    for (int j = 0; j < W; ++j) x[k][j] = 0.0f;
                }
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const int64_t c = c0 + k * 32 * W;
                if (c >= p.d) continue;
                if (id >= 0) {
#pragma unroll
                    for (int j = 0; j < W; ++j) x[k][j] = __fmul_rn(x[k][j], p.scale);
                }
                store_w<T, W>(dst + c, x[k]);
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
// 2. The sorted positions are cut into pieces of kPiece tokens.  A block sums
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

constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 4;                         // tokens a thread holds
constexpr int kSortTile = kSortThreads * kSortRounds;  // 1024
constexpr int kPiece = 32;

// A share of the table gradient's rows that a launch sets to zero.
struct ZeroShare {
    void *out;
    int64_t ld, d, row0, rows;  // ld and d in elements
    int esz, wide;              // wide: rows are whole numbers of 16-byte words on 16-byte boundaries
};
constexpr int kZeroBlockBytes = 1 << 15, kMaxZeroBlocks = 152 * 8;

// the work of block `at` of `blocks`
template <int THREADS>
__device__ __forceinline__ void zero_share(const ZeroShare &z, int64_t at, int64_t blocks) {
    if (z.wide) {
        const int64_t words = z.d * z.esz / 16, pitch = z.ld * z.esz / 16;
        uint4 *base = static_cast<uint4 *>(z.out) + z.row0 * pitch;
        if (words == pitch) {  // no gaps: one range
            const int64_t n = z.rows * words;
            for (int64_t i = at * THREADS + threadIdx.x; i < n; i += blocks * THREADS) base[i] = make_uint4(0, 0, 0, 0);
        } else {
            for (int64_t r = at; r < z.rows; r += blocks)
                for (int64_t i = threadIdx.x; i < words; i += THREADS) base[r * pitch + i] = make_uint4(0, 0, 0, 0);
        }
    } else {
        for (int64_t r = at; r < z.rows; r += blocks) {
            const int64_t row = (z.row0 + r) * z.ld;
            for (int64_t i = threadIdx.x; i < z.d; i += THREADS) {
                if (z.esz == 4)
                    static_cast<float *>(z.out)[row + i] = 0.0f;
                else
                    static_cast<uint16_t *>(z.out)[row + i] = 0;
            }
        }
    }
}

struct SortParams {
    ZeroShare zero;
    const void *ids;  // first pass
    const uint32_t *key_in, *pos_in;
    uint32_t *key_out, *pos_out;
    uint32_t *hist;  // [kDigits][tiles]
    int64_t tokens, vocab;
    int tiles, shift;  // blocks from `tiles` on set zeros
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

// exclusive prefix sums over `n` counts, in place, by one block
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(const SortParams p) {
    __shared__ uint32_t warp_sum[32];
    pdl_enter();
    if (blockIdx.x >= 1) {
        zero_share<kScanThreads>(p.zero, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    uint32_t *h = p.hist;
    const int64_t n = (int64_t)kDigits * p.tiles;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    uint32_t carry = 0;
    for (int64_t base = 0; base < n; base += kScanThreads) {
        const int64_t i = base + threadIdx.x;
        const uint32_t v = i < n ? h[i] : 0;
        uint32_t s = v;
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
        const uint32_t before = carry + (warp ? warp_sum[warp - 1] : 0);
        if (i < n) h[i] = before + s - v;
        carry += warp_sum[31];
        __syncthreads();
    }
}

// Each warp owns kSortRounds * 32 consecutive tokens and takes them 32 at a
// time: lanes with one digit find each other with a match, the digit's count
// in the warp's own counters gives the rank of the first of them.  The
// counters then become offsets by a prefix over the warps.
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
    uint32_t key[kSortRounds], pos[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t t = base + r * 32 + lane;
        const bool in = t < p.tokens;
        key[r] = in ? sort_key<I, FIRST>(p, t) : 0;
        pos[r] = in ? (FIRST ? (uint32_t)t : p.pos_in[t]) : 0;
        const uint32_t digit = in ? (key[r] >> p.shift) & (kDigits - 1) : kDigits;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        const uint32_t below = __popc(peers & ((1u << lane) - 1));
        uint32_t before = 0;
        if (in) before = count[warp][digit];
        __syncwarp();
        if (in && below == 0) count[warp][digit] = before + __popc(peers);
        __syncwarp();
        rank[r] = before + below;
    }
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

struct GradParams {
    const void *grad;
    void *out;
    const uint32_t *key, *pos;
    float *part;  // [2 * pieces][d rounded up to 8]: a piece's first and last run
    int64_t ldg, ldo, ldp, tokens, vocab, d;
    int64_t pieces;
    float scale;
    int accumulate;
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
    __shared__ uint32_t key[kPiece + 2], pos[kPiece];
    pdl_enter();
    const int64_t c = ((int64_t)blockIdx.y * kGradThreads + threadIdx.x) * W;
    const int64_t i0 = (int64_t)blockIdx.x * kPiece;
    const int count = (int)(p.tokens - i0 < kPiece ? p.tokens - i0 : kPiece);
    constexpr uint32_t kNone = 0xffffffffu;
    if (threadIdx.x < kPiece + 2) {
        const int64_t i = i0 - 1 + threadIdx.x;
        key[threadIdx.x] = i >= 0 && i < p.tokens ? p.key[i] : kNone;
    }
    if (threadIdx.x < count) pos[threadIdx.x] = p.pos[i0 + threadIdx.x];
    __syncthreads();
    if (c >= p.d) return;
    const TI *grad = static_cast<const TI *>(p.grad) + c;
    float sum[W];
    int begin = 0;  // of the open run
    constexpr int kFlight = W * sizeof(TI) >= 16 ? 8 : 16;
    for (int k0 = 0; k0 < count; k0 += kFlight) {
        Raw<TI, W> x[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
            if (k0 + f < count && key[k0 + f + 1] < p.vocab) x[f].load(grad + (int64_t)pos[k0 + f] * p.ldg);
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int k = k0 + f;
            if (k >= count || key[k + 1] >= p.vocab) break;
            const uint32_t v = key[k + 1];
            if (k == 0 || key[k] != v) {
                begin = k;
#pragma unroll
                for (int j = 0; j < W; ++j) sum[j] = x[f][j];
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) sum[j] = __fadd_rn(sum[j], x[f][j]);
            }
            if (k + 1 < count && key[k + 2] == v) continue;
            // the run ends here, or at the piece's end
            const bool from_before = begin == 0 && key[0] == v;
            const bool goes_on = k + 1 == count && key[k + 2] == v;
            if (!from_before && !goes_on) {
                finish_row<TO, W>(p, v, c, sum);
            } else {
                float *to = p.part + (2 * (int64_t)blockIdx.x + (from_before ? 0 : 1)) * p.ldp + c;
                store_w<float, W>(to, sum);
            }
        }
    }
}

// A block for each piece in which a run begins that later pieces go on with:
// the piece's own partial sum and those of the pieces after it.  The block's
// warps take consecutive shares of these pieces, which are then added in order.
constexpr int kJoinWarps = 8;
template <class TO, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) grad_join_kernel(const GradParams p) {
    __shared__ float part[kJoinWarps][32 * W];
    pdl_enter();
    const int64_t i1 = ((int64_t)blockIdx.x + 1) * kPiece;  // the first token of the next piece
    const uint32_t v = p.key[i1];
    if (v >= p.vocab || p.key[i1 - 1] != v) return;
    if (i1 > kPiece && p.key[i1 - kPiece] == v && p.key[i1 - kPiece - 1] == v) return;  // begins earlier
    // the run's end, and so the pieces 0 .. count-1 that begin with it after this one
    const int64_t end = i1 + lower_bound_warp(p.key + i1, p.tokens - i1, v + 1);
    const int64_t count = ceil_div<int64_t>(end - i1, kPiece);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = ((int64_t)blockIdx.y * 32 + lane) * W;
    const int64_t k0 = count * warp / kJoinWarps, k1 = count * (warp + 1) / kJoinWarps;
    float sum[W];
#pragma unroll
    for (int j = 0; j < W; ++j) sum[j] = 0.0f;
    if (c < p.d) {
        if (warp == 0) load_w<float, W>(p.part + (2 * (int64_t)blockIdx.x + 1) * p.ldp + c, sum);
        const float *from = p.part + 2 * ((int64_t)blockIdx.x + 1) * p.ldp + c;
        constexpr int kFlight = W > 4 ? 4 : 8;
        for (int64_t k = k0; k < k1; k += kFlight) {
            Raw<float, W> x[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f)
                if (k + f < k1) x[f].load(from + 2 * (k + f) * p.ldp);
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                if (k + f >= k1) break;
#pragma unroll
                for (int j = 0; j < W; ++j) sum[j] = __fadd_rn(sum[j], x[f][j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j) part[warp][j * 32 + lane] = sum[j];
    __syncthreads();
    if (warp != 0 || c >= p.d) return;
    for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int j = 0; j < W; ++j) sum[j] = __fadd_rn(sum[j], part[w][j * 32 + lane]);
    finish_row<TO, W>(p, v, c, sum);
}

struct GradPlan {
    int64_t key[2], pos[2], hist, part, bytes;  // offsets into the workspace
    int64_t pieces, ldp;
    int tiles, passes;
};

GradPlan plan_grad(int64_t tokens, int64_t vocab, int64_t d) {
    GradPlan g = {};
    auto take = [&](int64_t bytes) {
        const int64_t at = g.bytes;
        g.bytes += ceil_div<int64_t>(bytes, 256) * 256;
        return at;
    };
    g.tiles = (int)ceil_div<int64_t>(tokens, kSortTile);
    g.pieces = ceil_div<int64_t>(tokens, kPiece);
    g.ldp = ceil_div<int64_t>(d, 8) * 8;
    g.passes = 1;
    while (vocab >> (kDigitBits * g.passes)) ++g.passes;  // the key `vocab` itself has to fit
    for (int k = 0; k < 2; ++k) {
        g.key[k] = take(tokens * 4);
        g.pos[k] = take(tokens * 4);
    }
    g.hist = take((int64_t)kDigits * g.tiles * 4);
    g.part = take(2 * g.pieces * g.ldp * 4);
    return g;
}

int64_t zero_blocks(const ZeroShare &z) {
    const int64_t blocks = ceil_div<int64_t>(z.rows * z.d * z.esz, kZeroBlockBytes);
    return blocks < kMaxZeroBlocks ? blocks : kMaxZeroBlocks;
}

__global__ void __launch_bounds__(kSortThreads) zero_kernel(const ZeroShare z) {
    pdl_enter();
    zero_share<kSortThreads>(z, blockIdx.x, gridDim.x);
}

// The sorting launches (3 a pass); each also sets its share of `out` to zero,
// where `zero.rows` asks for it.
template <class I>
cudaError_t launch_sort(const GradPlan &g, char *ws, const void *ids, int64_t tokens, int64_t vocab, const ZeroShare &zero, cudaStream_t s) {
    const int launches = 3 * g.passes;
    int launch = 0;
    SortParams p = {};
    auto share = [&]() -> int64_t {  // sets p.zero; the blocks it takes
        p.zero = zero;
        p.zero.row0 = zero.rows * launch / launches;
        p.zero.rows = zero.rows * (launch + 1) / launches - p.zero.row0;
        ++launch;
        return zero_blocks(p.zero);
    };
    for (int pass = 0; pass < g.passes; ++pass) {
        const int from = (pass + 1) & 1, to = pass & 1;
        p.ids = ids;
        p.key_in = reinterpret_cast<uint32_t *>(ws + g.key[from]);
        p.pos_in = reinterpret_cast<uint32_t *>(ws + g.pos[from]);
        p.key_out = reinterpret_cast<uint32_t *>(ws + g.key[to]);
        p.pos_out = reinterpret_cast<uint32_t *>(ws + g.pos[to]);
        p.hist = reinterpret_cast<uint32_t *>(ws + g.hist);
        p.tokens = tokens;
        p.vocab = vocab;
        p.tiles = g.tiles;
        p.shift = pass * kDigitBits;
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

template <class TI, class TO, int W>
cudaError_t launch_sums(const GradParams &p, cudaStream_t s) {
    cudaError_t e = launch_2d(grad_pieces_kernel<TI, TO, W>, p.pieces, ceil_div<int64_t>(p.d, kGradThreads * W), kGradThreads, s, p);
    if (e != cudaSuccess || p.pieces < 2) return e;
    return launch_2d(grad_join_kernel<TO, W>, p.pieces - 1, ceil_div<int64_t>(p.d, 32 * W), kJoinWarps * 32, s, p);
}

template <class TI, class TO>
cudaError_t launch_grad(const GradParams &p, int width, cudaStream_t s) {
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
    if (plan.pieces > kMaxGrid || ceil_div<int64_t>(d, 32) > 65535) return RA_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *base = static_cast<char *>(ws);
    const ZeroShare zero{out, ld_out, d, 0, accumulate ? 0 : vocab, osz, o.aligned(16) && o.row_bytes() % 16 == 0};
    if (tokens == 0) return cuda_status(launch_pdl(zero_kernel, zero_blocks(zero), kSortThreads, 0, s, zero));
    cudaError_t e = id_bytes == 4 ? launch_sort<int32_t>(plan, base, ids, tokens, vocab, zero, s)
                                  : launch_sort<int64_t>(plan, base, ids, tokens, vocab, zero, s);
    if (e != cudaSuccess) return cuda_status(e);
    const int sorted = (plan.passes + 1) & 1;
    const GradParams p{grad, out,
                       reinterpret_cast<const uint32_t *>(base + plan.key[sorted]),
                       reinterpret_cast<const uint32_t *>(base + plan.pos[sorted]),
                       reinterpret_cast<float *>(base + plan.part),
                       ld_grad, ld_out, plan.ldp, tokens, vocab, d, plan.pieces, scale, accumulate};
    const int width = common_width(g, o, d, 16 / gsz);
    if (gsz == 4) return cuda_status(osz == 4 ? launch_grad<float, float>(p, width, s) : launch_grad<float, uint16_t>(p, width, s));
    return cuda_status(osz == 4 ? launch_grad<uint16_t, float>(p, width, s) : launch_grad<uint16_t, uint16_t>(p, width, s));
}

}  // extern "C"
