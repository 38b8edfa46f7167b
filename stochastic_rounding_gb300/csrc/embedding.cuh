// embedding.cuh -- rows of a table picked by token, and the table's gradient.
// Included into asr.cu (inside its anonymous namespace), after checkpoint.cuh.
//
//   y_t = s T[id_t];   dT_v = s sum over t with id_t = v of dy_t, in the tokens' order
//
// The gradient is the whole table's, and most of its bytes are zeros.  Tokens are
// sorted by id, stably, so that every row's tokens lie together and in order; the
// sorted list is cut into chunks of one length, a block each, whatever the ids --
// a token that makes up half of a batch is as even a share of the work as any.  A
// block adds its tokens' rows up in registers: a row that begins and ends within
// the chunk is written at once, one that reaches over an end leaves a binary32 sum
// in the workspace, and a last kernel adds those up, in order.  Rows without
// tokens are zeroed by the blocks that do not sort.
//
// The sort is by digits of up to nine bits, from the lowest, each by counts and
// ranks: a warp ranks 32 keys at a time (lanes of one digit find one another), the
// warps' counts are added up by digit.  Up to 8,192 tokens are one block's, in
// shared memory; more are cut into tiles of 8,192, with a launch each for their
// counts, the tiles' places, and the moves.

namespace embed {

using kept::live_of;

constexpr int kSortThreads = 1024;
constexpr int kTile = 8192;                     // keys a block sorts, eight a thread
constexpr int kRounds = kTile / kSortThreads;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kThreads = 256;
constexpr int kZeroRows = 64;                   // of the table, a block at a time

struct Ids {
    const void *p;
    uint64_t n;
    uint32_t wide;                              // 64-bit
    uint32_t vocab;
    uint32_t padding;                           // vocab or more: none
};

// The row of token t, or vocab where it has none.
__device__ __forceinline__ uint32_t key_of(const Ids &I, uint64_t t)
{
    uint32_t id;
    if (I.wide) {
        const uint64_t v = static_cast<const uint64_t *>(I.p)[t];
        id = v < I.vocab ? static_cast<uint32_t>(v) : I.vocab;
    } else {
        id = static_cast<const uint32_t *>(I.p)[t];
        id = id < I.vocab ? id : I.vocab;
    }
    return id == I.padding ? I.vocab : id;
}

// ---- lookup

struct LookupParams {
    Ids ids;
    kept::Matrix table;
    kept::Out y;
    uint64_t dim;
    float scale;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const __grid_constant__ LookupParams P, uint32_t spans)
{
    const uint32_t lane = threadIdx.x & 31;
    for (kept::Walk k(P.ids.n, spans); k.more(); k.next()) {
        const uint32_t id = key_of(P.ids, k.row);
        kept::Raw<DT> raw[kept::kUnits];
#pragma unroll
        for (int u = 0; u < kept::kUnits; ++u) {
            const uint64_t col = k.span * static_cast<uint64_t>(kept::kSpan) + u * 256 + lane * 8;
            raw[u] = kept::fetch<DT>(P.table.p, id * P.table.ld + col, id < P.ids.vocab ? live_of(P.dim, col) : 0, P.table.vec);
        }
#pragma unroll
        for (int u = 0; u < kept::kUnits; ++u) {
            const uint64_t col = k.span * static_cast<uint64_t>(kept::kSpan) + u * 256 + lane * 8;
            float v[8];
            kept::values(raw[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = id < P.ids.vocab ? __fmul_rn(v[i], P.scale) : __uint_as_float(0x7FC00000u);
            kept::store8<DT>(P.y.p, k.row * P.y.ld + col, live_of(P.dim, col), P.y.vec, v);
        }
    }
}

// ---- sort

// Ranks of a block's keys by one digit.  Warp w holds keys w * 256 .. + 255 of the
// tile, 32 a round.  Afterwards `counts` holds, for each warp and digit, how many
// keys of the digit the warps before have; totals[d] is the tile's.
__device__ __forceinline__ void rank_digits(const uint32_t key[kRounds], uint32_t live, uint32_t shift,
                                            uint16_t (*counts)[kBins], uint32_t *totals, uint16_t rank[kRounds])
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (uint32_t i = threadIdx.x; i < 32 * kBins / 2; i += kSortThreads) reinterpret_cast<uint32_t *>(counts)[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const bool in = (live >> r) & 1;
        const uint32_t d = in ? (key[r] >> shift) & (kBins - 1) : kBins;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
        const uint32_t before = peers & ((1u << lane) - 1);
        if (in) rank[r] = static_cast<uint16_t>(counts[warp][d] + __popc(before));
        __syncwarp();
        if (in && before == 0) counts[warp][d] = static_cast<uint16_t>(counts[warp][d] + __popc(peers));
        __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
        uint32_t sum = 0;
#pragma unroll 8
        for (int w = 0; w < 32; ++w) {
            const uint32_t c = counts[w][threadIdx.x];
            counts[w][threadIdx.x] = static_cast<uint16_t>(sum);
            sum += c;
        }
        totals[threadIdx.x] = sum;
    }
    __syncthreads();
}

// totals[d] becomes the sum of those before it.
__device__ __forceinline__ void scan_bins(uint32_t *totals, uint32_t *part)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t own = 0, v = 0;
    if (threadIdx.x < kBins) {
        own = v = totals[threadIdx.x];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= static_cast<uint32_t>(d)) v += o;
        }
        if (lane == 31) part[warp] = v;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
        for (uint32_t w = 0; w < warp; ++w) v += part[w];
        totals[threadIdx.x] = v - own;
    }
    __syncthreads();
}

struct SortShared {
    uint32_t key[kTile];
    uint16_t order[kTile];
    uint16_t counts[32][kBins];
    uint32_t totals[kBins];
    uint32_t part[32];
};

struct ZeroParams {
    void *p;                                    // vocab x dim
    uint64_t dim;
    uint32_t dtype, vec;
};

struct SortParams {
    Ids ids;
    uint32_t *key, *order;
    uint32_t bits;                              // of a key, vocab among them
    ZeroParams zero;
};

// Zeroes rows v0 .. v0 + kZeroRows - 1 of the table but those set in `taken`.
__device__ __forceinline__ void zero_rows(const ZeroParams &Z, uint32_t vocab, uint64_t v0, const uint32_t *taken)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint64_t size = Z.dtype == ASR_BF16 ? 2 : 4, bytes = Z.dim * size;
    for (uint32_t r = warp; r < kZeroRows && v0 + r < vocab; r += warps) {
        if ((taken[r >> 5] >> (r & 31)) & 1) continue;
        char *p = static_cast<char *>(Z.p) + (v0 + r) * bytes;
        if (Z.vec) {
            for (uint64_t i = lane * 16ull; i < bytes; i += 512) *reinterpret_cast<uint4 *>(p + i) = make_uint4(0, 0, 0, 0);
        } else if (Z.dtype == ASR_BF16) {
            for (uint64_t i = lane; i < Z.dim; i += 32) reinterpret_cast<uint16_t *>(p)[i] = 0;
        } else {
            for (uint64_t i = lane; i < Z.dim; i += 32) reinterpret_cast<float *>(p)[i] = 0.0f;
        }
    }
}

// Up to kTile tokens: block 0 sorts, the others zero the rows that no token has.
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ SortParams P)
{
    extern __shared__ __align__(16) unsigned char raw[];
    if (blockIdx.x > 0) {
        uint32_t *taken = reinterpret_cast<uint32_t *>(raw);
        const uint64_t v0 = (blockIdx.x - 1) * static_cast<uint64_t>(kZeroRows);
        if (threadIdx.x < kZeroRows / 32) taken[threadIdx.x] = 0;
        __syncthreads();
        for (uint64_t t = threadIdx.x; t < P.ids.n; t += kSortThreads) {
            const uint64_t d = key_of(P.ids, t) - v0;
            if (d < kZeroRows) atomicOr(taken + (d >> 5), 1u << (d & 31));
        }
        __syncthreads();
        zero_rows(P.zero, P.ids.vocab, v0, taken);
        return;
    }
    SortShared &S = *reinterpret_cast<SortShared *>(raw);
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = static_cast<uint32_t>(P.ids.n);
    uint32_t key[kRounds], live = 0;
    uint16_t from[kRounds], rank[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t t = warp * 256 + r * 32 + lane;
        key[r] = 0;
        from[r] = static_cast<uint16_t>(t);
        if (t < n) live |= 1u << r, key[r] = key_of(P.ids, t);
    }
    for (uint32_t shift = 0; shift < P.bits; shift += kDigitBits) {
        rank_digits(key, live, shift, S.counts, S.totals, rank);
        scan_bins(S.totals, S.part);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if ((live >> r) & 1) {
                const uint32_t d = (key[r] >> shift) & (kBins - 1), to = S.totals[d] + S.counts[warp][d] + rank[r];
                S.key[to] = key[r];
                S.order[to] = from[r];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if ((live >> r) & 1) {
                key[r] = S.key[warp * 256 + r * 32 + lane];
                from[r] = S.order[warp * 256 + r * 32 + lane];
            }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if ((live >> r) & 1) {
            P.key[warp * 256 + r * 32 + lane] = key[r];
            P.order[warp * 256 + r * 32 + lane] = from[r];
        }
}

// More tokens: one digit's counts of each tile, their places, and the moves.
struct TileParams {
    Ids ids;                                    // first digit: where the keys come from
    const uint32_t *key, *order;                // later ones
    uint32_t *key_out, *order_out;
    uint32_t *counts;                           // [bin][tile]
    uint32_t tiles, shift, first;
};

__global__ void __launch_bounds__(kSortThreads) tile_count_kernel(const __grid_constant__ TileParams P)
{
    __shared__ uint32_t bins[kBins];
    for (uint32_t i = threadIdx.x; i < kBins; i += kSortThreads) bins[i] = 0;
    __syncthreads();
    for (int r = 0; r < kRounds; ++r) {
        const uint64_t t = blockIdx.x * static_cast<uint64_t>(kTile) + r * kSortThreads + threadIdx.x;
        if (t < P.ids.n) atomicAdd(bins + (((P.first ? key_of(P.ids, t) : P.key[t]) >> P.shift) & (kBins - 1)), 1u);
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kBins; i += kSortThreads) P.counts[i * static_cast<uint64_t>(P.tiles) + blockIdx.x] = bins[i];
}

// Every count becomes the sum of those before it: one block.
__global__ void __launch_bounds__(kSortThreads) tile_scan_kernel(const __grid_constant__ TileParams P)
{
    __shared__ uint32_t part[32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t n = static_cast<uint64_t>(kBins) * P.tiles;
    uint32_t carry = 0;
    for (uint64_t at = 0; at < n; at += kSortThreads * 4) {
        const uint64_t i = at + threadIdx.x * 4;            // n is a multiple of 4
        uint4 c = make_uint4(0, 0, 0, 0);
        if (i < n) c = *reinterpret_cast<const uint4 *>(P.counts + i);
        const uint32_t own = c.x + c.y + c.z + c.w;
        uint32_t v = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= static_cast<uint32_t>(d)) v += o;
        }
        __syncthreads();
        if (lane == 31) part[warp] = v;
        __syncthreads();
        uint32_t before = 0, total = 0;
        for (uint32_t w = 0; w < 32; ++w) {
            before += w < warp ? part[w] : 0;
            total += part[w];
        }
        v += carry + before - own;
        carry += total;
        if (i < n) *reinterpret_cast<uint4 *>(P.counts + i) = make_uint4(v, v + c.x, v + c.x + c.y, v + c.x + c.y + c.z);
    }
}

struct TileShared {
    uint16_t counts[32][kBins];
    uint32_t totals[kBins];
};

__global__ void __launch_bounds__(kSortThreads) tile_move_kernel(const __grid_constant__ TileParams P)
{
    __shared__ TileShared S;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t t0 = blockIdx.x * static_cast<uint64_t>(kTile) + warp * 256 + lane;
    uint32_t key[kRounds], from[kRounds], live = 0;
    uint16_t rank[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint64_t t = t0 + r * 32;
        key[r] = from[r] = 0;
        if (t < P.ids.n) {
            live |= 1u << r;
            key[r] = P.first ? key_of(P.ids, t) : P.key[t];
            from[r] = P.first ? static_cast<uint32_t>(t) : P.order[t];
        }
    }
    rank_digits(key, live, P.shift, S.counts, S.totals, rank);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if ((live >> r) & 1) {
            const uint32_t d = (key[r] >> P.shift) & (kBins - 1);
            const uint64_t to = static_cast<uint64_t>(P.counts[d * static_cast<uint64_t>(P.tiles) + blockIdx.x]) +
                                S.counts[warp][d] + rank[r];
            P.key_out[to] = key[r];
            P.order_out[to] = from[r];
        }
}

// The first place in the sorted keys that holds `key` or more.
__device__ __forceinline__ uint64_t lower_bound(const uint32_t *keys, uint64_t n, uint64_t key)
{
    uint64_t lo = 0, hi = n;
    while (lo < hi) {
        const uint64_t mid = (lo + hi) / 2;
        if (keys[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

struct SparseZeroParams {
    const uint32_t *key;
    uint64_t n;
    uint32_t vocab;
    ZeroParams zero;
};

// Zeroes the rows without tokens once the keys are sorted.
__global__ void __launch_bounds__(kThreads) zero_kernel(const __grid_constant__ SparseZeroParams P)
{
    __shared__ uint32_t taken[kZeroRows / 32];
    const uint64_t v0 = blockIdx.x * static_cast<uint64_t>(kZeroRows);
    if (threadIdx.x < kZeroRows / 32) taken[threadIdx.x] = 0;
    __syncthreads();
    const uint64_t lo = lower_bound(P.key, P.n, v0), hi = lower_bound(P.key, P.n, v0 + kZeroRows);
    for (uint64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        const uint32_t d = P.key[i] - static_cast<uint32_t>(v0);
        atomicOr(taken + (d >> 5), 1u << (d & 31));
    }
    __syncthreads();
    zero_rows(P.zero, P.vocab, v0, taken);
}

// ---- sums

struct SumParams {
    const uint32_t *key, *order;
    uint64_t n;                                 // tokens
    uint32_t chunk, chunks, vocab;
    uint64_t dim;
    kept::Matrix dy;
    kept::Out out;
    float *head, *tail;                         // [chunk][dim]: sums of a row that began before, that goes on after
    float scale;
};

// What is known of a chunk's ends.
struct Ends {
    uint64_t begin, end;
    bool open, on;                              // its first key began before; its last goes on after
};

__device__ __forceinline__ Ends ends_of(const SumParams &P, uint64_t c)
{
    Ends E;
    E.begin = c * P.chunk;
    E.end = E.begin + P.chunk < P.n ? E.begin + P.chunk : P.n;
    E.open = c > 0 && P.key[E.begin - 1] == P.key[E.begin];
    E.on = E.end < P.n && P.key[E.end] == P.key[E.end - 1];
    return E;
}

template <int OT>
__device__ __forceinline__ void store_row(const SumParams &P, uint32_t row, uint64_t col, int live, float v[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], P.scale);
    kept::store8<OT>(P.out.p, row * P.out.ld + col, live, P.out.vec, v);
}

__device__ __forceinline__ void store_sum(float *p, uint64_t dim, uint64_t c, uint64_t col, int live, const float v[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < live) p[c * dim + col + i] = v[i];
}

// A block a chunk and 8 columns a thread.
constexpr int kAhead = 4;                       // rows loaded before they are added up

template <int DT, int OT>
__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ SumParams P)
{
    const uint64_t c = blockIdx.x, col = (blockIdx.y * static_cast<uint64_t>(blockDim.x) + threadIdx.x) * 8;
    const int live = live_of(P.dim, col);
    const Ends E = ends_of(P, c);
    float acc[8] = {};
    bool first = true;                          // still in the chunk's first row
    for (uint64_t i0 = E.begin; i0 < E.end; i0 += kAhead) {
        uint32_t key[kAhead + 1];
        float v[kAhead][8];
#pragma unroll
        for (int a = 0; a <= kAhead; ++a) key[a] = i0 + a < P.n ? P.key[i0 + a] : P.vocab;
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const bool in = i0 + a < E.end && key[a] < P.vocab;
            muon::load8(P.dy.p, DT, in ? P.order[i0 + a] * P.dy.ld + col : 0, in ? live : 0, P.dy.vec, v[a]);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (i0 + a >= E.end || key[a] >= P.vocab) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], v[a][i]);
            const bool last = i0 + a + 1 == E.end;
            if (!last && key[a + 1] == key[a]) continue;
            if (first && E.open) store_sum(P.head, P.dim, c, col, live, acc);
            else if (last && E.on) store_sum(P.tail, P.dim, c, col, live, acc);
            else store_row<OT>(P, key[a], col, live, acc);
            first = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        }
    }
}

// Rows that reach over chunks' ends, by the chunk where they begin: the sum there
// and those of the chunks that go on with it, in order.
template <int OT>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ SumParams P)
{
    const uint64_t c = blockIdx.x, col = (blockIdx.y * static_cast<uint64_t>(blockDim.x) + threadIdx.x) * 8;
    const int live = live_of(P.dim, col);
    const Ends E = ends_of(P, c);
    const uint32_t key = P.key[E.end - 1];
    if (!E.on || key >= P.vocab || (E.open && P.key[E.begin] == key)) return;
    // how many chunks go on with it: they follow one another
    uint64_t last = c + 1;
    for (int more = static_cast<int>(blockDim.x); more == static_cast<int>(blockDim.x); last += more) {
        const uint64_t d = last + threadIdx.x;
        more = __syncthreads_count(d < P.chunks && P.key[d * P.chunk] == key);
    }
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = i < live ? P.tail[c * P.dim + col + i] : 0.0f;
#pragma unroll 4
    for (uint64_t d = c + 1; d < last; ++d)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) acc[i] = __fadd_rn(acc[i], P.head[d * P.dim + col + i]);
    store_row<OT>(P, key, col, live, acc);
}

// ------------------------------------------------------------------ host

constexpr uint64_t kMaxTokens = 1ull << 28, kMaxVocab = 1ull << 28;

asr_status ids_ok(const void *ids, int32_t index, uint64_t tokens, uint64_t vocab, uint64_t dim)
{
    if (tokens > kMaxTokens || vocab > kMaxVocab || dim > kept::kMaxCols) return ASR_ERR_INVALID_VALUE;
    if (tokens && (!ids || (reinterpret_cast<uintptr_t>(ids) & (index == ASR_I64 ? 7u : 3u)))) return ASR_ERR_INVALID_VALUE;
    return ASR_OK;
}

Ids ids_of(const void *ids, int32_t index, uint64_t tokens, uint64_t vocab, int64_t padding)
{
    return Ids{ids, tokens, index == ASR_I64 ? 1u : 0u, static_cast<uint32_t>(vocab),
               padding >= 0 && static_cast<uint64_t>(padding) < vocab ? static_cast<uint32_t>(padding) : 0xFFFFFFFFu};
}

asr_status setup()
{
    static std::atomic<uint64_t> ready{0}, opted{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && !(opted.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortShared));
        if (e == cudaSuccess) opted.fetch_or(bit, std::memory_order_release);
    }
    if (e != cudaSuccess) return cuda_fail(e);
    return kept::load_once(ready, lookup_kernel<ASR_F32>, lookup_kernel<ASR_BF16>, sort_kernel, tile_count_kernel,
                           tile_scan_kernel, tile_move_kernel, zero_kernel, sum_kernel<ASR_F32, ASR_F32>,
                           sum_kernel<ASR_F32, ASR_BF16>, sum_kernel<ASR_BF16, ASR_F32>, sum_kernel<ASR_BF16, ASR_BF16>,
                           join_kernel<ASR_F32>, join_kernel<ASR_BF16>);
}

asr_status lookup(const void *ids, int32_t index, uint64_t tokens, const void *table, uint64_t table_ld, uint64_t vocab,
                  uint64_t dim, double scale, void *y, uint64_t y_ld, int32_t dtype, cudaStream_t stream)
{
    if (!kept::dtype_ok(dtype) || (index != ASR_I32 && index != ASR_I64)) return ASR_ERR_UNSUPPORTED_DTYPE;
    asr_status st = ids_ok(ids, index, tokens, vocab, dim);
    if (st == ASR_OK && !std::isfinite(scale)) st = ASR_ERR_INVALID_VALUE;
    if (st != ASR_OK || tokens == 0 || dim == 0) return st;
    if ((vocab && !kept::matrix_ok(table, dtype, table_ld, dim)) || !kept::matrix_ok(y, dtype, y_ld, dim))
        return ASR_ERR_INVALID_VALUE;
    st = setup();
    if (st != ASR_OK) return st;
    LookupParams P;
    P.ids = ids_of(ids, index, tokens, vocab, -1);
    P.table = kept::matrix(table, table_ld);
    P.y = kept::out(y, y_ld);
    P.dim = dim;
    P.scale = static_cast<float>(scale);
    auto kernel = dtype == ASR_BF16 ? lookup_kernel<ASR_BF16> : lookup_kernel<ASR_F32>;
    return kept::walk(ASR_KERNEL_EMBEDDING, kernel, P, tokens, dim, kept::kSpan, stream);
}

// Chunks of eight tokens, longer where there would be more than 4,096 of them: what
// reaches over their ends takes 2 dim sums of workspace each.
uint32_t chunk_of(uint64_t tokens)
{
    const uint64_t c = (tokens + 4095) / 4096;
    return static_cast<uint32_t>(c < 8 ? 8 : (c + kAhead - 1) / kAhead * kAhead);
}

struct Layout {
    uint64_t key[2], order[2], counts, head, tail, bytes;
    uint32_t tiles;
};

Layout layout(uint64_t tokens, uint64_t dim)
{
    Layout L;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t was = at;
        at += muon::up(bytes, 256);
        return was;
    };
    L.tiles = static_cast<uint32_t>((tokens + kTile - 1) / kTile);
    const uint64_t chunks = (tokens + chunk_of(tokens) - 1) / chunk_of(tokens);
    for (int i = 0; i < 2; ++i) {
        const bool used = i == 0 || L.tiles > 1;
        L.key[i] = take(used ? tokens * 4 : 0);
        L.order[i] = take(used ? tokens * 4 : 0);
    }
    L.counts = take(L.tiles > 1 ? static_cast<uint64_t>(kBins) * L.tiles * 4 : 0);
    L.head = take(chunks * dim * 4);
    L.tail = take(chunks * dim * 4);
    L.bytes = at;
    return L;
}

template <int DT>
void (*sums_of(bool bf))(const SumParams)
{
    return bf ? sum_kernel<DT, ASR_BF16> : sum_kernel<DT, ASR_F32>;
}

asr_status grads(const void *ids, int32_t index, uint64_t tokens, const void *dy, uint64_t dy_ld, int32_t dy_dtype,
                 uint64_t vocab, uint64_t dim, double scale, int64_t padding, void *dtable, int32_t dtable_dtype, void *ws,
                 uint64_t ws_bytes, cudaStream_t stream)
{
    if (!kept::dtype_ok(dy_dtype) || !kept::dtype_ok(dtable_dtype) || (index != ASR_I32 && index != ASR_I64))
        return ASR_ERR_UNSUPPORTED_DTYPE;
    asr_status st = ids_ok(ids, index, tokens, vocab, dim);
    if (st == ASR_OK && !std::isfinite(scale)) st = ASR_ERR_INVALID_VALUE;
    if (st != ASR_OK || vocab == 0 || dim == 0) return st;
    if (!dtable || !muon::element_aligned(dtable, dtable_dtype) || (tokens && !kept::matrix_ok(dy, dy_dtype, dy_ld, dim)))
        return ASR_ERR_INVALID_VALUE;
    const Layout L = layout(tokens, dim);
    if (tokens && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < L.bytes)) return ASR_ERR_INVALID_VALUE;
    st = setup();
    if (st != ASR_OK) return st;
    char *w = static_cast<char *>(ws);
    auto words = [&](uint64_t at) { return reinterpret_cast<uint32_t *>(w + at); };
    const Ids I = ids_of(ids, index, tokens, vocab, padding);
    const ZeroParams Z{dtable, dim, static_cast<uint32_t>(dtable_dtype),
                       aligned16(dtable) && dim % (dtable_dtype == ASR_BF16 ? 8 : 4) == 0 ? 1u : 0u};
    uint32_t bits = 1;
    while ((vocab >> bits) != 0) ++bits;
    const unsigned zero_blocks = static_cast<unsigned>((vocab + kZeroRows - 1) / kZeroRows);
    int now = 0;
    if (L.tiles <= 1) {
        SortParams P;
        P.ids = I;
        P.key = words(L.key[0]);
        P.order = words(L.order[0]);
        P.bits = bits;
        P.zero = Z;
        sort_kernel<<<zero_blocks + 1, kSortThreads, sizeof(SortShared), stream>>>(P);
        st = launched(ASR_KERNEL_EMBEDDING);
    } else {
        TileParams P;
        P.ids = I;
        P.counts = words(L.counts);
        P.tiles = L.tiles;
        for (uint32_t shift = 0; shift < bits && st == ASR_OK; shift += kDigitBits) {
            P.shift = shift;
            P.first = shift == 0;
            P.key = words(L.key[now]);
            P.order = words(L.order[now]);
            now ^= 1;
            P.key_out = words(L.key[now]);
            P.order_out = words(L.order[now]);
            tile_count_kernel<<<L.tiles, kSortThreads, 0, stream>>>(P);
            st = launched(ASR_KERNEL_EMBEDDING);
            if (st != ASR_OK) return st;
            tile_scan_kernel<<<1, kSortThreads, 0, stream>>>(P);
            st = launched(ASR_KERNEL_EMBEDDING);
            if (st != ASR_OK) return st;
            tile_move_kernel<<<L.tiles, kSortThreads, 0, stream>>>(P);
            st = launched(ASR_KERNEL_EMBEDDING);
        }
        if (st != ASR_OK) return st;
        const SparseZeroParams P0{words(L.key[now]), tokens, static_cast<uint32_t>(vocab), Z};
        zero_kernel<<<zero_blocks, kThreads, 0, stream>>>(P0);
        st = launched(ASR_KERNEL_EMBEDDING);
    }
    if (st != ASR_OK || tokens == 0) return st;
    SumParams P;
    P.key = words(L.key[now]);
    P.order = words(L.order[now]);
    P.n = tokens;
    P.chunk = chunk_of(tokens);
    P.chunks = static_cast<uint32_t>((tokens + P.chunk - 1) / P.chunk);
    P.vocab = static_cast<uint32_t>(vocab);
    P.dim = dim;
    P.dy = kept::matrix(dy, dy_ld);
    P.out = kept::out(dtable, dim);
    P.head = reinterpret_cast<float *>(w + L.head);
    P.tail = reinterpret_cast<float *>(w + L.tail);
    P.scale = static_cast<float>(scale);
    const unsigned threads = dim >= kThreads * 8 ? kThreads : static_cast<unsigned>((dim + 255) / 256 * 32);
    const dim3 grid(P.chunks, static_cast<unsigned>((dim + threads * 8 - 1) / (threads * 8)));
    const bool bf = dtable_dtype == ASR_BF16;
    (dy_dtype == ASR_BF16 ? sums_of<ASR_BF16>(bf) : sums_of<ASR_F32>(bf))<<<grid, threads, 0, stream>>>(P);
    st = launched(ASR_KERNEL_EMBEDDING);
    if (st != ASR_OK) return st;
    (bf ? join_kernel<ASR_BF16> : join_kernel<ASR_F32>)<<<grid, threads, 0, stream>>>(P);
    return launched(ASR_KERNEL_EMBEDDING);
}

}  // namespace embed
