// embedding.cuh -- rows of a table picked by token, and the table's gradient.
// Included into asr.cu (inside its anonymous namespace), after checkpoint.cuh.
//
//   y_t = s T[id_t];   dT_v = s sum over t with id_t = v of dy_t, in the tokens' order
//
// The gradient is the whole table's, and most of its bytes are zeros.  Tokens are
// sorted by id, stably, so that every row's tokens lie together and in order; the
// sorted list is cut into chunks of one length, a block each (and a slice of the
// columns), whatever the ids -- a token that makes up half of a batch is as even a
// share of the work as any.  A block adds its tokens' rows up in registers: a row that
// begins and ends within the chunk is written at once, one that reaches over an end
// leaves a binary32 sum in the workspace, and the last of its blocks to finish adds
// those up, in order.
// Rows without tokens are zeroed beside the sort, as many as it takes the time of, and
// beside the sums.
//
// The sort is by digits of up to ten bits, from the lowest, each by counts and
// ranks: a warp ranks 32 keys at a time (lanes of one digit find one another), the
// warps' counts are added up by digit.  Up to 16,384 tokens are a cluster's of eight
// blocks, which read one another's counts and hand the keys to one another's shared
// memory (by one block alone 8,192 tokens took 20 us: its instructions); more are cut
// into tiles of 4,096, with a launch each for their counts, the tiles' places, and the
// moves.
//
// Bound by bytes: 8,192 tokens of a bf16 table of 128,256 x 4,096, with the time of its
// bytes at 6,697 GB/s: lookup 20.5 us (20.1), gradient 178 (167), 8 of them the sort's,
// with zeros beside it; 32,768 tokens 254 (197), the sort's launches and one block's
// sums of all counts in front of everything; 262,144 tokens of 1,024 columns 217 to 221
// (120).  Tokens of one id only have the last block of each slice add up all chunks: 8,192
// tokens 199, 262,144 tokens 956.

namespace embed {

using kept::live_of;

constexpr int kCluster = 8;
constexpr int kSortThreads = 256;
constexpr int kSortRounds = 8;                  // of 32 keys, a warp at most
constexpr int kSort = kCluster * kSortThreads * kSortRounds;        // keys a cluster sorts
constexpr int kTileThreads = 512;
constexpr int kTileRounds = 8;
constexpr int kTile = kTileThreads * kTileRounds;       // keys of one block of many
constexpr int kDigitBits = 10;
constexpr int kBins = 1 << kDigitBits;
constexpr int kThreads = 256;
constexpr int kZeroRows = 64;                   // of the table, a block at most
constexpr uint64_t kZeroBytes = 256 << 10;      // of zeros, a block beside the sort

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
    uint32_t dim;
    float scale;
};

template <int DT>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const __grid_constant__ LookupParams P, uint32_t spans)
{
    __shared__ kept::Stage stage;               // rows are aligned: not used
    const uint32_t lane = (threadIdx.x & 31) * 16;
    for (kept::Walk k(static_cast<uint32_t>(P.ids.n), spans); k.more(); k.next()) {
        const uint32_t id = key_of(P.ids, k.row), col = k.span * kept::kSpan + lane;
        const kept::Pair<DT> raw = kept::fetch16<DT, false>(P.table, id, col, id < P.ids.vocab ? P.dim : 0, P.table.vec, stage);
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            kept::values(raw.h[h], v[h]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[h][i] = id < P.ids.vocab ? __fmul_rn(v[h][i], P.scale) : __uint_as_float(0x7FC00000u);
        }
        kept::store16<DT, false>(P.y, k.row, col, P.dim, P.y.vec, v, stage);
    }
}

// Rows off alignment.
template <int DT>
__global__ void __launch_bounds__(kThreads) lookup_loose_kernel(const __grid_constant__ LookupParams P, uint32_t spans)
{
    for (kept::Walk k(static_cast<uint32_t>(P.ids.n), spans); k.more(); k.next()) {
        const uint32_t id = key_of(P.ids, k.row), first = k.span * kept::kSpan;
        float x[kept::kLoose];
        kept::fetch_loose<DT>(P.table, id, first, id < P.ids.vocab ? P.dim : 0, x);
#pragma unroll
        for (int i = 0; i < kept::kLoose; ++i)
            kept::store_loose1<DT>(P.y, k.row, first, P.dim, i, id < P.ids.vocab ? __fmul_rn(x[i], P.scale) : __uint_as_float(0x7FC00000u));
    }
}

// ---- sort

// Ranks of a block's keys by one digit.  Warp w holds keys w * rounds * 32 on, 32 a
// round.  Afterwards `counts` holds, for each warp and digit, how many keys of the
// digit the warps before have; totals[d] is the block's.
template <int ROUNDS, int WARPS>
__device__ __forceinline__ void rank_digits(const uint32_t key[ROUNDS], uint32_t live, uint32_t rounds, uint32_t shift,
                                            uint32_t bins, uint16_t (*counts)[kBins], uint32_t *totals,
                                            uint16_t rank[ROUNDS])
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (uint32_t i = lane; i < bins / 2; i += 32) reinterpret_cast<uint32_t *>(counts[warp])[i] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r >= rounds) break;
        const bool in = (live >> r) & 1;
        const uint32_t d = in ? (key[r] >> shift) & (bins - 1) : bins;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
        const uint32_t before = peers & ((1u << lane) - 1);
        if (in) rank[r] = static_cast<uint16_t>(counts[warp][d] + __popc(before));
        __syncwarp();
        if (in && before == 0) counts[warp][d] = static_cast<uint16_t>(counts[warp][d] + __popc(peers));
        __syncwarp();
    }
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < bins; d += WARPS * 32) {
        uint32_t c[WARPS], sum = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) c[w] = counts[w][d];
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            counts[w][d] = static_cast<uint16_t>(sum);
            sum += c[w];
        }
        totals[d] = sum;
    }
}

struct ZeroParams {
    void *p;                                    // vocab x dim
    uint64_t dim;
    uint32_t dtype;
};

// Zeroes rows v0 .. v0 + rows - 1 of the table but those set in `taken`.
__device__ __forceinline__ void zero_rows(const ZeroParams &Z, uint64_t v0, uint32_t rows, const uint32_t *taken)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint64_t size = Z.dtype == ASR_BF16 ? 2 : 4, bytes = Z.dim * size;
    for (uint32_t r = warp; r < rows; r += warps) {
        if ((taken[r >> 5] >> (r & 31)) & 1) continue;
        char *p = static_cast<char *>(Z.p) + (v0 + r) * bytes, *const end = p + bytes;
        // up to 16 bytes' alignment value by value, then in 16 bytes, then the rest
        char *const even = p + ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15);
        const uint64_t whole = even < end ? static_cast<uint64_t>(end - even) / 16 * 16 : 0;
        for (uint64_t i = lane * 16ull; i < whole; i += 512) *reinterpret_cast<uint4 *>(even + i) = make_uint4(0, 0, 0, 0);
        char *const rest = even + whole;        // past `end` where the row ends before its first 16 bytes
        if (Z.dtype == ASR_BF16) {
            if (p + lane * 2 < (even < end ? even : end)) reinterpret_cast<uint16_t *>(p)[lane] = 0;
            if (rest + lane * 2 < end) reinterpret_cast<uint16_t *>(rest)[lane] = 0;
        } else {
            if (p + lane * 4 < (even < end ? even : end)) reinterpret_cast<float *>(p)[lane] = 0.0f;
            if (rest + lane * 4 < end) reinterpret_cast<float *>(rest)[lane] = 0.0f;
        }
    }
}

struct SortParams {
    Ids ids;
    uint32_t *key, *order;
    uint32_t passes, width;                     // digits of a key (vocab among them) and their bits
    uint32_t log_rounds;                        // of 32 keys a warp
    uint32_t rows;                              // a block zeroes
    uint32_t *arrived, counters;                // zeroed for the sums
    ZeroParams zero;
};

struct __align__(16) SortShared {
    uint64_t item[kSortThreads * kSortRounds];  // keys and where they came from
    uint16_t counts[kSortThreads / 32][kBins];
    uint32_t totals[kBins], base[kBins];        // of this block; places of its keys of each digit
    uint32_t part[kSortThreads / 32];
    uint32_t taken[kZeroRows / 32];
};

__device__ __forceinline__ uint4 remote_words(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Up to kSort tokens: the first cluster sorts, the other blocks zero rows that no token
// has.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads)
    sort_kernel(const __grid_constant__ SortParams P)
{
    __shared__ SortShared S;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x >= kCluster) {
        const uint64_t v0 = (blockIdx.x - kCluster) * static_cast<uint64_t>(P.rows);
        if (v0 >= P.ids.vocab) return;
        const uint32_t rows = P.ids.vocab - v0 < P.rows ? static_cast<uint32_t>(P.ids.vocab - v0) : P.rows;
        if (threadIdx.x < kZeroRows / 32) S.taken[threadIdx.x] = 0;
        __syncthreads();
#pragma unroll 4
        for (uint64_t t = threadIdx.x; t < P.ids.n; t += kSortThreads) {
            const uint64_t d = key_of(P.ids, t) - v0;
            if (d < rows) atomicOr(S.taken + (d >> 5), 1u << (d & 31));
        }
        __syncthreads();
        zero_rows(P.zero, v0, rows, S.taken);
        return;
    }
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = blockIdx.x;
    const uint32_t n = static_cast<uint32_t>(P.ids.n), rounds = 1u << P.log_rounds, log_share = 8 + P.log_rounds;
    const uint32_t at = warp * rounds * 32 + lane, bins = 1u << P.width;       // place in the block's share
    static_assert(kSortThreads == 1 << 8, "a block's share is 2^log_share keys");
    for (uint32_t i = block * kSortThreads + threadIdx.x; i < P.counters; i += kCluster * kSortThreads) P.arrived[i] = 0;
    uint32_t key[kSortRounds], live = 0;
    uint16_t from[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const uint32_t t = (block << log_share) + at + r * 32;
        key[r] = 0;
        from[r] = static_cast<uint16_t>(t);
        if (r < rounds && t < n) live |= 1u << r, key[r] = key_of(P.ids, t);
    }
    for (uint32_t pass = 0, shift = 0; pass < P.passes; ++pass, shift += P.width) {
        rank_digits<kSortRounds, kSortThreads / 32>(key, live, rounds, shift, bins, S.counts, S.totals, rank);
        gemm::cluster_sync();
        // four digits a thread: all blocks' keys of them, those of the blocks before, and the digits before
        uint32_t all[4] = {}, before[4] = {};
        if (threadIdx.x * 4 < bins) {
            uint4 c[kCluster];
#pragma unroll
            for (int b = 0; b < kCluster; ++b) c[b] = remote_words(gemm::peer_addr(smem_addr(S.totals + threadIdx.x * 4), b));
#pragma unroll
            for (int b = 0; b < kCluster; ++b) {
                const uint32_t w[4] = {c[b].x, c[b].y, c[b].z, c[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t k = threadIdx.x * 4 + i < bins ? w[i] : 0;
                    all[i] += k;
                    before[i] += b < block ? k : 0;
                }
            }
        }
        const uint32_t own = all[0] + all[1] + all[2] + all[3];
        uint32_t v = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= static_cast<uint32_t>(d)) v += o;
        }
        if (lane == 31) S.part[warp] = v;
        __syncthreads();
        v -= own;
        for (uint32_t w = 0; w < warp; ++w) v += S.part[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            S.base[threadIdx.x * 4 + i] = v + before[i];
            v += all[i];
        }
        __syncthreads();
        const bool last = pass + 1 == P.passes;
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r)
            if ((live >> r) & 1) {
                const uint32_t d = (key[r] >> shift) & (bins - 1), to = S.base[d] + S.counts[warp][d] + rank[r];
                if (last) {
                    P.key[to] = key[r];
                    P.order[to] = from[r];
                } else {
                    const uint32_t p = gemm::peer_addr(smem_addr(S.item + (to & ((1u << log_share) - 1))), to >> log_share);
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(p),
                                 "l"(static_cast<uint64_t>(key[r]) << 32 | from[r]) : "memory");
                }
            }
        // what the others read of this block has been read, and what they hand it is there
        gemm::cluster_sync();
        if (last) break;
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r)
            if ((live >> r) & 1) {
                const uint64_t v = S.item[at + r * 32];
                key[r] = static_cast<uint32_t>(v >> 32);
                from[r] = static_cast<uint16_t>(v);
            }
    }
}

// More tokens: one digit's counts of each tile, their places, and the moves.
struct TileParams {
    Ids ids;                                    // first digit: where the keys come from
    const uint32_t *key, *order;                // later ones
    uint32_t *key_out, *order_out;
    uint32_t *counts;                           // [bin][tile]
    uint32_t tiles, shift, bins, first;
    uint32_t *arrived, counters;                // zeroed for the sums, with the first digit
};

__global__ void __launch_bounds__(kTileThreads) tile_count_kernel(const __grid_constant__ TileParams P)
{
    __shared__ uint32_t bins[kBins];
    for (uint32_t i = threadIdx.x; i < P.bins; i += kTileThreads) bins[i] = 0;
    __syncthreads();
    if (P.first)
        for (uint32_t i = blockIdx.x * kTileThreads + threadIdx.x; i < P.counters; i += gridDim.x * kTileThreads) P.arrived[i] = 0;
    for (int r = 0; r < kTileRounds; ++r) {
        const uint64_t t = blockIdx.x * static_cast<uint64_t>(kTile) + r * kTileThreads + threadIdx.x;
        if (t < P.ids.n) atomicAdd(bins + (((P.first ? key_of(P.ids, t) : P.key[t]) >> P.shift) & (P.bins - 1)), 1u);
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < P.bins; i += kTileThreads) P.counts[i * static_cast<uint64_t>(P.tiles) + blockIdx.x] = bins[i];
}

// Every count becomes the sum of those before it: one block.
constexpr int kScanThreads = 1024;

__global__ void __launch_bounds__(kScanThreads) tile_scan_kernel(const __grid_constant__ TileParams P)
{
    __shared__ uint32_t part[32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t n = static_cast<uint64_t>(P.bins) * P.tiles;
    uint32_t carry = 0;
    for (uint64_t at = 0; at < n; at += kScanThreads * 4) {
        const uint64_t i = at + threadIdx.x * 4;            // n may end within the four: two bins of an odd number of tiles
        uint32_t c[4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) c[k] = P.counts[i + k];
        const uint32_t own = c[0] + c[1] + c[2] + c[3];
        uint32_t v = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= static_cast<uint32_t>(d)) v += o;
        }
        __syncthreads();
        if (lane == 31) part[warp] = v;
        __syncthreads();
        uint32_t mine = part[lane], before = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (lane >= static_cast<uint32_t>(d)) before += o;
        }
        const uint32_t total = __shfl_sync(0xFFFFFFFFu, before, 31);
        v += carry + __shfl_sync(0xFFFFFFFFu, before - mine, warp) - own;
        carry += total;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (i + k < n) P.counts[i + k] = v;
            v += c[k];
        }
    }
}

struct TileShared {
    uint16_t counts[kTileThreads / 32][kBins];
    uint32_t totals[kBins];
};

__global__ void __launch_bounds__(kTileThreads) tile_move_kernel(const __grid_constant__ TileParams P)
{
    __shared__ TileShared S;
    const uint32_t warp = threadIdx.x >> 5;
    const uint64_t t0 = blockIdx.x * static_cast<uint64_t>(kTile) + warp * (kTileRounds * 32) + (threadIdx.x & 31);
    uint32_t key[kTileRounds], from[kTileRounds], live = 0;
    uint16_t rank[kTileRounds];
#pragma unroll
    for (int r = 0; r < kTileRounds; ++r) {
        const uint64_t t = t0 + r * 32;
        key[r] = from[r] = 0;
        if (t < P.ids.n) {
            live |= 1u << r;
            key[r] = P.first ? key_of(P.ids, t) : P.key[t];
            from[r] = P.first ? static_cast<uint32_t>(t) : P.order[t];
        }
    }
    rank_digits<kTileRounds, kTileThreads / 32>(key, live, kTileRounds, P.shift, P.bins, S.counts, S.totals, rank);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTileRounds; ++r)
        if ((live >> r) & 1) {
            const uint32_t d = (key[r] >> P.shift) & (P.bins - 1);
            const uint64_t to = static_cast<uint64_t>(P.counts[d * static_cast<uint64_t>(P.tiles) + blockIdx.x]) +
                                S.counts[warp][d] + rank[r];
            P.key_out[to] = key[r];
            P.order_out[to] = from[r];
        }
}

// The first place in the sorted keys that holds `key` or more: 33 parts a step, by a warp.
__device__ __forceinline__ uint64_t lower_bound(const uint32_t *keys, uint64_t n, uint64_t key)
{
    const uint32_t lane = threadIdx.x & 31;
    uint64_t lo = 0, hi = n;                    // keys before lo are less, from hi on not
    while (lo < hi) {
        const uint64_t part = (hi - lo + 32) / 33, at = lo + (lane + 1) * part - 1;
        const bool less = at < hi && keys[at] < key;
        const uint32_t below = __popc(__ballot_sync(0xFFFFFFFFu, less));
        const uint64_t end = lo + (below + 1) * part - 1;
        lo += below * part;
        hi = below < 32 && end < hi ? end : hi;
    }
    return lo;
}

// ---- sums

struct SumParams {
    const uint32_t *key, *order;
    uint64_t n;                                 // tokens
    uint32_t chunk, chunks, slices, vocab;
    uint64_t dim, pitch;                        // of a row of sums
    kept::Matrix dy;
    kept::Out out;
    float *head, *tail;                         // [chunk][pitch]: sums of a row that began before, that goes on after
    uint32_t *arrived;                          // [chunk][slice]: blocks that have left theirs of the row that goes on there
    float scale;
    uint32_t zero_from;                         // rows before are zeroed already
    ZeroParams zero;
};

// A warp's 256 columns of a row, eight a lane from `col` on.  OFF: rows off alignment.
template <int OT, bool OFF>
__device__ __forceinline__ void store_row(const SumParams &P, uint32_t row, uint32_t col, int live, float v[8], kept::Stage &S)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], P.scale);
    if (OFF) {
        const uint32_t lane = threadIdx.x & 31, first = col - lane * 8;
        __syncwarp();
        kept::put_staged<OT>(S, lane, kept::rounded<OT>(v));
        kept::stage_out<OT, 8>(S, [&](uint32_t e) -> void * {
            return first + e < P.dim ? static_cast<char *>(P.out.p) + kept::place(row, P.out.ld, first + e) * (OT == ASR_BF16 ? 2 : 4)
                                     : nullptr;
        });
    } else {
        kept::store8<OT>(P.out, row, col, live, P.out.vec, v);
    }
}

__device__ __forceinline__ void store_sum(float *p, const float v[8])
{
    __stcg(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcg(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}

__device__ __forceinline__ void add_sum(float acc[8], const float *p)
{
    const float4 a = __ldcg(reinterpret_cast<const float4 *>(p)), b = __ldcg(reinterpret_cast<const float4 *>(p) + 1);
    acc[0] = __fadd_rn(acc[0], a.x), acc[1] = __fadd_rn(acc[1], a.y), acc[2] = __fadd_rn(acc[2], a.z);
    acc[3] = __fadd_rn(acc[3], a.w), acc[4] = __fadd_rn(acc[4], b.x), acc[5] = __fadd_rn(acc[5], b.y);
    acc[6] = __fadd_rn(acc[6], b.z), acc[7] = __fadd_rn(acc[7], b.w);
}

// Block c has left its sum of `row`, which reaches over chunks' ends (`began`: from
// before this one).  The last one to do so adds them all up: of the chunk where the row
// begins its tail, of the others their heads, in order.  All threads of the block come
// here together.
template <int OT, bool OFF>
__device__ __forceinline__ void join(const SumParams &P, uint32_t c, uint32_t row, bool began, uint32_t slice, uint32_t col,
                                     int live, kept::Stage &S)
{
    __shared__ uint32_t ends[2], before;
    __threadfence();                            // what this thread has left, before its block is counted
    __syncthreads();
    if (threadIdx.x < 32) {
        // the chunks that begin with the row follow one another: 32 a look
        uint32_t first = c, last = c;
        for (uint32_t up = 32, down = began ? 32 : 0; up == 32 || down == 32;) {
            const uint64_t d = static_cast<uint64_t>(last) + 1 + threadIdx.x;
            const uint32_t e = first - threadIdx.x;
            const bool after = up == 32 && d < P.chunks && P.key[d * P.chunk] == row;
            const bool before = down == 32 && threadIdx.x < first && P.key[static_cast<uint64_t>(e) * P.chunk - 1] == row;
            up = __popc(__ballot_sync(0xFFFFFFFFu, after));
            down = __popc(__ballot_sync(0xFFFFFFFFu, before));
            last += up;
            first -= down;
        }
        if (threadIdx.x == 0) {
            ends[0] = first;
            ends[1] = last;
            before = atomicAdd(P.arrived + static_cast<uint64_t>(first) * P.slices + slice, 1u);
            __threadfence();
        }
    }
    __syncthreads();
    const uint32_t first = ends[0], last = ends[1];
    if (before != last - first) return;
    float acc[8] = {};
    if (live) {
        add_sum(acc, P.tail + first * P.pitch + col);
#pragma unroll 8
        for (uint32_t d = first + 1; d <= last; ++d) add_sum(acc, P.head + d * P.pitch + col);
    }
    store_row<OT, OFF>(P, row, col, live, acc, S);
}

// A block a chunk and a slice of the columns, eight a thread; the blocks behind those
// zero rows without tokens.
constexpr int kSumThreads = 128;                // at most
constexpr int kPiece = 64;                      // tokens whose keys are at hand

template <int DT, int OT, bool OFF>
__global__ void __launch_bounds__(kSumThreads, OFF ? 4 : 6) sum_kernel(const __grid_constant__ SumParams P)
{
    constexpr int kAhead = DT == ASR_BF16 && !OFF ? 8 : 4;          // rows fetched before they are added up
    __shared__ kept::Stage stages[OFF ? kSumThreads / 32 : 1];
    kept::Stage &stage = stages[OFF ? threadIdx.x >> 5 : 0];
    __shared__ uint32_t key[kPiece + 2], order[kPiece];     // keys from the one before on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t sums = P.chunks * P.slices;
    if (blockIdx.x >= sums) {
        const uint64_t v0 = P.zero_from + (blockIdx.x - sums) * static_cast<uint64_t>(kZeroRows);
        const uint32_t rows = P.vocab - v0 < kZeroRows ? static_cast<uint32_t>(P.vocab - v0) : kZeroRows;
        uint32_t *taken = key;
        if (threadIdx.x < kZeroRows / 32) taken[threadIdx.x] = 0;
        __syncthreads();
        const uint64_t lo = lower_bound(P.key, P.n, v0), hi = lower_bound(P.key, P.n, v0 + rows);
        // a row's tokens may be many: each is looked for on its own
        for (uint32_t d = threadIdx.x; d < rows; d += blockDim.x) {
            uint64_t a = lo, b = hi;
            while (a < b) {
                const uint64_t mid = (a + b) / 2;
                if (P.key[mid] < v0 + d) a = mid + 1;
                else b = mid;
            }
            if (a < hi && P.key[a] == v0 + d) atomicOr(taken + (d >> 5), 1u << (d & 31));
        }
        __syncthreads();
        zero_rows(P.zero, v0, rows, taken);
        return;
    }
    const uint32_t c = blockIdx.x / P.slices, slice = blockIdx.x % P.slices;
    const uint32_t col = (slice * blockDim.x + threadIdx.x) * 8, warp_col = col - (threadIdx.x & 31) * 8;
    const int live = live_of(static_cast<uint32_t>(P.dim), col);
    const uint64_t begin = static_cast<uint64_t>(c) * P.chunk, end = begin + P.chunk < P.n ? begin + P.chunk : P.n;
    float acc[8] = {};
    bool first = true;                          // still in the chunk's first row
    bool began = false, goes_on = false;        // that one before the chunk; the last one after it
    uint32_t front = 0, back = 0;
    for (uint64_t i0 = begin; i0 < end; i0 += kPiece) {
        const uint32_t n = end - i0 < kPiece ? static_cast<uint32_t>(end - i0) : kPiece;
        __syncthreads();
        for (uint32_t j = threadIdx.x; j < kPiece + 2; j += blockDim.x) {
            const uint64_t i = i0 + j;          // of the key before place i0 + j - 1's
            key[j] = j <= n + 1 && i > 0 && i <= P.n ? P.key[i - 1] : P.vocab;
            if (j < kPiece) order[j] = j < n ? P.order[i0 + j] : 0;
        }
        __syncthreads();
        const uint32_t *const keys = key + 1;
        if (i0 == begin) {
            front = keys[0];
            began = begin > 0 && key[0] == front;
        }
        back = keys[n - 1];
        goes_on = i0 + n < P.n && keys[n] == back;
        for (uint32_t a0 = 0; a0 < n && keys[a0] < P.vocab; a0 += kAhead) {
            kept::Raw<DT> raw[kAhead];
            if (OFF) {
                // all rows' values side by side first, then each in turn through shared memory
                using Word = typename kept::WordOf<DT>::type;
                Word v[kAhead][8];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const bool in = a0 + a < n && keys[a0 + a] < P.vocab;
                    const Word *from = static_cast<const Word *>(P.dy.p) + kept::place(in ? order[a0 + a] : 0, P.dy.ld, warp_col);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t e = 32 * i + (threadIdx.x & 31);
                        v[a][i] = in && warp_col + e < P.dim ? from[e] : static_cast<Word>(0);
                    }
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) reinterpret_cast<Word *>(stage.w)[32 * i + (threadIdx.x & 31)] = v[a][i];
                    __syncwarp();
                    raw[a] = kept::staged<DT>(stage, threadIdx.x & 31);
                }
            } else {
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const bool in = a0 + a < n && keys[a0 + a] < P.vocab;
                    raw[a] = kept::fetch<DT>(P.dy, in ? order[a0 + a] : 0, col, in ? live : 0, P.dy.vec);
                }
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (a0 + a >= n || keys[a0 + a] >= P.vocab) break;
                float v[8];
                kept::values(raw[a], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], v[i]);
                const bool last = i0 + a0 + a + 1 == end;
                if (!last && keys[a0 + a + 1] == keys[a0 + a]) continue;
                if (first && began) {
                    if (live) store_sum(P.head + c * P.pitch + col, acc);
                } else if (last && goes_on) {
                    if (live) store_sum(P.tail + c * P.pitch + col, acc);
                } else {
                    store_row<OT, OFF>(P, keys[a0 + a], col, live, acc, stage);
                }
                first = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
            }
        }
    }
    // the chunk's first row, if it began before, and its last, if that goes on and is not the same
    if (began && front < P.vocab) join<OT, OFF>(P, c, front, true, slice, col, live, stage);
    if (goes_on && back < P.vocab && !(began && front == back)) join<OT, OFF>(P, c, back, false, slice, col, live, stage);
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

using SumKernel = void (*)(const SumParams);

template <int DT, bool OFF>
SumKernel sums_of(int32_t out)
{
    return out == ASR_BF16 ? sum_kernel<DT, ASR_BF16, OFF> : sum_kernel<DT, ASR_F32, OFF>;
}

SumKernel sums_of(int32_t dy, int32_t out, bool off)
{
    if (off) return dy == ASR_BF16 ? sums_of<ASR_BF16, true>(out) : sums_of<ASR_F32, true>(out);
    return dy == ASR_BF16 ? sums_of<ASR_BF16, false>(out) : sums_of<ASR_F32, false>(out);
}

asr_status setup()
{
    static std::atomic<uint64_t> ready{0};
    return kept::load_once(ready, lookup_kernel<ASR_F32>, lookup_kernel<ASR_BF16>, lookup_loose_kernel<ASR_F32>,
                           lookup_loose_kernel<ASR_BF16>, sort_kernel, tile_count_kernel,
                           tile_scan_kernel, tile_move_kernel, sums_of(ASR_F32, ASR_F32, false),
                           sums_of(ASR_F32, ASR_BF16, false), sums_of(ASR_BF16, ASR_F32, false),
                           sums_of(ASR_BF16, ASR_BF16, false), sums_of(ASR_F32, ASR_F32, true), sums_of(ASR_F32, ASR_BF16, true),
                           sums_of(ASR_BF16, ASR_F32, true), sums_of(ASR_BF16, ASR_BF16, true));
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
    P.table = kept::matrix(table, table_ld, dtype);
    P.y = kept::out(y, y_ld, dtype);
    P.dim = static_cast<uint32_t>(dim);
    P.scale = static_cast<float>(scale);
    auto kernel = dtype == ASR_BF16 ? lookup_kernel<ASR_BF16> : lookup_kernel<ASR_F32>;
    if (!P.table.vec || !P.y.vec) kernel = dtype == ASR_BF16 ? lookup_loose_kernel<ASR_BF16> : lookup_loose_kernel<ASR_F32>;
    return kept::walk(ASR_KERNEL_EMBEDDING, kernel, P, tokens, dim, kept::kSpan, stream);
}

// Columns go to blocks of up to 128 threads, and tokens to chunks of 8 to 64, in eights,
// that make about 1,216 blocks (eight an SM; of 8,192 x 4,096 tokens 32 make 1,024):
// shorter ones leave more sums in the workspace, longer ones are too few.  More than
// 524,288 tokens go to longer chunks, of any length: never more than 8,192 of them, each of
// which takes two rows of sums.
unsigned threads_of(uint64_t dim)
{
    return dim >= kSumThreads * 8 ? kSumThreads : static_cast<unsigned>((dim + 255) / 256 * 32);
}

uint64_t slices_of(uint64_t dim) { return (dim + threads_of(dim) * 8 - 1) / (threads_of(dim) * 8); }

uint32_t chunk_of(uint64_t tokens, uint64_t dim)
{
    const uint64_t even = (tokens * slices_of(dim) / 1216 + 7) / 8 * 8, least = (tokens + 8191) / 8192;
    const uint64_t c = even < 8 ? 8 : even > 64 ? 64 : even;
    return static_cast<uint32_t>(c < least ? least : c);
}

struct Layout {
    uint64_t key[2], order[2], counts, arrived, head, tail, bytes;
    uint32_t tiles, counters;                   // no tiles: one cluster sorts
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
    L.tiles = tokens <= kSort ? 0 : static_cast<uint32_t>((tokens + kTile - 1) / kTile);
    const uint64_t chunk = chunk_of(tokens, dim), chunks = (tokens + chunk - 1) / chunk;
    for (int i = 0; i < 2; ++i) {
        const bool used = i == 0 || L.tiles;
        L.key[i] = take(used ? tokens * 4 : 0);
        L.order[i] = take(used ? tokens * 4 : 0);
    }
    L.counts = take(static_cast<uint64_t>(kBins) * L.tiles * 4);
    L.counters = static_cast<uint32_t>(chunks * slices_of(dim));
    L.arrived = take(L.counters * 4ull);
    L.head = take(chunks * muon::up(dim, 8) * 4);
    L.tail = take(chunks * muon::up(dim, 8) * 4);
    L.bytes = at;
    return L;
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
    const ZeroParams Z{dtable, dim, static_cast<uint32_t>(dtable_dtype)};
    uint32_t bits = 1;
    while ((vocab >> bits) != 0) ++bits;
    const uint32_t passes = (bits + kDigitBits - 1) / kDigitBits, width = (bits + passes - 1) / passes;
    int now = 0;
    uint64_t zeroed = 0;
    if (L.tiles == 0) {
        // as many zeros beside the sort as the GPU writes meanwhile: a block an SM
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e);
        const uint64_t row = dim * (dtable_dtype == ASR_BF16 ? 2 : 4), fit = kZeroBytes / row;
        SortParams P;
        P.ids = I;
        P.key = words(L.key[0]);
        P.order = words(L.order[0]);
        P.passes = passes;
        P.width = width;
        P.log_rounds = 0;
        while ((static_cast<uint64_t>(kCluster * kSortThreads) << P.log_rounds) < tokens) ++P.log_rounds;
        P.rows = static_cast<uint32_t>(fit < 1 ? 1 : fit > kZeroRows ? kZeroRows : fit);
        P.arrived = words(L.arrived);
        P.counters = tokens ? L.counters : 0;
        P.zero = Z;
        const uint64_t all = (vocab + P.rows - 1) / P.rows, beside = tokens ? static_cast<uint64_t>(sms) : all;
        const unsigned blocks = static_cast<unsigned>(all < beside ? all : beside);
        zeroed = static_cast<uint64_t>(blocks) * P.rows;
        sort_kernel<<<(kCluster + blocks + kCluster - 1) / kCluster * kCluster, kSortThreads, 0, stream>>>(P);
        st = launched(ASR_KERNEL_EMBEDDING);
    } else {
        TileParams P;
        P.ids = I;
        P.counts = words(L.counts);
        P.tiles = L.tiles;
        P.bins = 1u << width;
        P.arrived = words(L.arrived);
        P.counters = L.counters;
        for (uint32_t pass = 0; pass < passes; ++pass) {
            P.shift = pass * width;
            P.first = pass == 0;
            P.key = words(L.key[now]);
            P.order = words(L.order[now]);
            now ^= 1;
            P.key_out = words(L.key[now]);
            P.order_out = words(L.order[now]);
            tile_count_kernel<<<L.tiles, kTileThreads, 0, stream>>>(P);
            st = launched(ASR_KERNEL_EMBEDDING);
            if (st != ASR_OK) return st;
            tile_scan_kernel<<<1, kScanThreads, 0, stream>>>(P);
            st = launched(ASR_KERNEL_EMBEDDING);
            if (st != ASR_OK) return st;
            tile_move_kernel<<<L.tiles, kTileThreads, 0, stream>>>(P);
            st = launched(ASR_KERNEL_EMBEDDING);
            if (st != ASR_OK) return st;
        }
    }
    if (st != ASR_OK || tokens == 0) return st;
    SumParams P;
    P.key = words(L.key[now]);
    P.order = words(L.order[now]);
    P.n = tokens;
    P.chunk = chunk_of(tokens, dim);
    P.chunks = static_cast<uint32_t>((tokens + P.chunk - 1) / P.chunk);
    P.slices = static_cast<uint32_t>(slices_of(dim));
    P.vocab = static_cast<uint32_t>(vocab);
    P.dim = dim;
    P.pitch = muon::up(dim, 8);
    P.dy = kept::matrix(dy, dy_ld, dy_dtype);
    P.out = kept::out(dtable, dim, dtable_dtype);
    P.head = reinterpret_cast<float *>(w + L.head);
    P.tail = reinterpret_cast<float *>(w + L.tail);
    P.arrived = words(L.arrived);
    P.scale = static_cast<float>(scale);
    P.zero_from = static_cast<uint32_t>(zeroed < vocab ? zeroed : vocab);
    P.zero = Z;
    const unsigned threads = threads_of(dim), sums = P.chunks * P.slices;
    const unsigned zeros = static_cast<unsigned>((vocab - P.zero_from + kZeroRows - 1) / kZeroRows);
    return prod::launch_early(ASR_KERNEL_EMBEDDING, sums_of(dy_dtype, dtable_dtype, !P.dy.vec || !P.out.vec), dim3(sums + zeros),
                              threads, P, stream);
}

}  // namespace embed
