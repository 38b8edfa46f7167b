// product.cuh -- batched matrix products with f16 operands on the
// 5th-generation tensor cores: the kernel of the Newton-Schulz orthogonalisation
// (muon.cuh), and what the 8-bit integer product's (int8_product.cuh) shares with
// it.  Included into asr.cu (inside its anonymous namespace), after gemm_sr.cuh,
// whose cluster, barrier and tensor-map helpers it uses.
//
// out_z = epilogue(A_z . B_z^T) for the matrices z of a stack, with binary32
// sums.  The shape is gemm_sr.cuh's two-SM kernel: 256 x 256 tiles on clusters
// of two CTAs, tcgen05.mma.cta_group::2 (kind::f16), 128-deep K slices in a
// 3-stage ring of 64 KB, two TMEM accumulators.  What differs:
//   - operands are f16, in a workspace that the library lays out itself (rows
//     a multiple of 32 bytes apart), so every size and alignment of the
//     caller's matrices takes this one path;
//   - an operand is stored with the contraction contiguous ("K-major") or
//     across it ("MN-major"): X X^T and B X, or X^T X and X B, are formed from
//     the one row-major X, and nothing is ever transposed in memory;
//   - a product whose result is symmetric computes the tiles on and above the
//     diagonal and writes each of the others as a mirror image: half the work;
//   - sixteen epilogue warps: a tile's epilogue is exposed at a launch's end (last
//     products of ortho and Muon steps 31 and 87 us, with eight warps that took 32
//     columns at a time 49 and 111 us); what they read for a block is on its way
//     while they finish the one before (3 stacked 515 x 1,365: 161 us, 165 with
//     the loads where they are used);
//   - the tiles of a last round that would leave most pairs idle go in halves or
//     quarters of their columns.
// What bounds it: large products run at the tensor cores' sustained rate under
// the power limit (8,192 x 14,336 x 4,096 integers: 528 us alone, 1,820 TFLOP/s);
// short ones at the L2's (a 256 x 256 tile moves 64 bytes a cycle and SM), or,
// below about 10 us, at the chain of launch (1.4 us after the last kernel's end),
// first copies (1.6 us), epilogue and exit (2 us).
//
// A K-half of a stage (64 of K, 16 KB an operand and CTA) in shared memory:
//   K-major    128 rows of 128 bytes, 128-byte swizzle; a K=16 step is 32 bytes;
//   MN-major   two blocks of 64 rows' columns: 64 K-lines of 128 bytes each
//              (64 values across), 128-byte swizzle; groups of 8 K-lines are
//              1,024 bytes apart (stride offset), the blocks 8,192 (leading
//              offset); a K=16 step is 2,048 bytes.

namespace prod {

using gemm::cluster_rank;
using gemm::cluster_sync;
using gemm::mbar_arrive_remote;
using gemm::mbar_wait_cluster;
using gemm::mma_bf16_pair;          // the instruction descriptor names the operand type
using gemm::mma_commit_pair;
using gemm::pair_wait;
using gemm::peer_addr;
using gemm::st_global_v8;
using gemm::tile_coords;

constexpr int kTile = 256;                      // tile rows and columns of a CTA pair
constexpr int kBK = 128;                        // K per stage, two halves of 64
constexpr int kStages = 3;
constexpr int kEpi = 16;                        // epilogue warps: four per TMEM lane quarter
constexpr int kThreads = 64 + 32 * kEpi;
constexpr int kSpan = kTile / (kEpi / 4);       // columns per epilogue warp
static_assert(kSpan == 64, "two words a lane hold a warp's column gains");
constexpr uint32_t kHalfBytes = 128 * 64 * 2;   // a K-half of one operand in one CTA
constexpr uint32_t kStageBytes = 4 * kHalfBytes;
constexpr int kAccBufs = 2;
constexpr uint32_t kTmemCols = kTile * kAccBufs;
constexpr int kBars = kStages * 3 + 2 * kAccBufs + 1;
constexpr int kBlock = 16;                      // columns an epilogue warp finishes at a time
// Per epilogue warp, 32 rows x 16 columns of binary32 on their way out.
constexpr uint32_t kWarpStage = 32 * kBlock * 4;
constexpr int kBarBytes = (kBars * 8 + 16 + 127) / 128 * 128;
constexpr int kSmem = 1024 + kStages * kStageBytes + kBarBytes + kEpi * kWarpStage;
constexpr int kGroupM = 16;                     // tile order: rows of tiles walked across together (8: 1 % slower)
constexpr int kMaxBatch = 64;                   // matrices per launch

// What the epilogue makes of a sum.  "Stored" values are f16 at 2^12 times the
// matrix, S and P with their diagonals' rounding kept besides (see muon.cuh).
enum Op {
    kGram,      // stored S = alpha * sum, symmetric; its diagonal
    kPoly,      // stored P = alpha * sum + beta * (stored S) + shift on the diagonal, symmetric; its rows' gains
    kNext,      // stored X' = alpha * gain * sum
    kOut,       // caller's bf16 matrix = alpha * sum, to nearest
    kParam,     // caller's parameter p = p * beta - alpha * sum, f32 or rounded to bf16
    kScaled     // caller's matrix = sum * row scale * column scale (int8_product.cuh)
};

struct Slot {                       // one matrix of the stack: the caller's
    void *ptr;
    uint64_t base;                  // global index of its first element (kParam)
};

struct Params {
    uint32_t m, n, k, batch;
    uint32_t tiles_m, tiles_n, per_matrix;
    uint32_t wide, narrow;          // work items: whole tiles, then parts of the last ones
    uint32_t parts;                 // 1, 2 or 4: a narrow item is 256 / parts columns
    float alpha, beta, shift;
    uint32_t ld;                    // stored output (and S): elements between rows
    uint64_t stride;                // and between matrices
    __half *out;
    const __half *aux;
    float *diag, *gain;             // of S, before its rounding; of P's rows.  `side` between matrices
    uint32_t side;
    // the caller's output
    uint64_t out_ld;
    uint32_t out_dtype;             // asr_dtype
    uint32_t rounding;              // asr_rounding
    uint32_t vec;                   // rows are 32-byte aligned throughout: 256-bit accesses
    uint32_t step;
    const float *row_scale, *col_scale;
    RoundKeys keys;
    Slot slot[kMaxBatch];
};

__host__ __device__ constexpr uint32_t instr_desc(uint32_t n, bool a_mn, bool b_mn)
{
    return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) |
           (uint32_t(kTile >> 4) << 24);
}

template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(MN ? 8192u >> 4 : 1u) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                                 uint32_t cluster_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
        : "memory");
}

// Word of row r, column c of a staging area: columns change places by row, so
// that neither 32 rows of a column nor two whole rows collide in a bank.
__device__ __forceinline__ uint32_t staged(uint32_t r, uint32_t c) { return r * kBlock + (c ^ ((r >> 1) & 15u)); }

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack_f16(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Tile w of a matrix whose result is symmetric: column nt of the upper
// triangle holds nt + 1 tiles.
__device__ __forceinline__ void triangle_coords(uint32_t w, uint32_t &mt, uint32_t &nt)
{
    uint32_t c = static_cast<uint32_t>((sqrtf(8.0f * static_cast<float>(w) + 1.0f) - 1.0f) * 0.5f);
    while (c * (c + 1) / 2 > w) --c;
    while ((c + 1) * (c + 2) / 2 <= w) ++c;
    nt = c;
    mt = w - c * (c + 1) / 2;
}

// One lane of the warp, the same each time.  The producer and the MMA warp run
// their loops with all lanes and let one issue: their addresses and descriptors
// then stay in uniform registers.  Issued by a lone lane, each tcgen05.mma cost
// about 90 cycles (measured at M = 128, where one with N = 48 takes 25).
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0); }

// A wait by all lanes of a warp, which go on, or give up, together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xFFFFFFFFu, pair_wait(bar, parity, limit_ns));
}

struct Item {
    uint32_t z, m0, n0, width;
    bool mirror;
};

template <bool SYM>
__device__ __forceinline__ Item work_item(const Params &P, uint32_t t)
{
    Item it;
    uint32_t whole = t, part = 0;
    it.width = kTile;
    if (t >= P.wide) {
        whole = P.wide + (t - P.wide) / P.parts;
        part = (t - P.wide) & (P.parts - 1);
        it.width = kTile / P.parts;
    }
    it.z = whole / P.per_matrix;
    uint32_t mt, nt;
    if (SYM) triangle_coords(whole % P.per_matrix, mt, nt);
    else tile_coords(whole % P.per_matrix, P.tiles_m, P.tiles_n, mt, nt, kGroupM);
    it.m0 = mt * kTile;
    it.n0 = nt * kTile + part * it.width;
    it.mirror = SYM && mt != nt;
    return it;
}

__device__ __forceinline__ void ld_global_v8(const void *p, uint32_t w[8])
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

// An element of P's diagonal from S's before its rounding to s: what the rounding
// took away enters b S whole and c S S to first order.
__device__ __forceinline__ float with_diagonal(float x, float s, float diagonal, float alpha, float beta)
{
    return fmaf(diagonal - s, fmaf(2.0f * alpha, s, beta), x);
}

// What P's row is multiplied with after its product, so that its rounded diagonal
// counts as x.  (Below 1, 2^-12 of P, f16 is not exact to 2^-11.)
__device__ __forceinline__ float gain_of(float x)
{
    const float h = __half2float(__float2half_rn(x));
    return fabsf(h) >= 1.0f ? 1.0f + __fdividef(x - h, h) : 1.0f;
}

// Element i of sixteen, without an address.
__device__ __forceinline__ float pick(const float x[16], uint32_t i)
{
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = i & 8u ? x[q + 8] : x[q];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = i & 4u ? v[q + 4] : v[q];
#pragma unroll
    for (int q = 0; q < 2; ++q) v[q] = i & 2u ? v[q + 2] : v[q];
    return i & 1u ? v[1] : v[0];
}

// 16 sums of this lane's row `row`, columns col .. col+15, to a stored matrix.
// Rows past m are not written; columns are, up to the row's padding (their
// sums are zero: operands read as zeros there).  `prior`: the stored S there,
// `diagonal`: its diagonal in this row (kPoly).  Where the tile has a mirror image, the block goes out a second time,
// turned in the warp's staging area: lane l takes rows 16 (l / 16) on of column l % 16.
template <int OP>
__device__ __forceinline__ void store_stored(const Params &P, const Item &it, uint32_t row, uint32_t col,
                                             const uint32_t v[16], const uint32_t prior[8], float diagonal,
                                             float *stage, int lane)
{
    __half *mat = P.out + it.z * P.stride;
    const uint32_t d = row - col;
    const bool crosses = d < 16u && row < P.m;          // the diagonal passes through
    float x[16];
    if constexpr (OP == kPoly) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float2 s = unpack_f16(prior[q]);
            x[2 * q] = fmaf(P.alpha, __uint_as_float(v[2 * q]), P.beta * s.x);
            x[2 * q + 1] = fmaf(P.alpha, __uint_as_float(v[2 * q + 1]), P.beta * s.y);
        }
        if (crosses) {
            float t[16];
#pragma unroll
            for (int q = 0; q < 8; ++q) t[2 * q] = unpack_f16(prior[q]).x, t[2 * q + 1] = unpack_f16(prior[q]).y;
            const float y = with_diagonal(pick(x, d) + P.shift, pick(t, d), diagonal, P.alpha, P.beta);
#pragma unroll
            for (int q = 0; q < 16; ++q) x[q] = d == static_cast<uint32_t>(q) ? y : x[q];
            P.gain[it.z * P.side + row] = gain_of(y);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) x[q] = P.alpha * __uint_as_float(v[q]);
        if (OP == kGram && crosses) P.diag[it.z * P.side + row] = pick(x, d);
    }
    if (row < P.m) {
        uint32_t w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = pack_f16(x[2 * q], x[2 * q + 1]);
        st_global_v8(mat + static_cast<uint64_t>(row) * P.ld + col, w);
    }
    if (OP != kNext && it.mirror) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 16; ++q) stage[staged(lane, q)] = x[q];
        __syncwarp();
        const uint32_t c = lane & 15, r = lane & 16, row0 = row - lane + r;
        uint32_t w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = pack_f16(stage[staged(r + 2 * q, c)], stage[staged(r + 2 * q + 1, c)]);
        if (col + c < P.n && row0 < P.m) st_global_v8(mat + static_cast<uint64_t>(col + c) * P.ld + row0, w);
    }
}

// The raw words of a block's parameters.  Full blocks of aligned matrices: the 16
// of the lane's own row (bf16: eight words).  Others: one of every second row,
// in a word each, the lanes along two rows (see finish_block).
__device__ __forceinline__ void load_params(const Params &P, const void *ptr, uint32_t row, uint32_t col, int lane,
                                            uint32_t p[16])
{
    const uint16_t *in16 = static_cast<const uint16_t *>(ptr);
    const float *in32 = static_cast<const float *>(ptr);
    const bool bf16 = P.out_dtype == ASR_BF16;
    const uint64_t at = static_cast<uint64_t>(row) * P.out_ld + col;
    if (P.vec && P.n - col >= kBlock) {
        if (row >= P.m) return;
        if (bf16) {
            ld_global_v8(in16 + at, p);
        } else {
            ld_global_v8(in32 + at, p);
            ld_global_v8(in32 + at + 8, p + 8);
        }
        return;
    }
    const uint32_t c = lane & 15, first = row - lane + (lane >> 4);
    const uint64_t a = static_cast<uint64_t>(first) * P.out_ld + col + c;
#pragma unroll
    for (int q = 0; q < 16; ++q)
        p[q] = col + c >= P.n || first + 2 * q >= P.m ? 0u
               : bf16                                 ? in16[a + 2 * q * P.out_ld]
                                                      : __float_as_uint(in32[a + 2 * q * P.out_ld]);
}

__device__ __forceinline__ float param_value(const Params &P, const uint32_t p[16], int q)
{
    return P.out_dtype == ASR_BF16 ? (q & 1 ? bf16_hi(p[q >> 1]) : bf16_lo(p[q >> 1])) : __uint_as_float(p[q]);
}

// 16 finished values of one row to bf16 words; random bits of elements e on.
__device__ __forceinline__ void round16(const Params &P, const float x[16], uint64_t e, uint32_t w[8])
{
    if (P.rounding == ASR_ROUND_SR) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t r[8];
            if ((e & 3u) == 0) unit_words<true>(e, 8 * u, P.step, P.keys, r);
            else unit_words<false>(e, 8 * u, P.step, P.keys, r);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[4 * u + q] = sr_pack2<true>(x[8 * u + 2 * q], x[8 * u + 2 * q + 1], r[2 * q], r[2 * q + 1]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = pack_bf16(round_rne(x[2 * q]), round_rne(x[2 * q + 1]));
    }
}

// 16 sums x of row `row`, columns col .. col+15, to the caller's matrix.  Each
// lane finishes its own row; full blocks of aligned matrices are stored from
// there (`params`: what load_params gave; `next` is called when they are used up,
// and may load others), others pass through the staging area,
// in which the lanes lie along two rows at a time, whatever the row pitch: a
// lane that stores (and loads) its own row alone touches a sector an element.
template <int OP, typename Next>
__device__ __forceinline__ void finish_block(const Params &P, uint32_t z, uint32_t row, uint32_t col, float x[16],
                                             const uint32_t *params, const float *col_scale, float *stage, int lane,
                                             Next next)
{
    const uint32_t row0 = row - lane, live = P.n - col < 16 ? P.n - col : 16;
    const bool direct = P.vec && live == 16, bf16 = P.out_dtype == ASR_BF16, in = row < P.m;
    const Slot S = P.slot[z];
    uint16_t *out16 = static_cast<uint16_t *>(S.ptr);
    float *out32 = static_cast<float *>(S.ptr);
    const uint64_t at = static_cast<uint64_t>(row) * P.out_ld + col;
    const uint32_t c = lane & 15, r0 = lane >> 4;
    if constexpr (OP == kParam) {
        if (direct) {
#pragma unroll
            for (int q = 0; q < 16; ++q)
                x[q] = __fsub_rn(__fmul_rn(param_value(P, params, q), P.beta), __fmul_rn(P.alpha, x[q]));
        } else {
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 16; ++q)
                stage[staged(r0 + 2 * q, c)] = bf16 ? bf16_lo(params[q]) : __uint_as_float(params[q]);
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 16; ++q)
                x[q] = __fsub_rn(__fmul_rn(stage[staged(lane, q)], P.beta), __fmul_rn(P.alpha, x[q]));
        }
    }
    next();
    if constexpr (OP == kScaled) {
        // written by a kernel that may have been running when this one started: an
        // ordinary load (the read-only path is for what nobody writes meanwhile)
        const float rs = in ? P.row_scale[row] : 0.0f;
#pragma unroll
        for (int q = 0; q < 16; ++q) x[q] = __fmul_rn(__fmul_rn(x[q], rs), col_scale[q]);
    }
    if constexpr (OP == kOut) {
#pragma unroll
        for (int q = 0; q < 16; ++q) x[q] *= P.alpha;
    }
    uint32_t w[8];
    if (bf16) round16(P, x, S.base + static_cast<uint64_t>(row) * P.n + col, w);
    if (direct) {
        if (!in) return;
        if (bf16) {
            st_global_v8(out16 + at, w);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = __float_as_uint(x[8 * h + q]);
                st_global_v8(out32 + at + 8 * h, v);
            }
        }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 16; ++q)
        stage[staged(lane, q)] = bf16 ? __uint_as_float(w[q >> 1] >> ((q & 1) * 16)) : x[q];
    __syncwarp();
#pragma unroll 8
    for (uint32_t r = r0; r < 32; r += 2) {
        const uint64_t a = static_cast<uint64_t>(row0 + r) * P.out_ld + col + c;
        if (row0 + r < P.m && c < live) {
            const float v = stage[staged(r, c)];
            if (bf16) out16[a] = static_cast<uint16_t>(__float_as_uint(v));
            else out32[a] = v;
        }
    }
}

// Persistent over work items: cluster c takes items c, c + clusters, ...
// The roles and barriers are those of gemm_sr.cuh's pair kernel.
template <bool A_MN, bool B_MN, int OP>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_b_part, const __grid_constant__ Params P, uint64_t limit_ns)
{
    constexpr bool kSym = OP == kGram || OP == kPoly;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + kStages * kStageBytes;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s, int j) { return bars + 8u * (kStages + 2 * s + j); };
    auto acc_full = [&](int b) { return bars + 8u * (3 * kStages + b); };
    auto acc_empty = [&](int b) { return bars + 8u * (3 * kStages + kAccBufs + b); };
    const uint32_t drained = bars + 8u * (kBars - 1);
    const uint32_t tmem_slot = drained + 8u;
    const uint32_t *tmem_slot_ptr = reinterpret_cast<const uint32_t *>(smem_raw + (tmem_slot - raw));

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const uint32_t cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    const uint32_t items = P.wide + P.narrow;
    const uint32_t kblocks = (P.k + kBK - 1) / kBK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s, 0), 1);
            mbar_init(empty(s, 1), 1);
        }
        for (int b = 0; b < kAccBufs; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 2 * kEpi);
        }
        mbar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot_ptr, 0);
    // the operands may be the previous kernel's output
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ------------------------------------------------------- producer
        uint32_t g = 0, s = 0, phase = 0;
        bool wrapped = false, ok = true;
        const uint32_t full0 = peer_addr(full(0), 0);
        for (uint32_t t = cluster; ok && t < items; t += clusters) {
            const Item it = work_item<kSym>(P, t);
            const bool narrow = it.width != kTile;
            uint32_t ra = it.m0 + rank * 128, rb = it.n0 + rank * (it.width / 2);
            // rows wholly past the matrix: any rows do, their sums are not stored
            const bool a2 = ra + 64 < P.m, b2 = rb + 64 < P.n;
            if (ra >= P.m) ra = 0;
            if (rb >= P.n) rb = 0;
            // B in this CTA: half of the item's columns, or (stored across) blocks of 64 of them
            const uint32_t bytes_b = !narrow ? kHalfBytes : B_MN ? kHalfBytes / 2 : kHalfBytes / P.parts;
            const uint32_t bytes = 4 * (kHalfBytes + bytes_b);
            const int32_t z = static_cast<int32_t>(it.z);
            for (uint32_t kb = 0; kb < kblocks; ++kb, ++g) {
                const uint32_t bar = full0 + 8u * s;
                const uint32_t dst = base + s * kStageBytes;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (wrapped && !warp_wait(empty(s, j), phase ^ 1u, limit_ns)) {
                        ok = false;
                        break;
                    }
                    if (!elect_one()) continue;
                    if (j == 0 && leader) mbar_arrive_expect_tx(full(s), bytes);
                    const int32_t k0 = static_cast<int32_t>(kb * kBK + j * 64);
                    const uint32_t da = dst + j * kHalfBytes, db = dst + (2 + j) * kHalfBytes;
                    if (A_MN) {
                        tma_load_3d_pair(da, &map_a, static_cast<int32_t>(ra), k0, z, bar);
                        tma_load_3d_pair(da + 8192, &map_a, static_cast<int32_t>(a2 ? ra + 64 : ra), k0, z, bar);
                    } else {
                        tma_load_3d_pair(da, &map_a, k0, static_cast<int32_t>(ra), z, bar);
                    }
                    if (B_MN) {
                        tma_load_3d_pair(db, &map_b, static_cast<int32_t>(rb), k0, z, bar);
                        if (!narrow)
                            tma_load_3d_pair(db + 8192, &map_b, static_cast<int32_t>(b2 ? rb + 64 : rb), k0, z, bar);
                    } else {
                        tma_load_3d_pair(db, narrow ? &map_b_part : &map_b, k0, static_cast<int32_t>(rb), z, bar);
                    }
                }
                if (!ok) break;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1u;
                    wrapped = true;
                }
            }
        }
        for (uint32_t q = 0; q < static_cast<uint32_t>(kStages) && q < g; ++q) {
            const uint32_t last_use = (g - 1 - q) / kStages;
            for (int j = 0; j < 2; ++j) warp_wait(empty(static_cast<int>(q), j), last_use & 1u, limit_ns);
        }
    } else if (warp == 1 && leader) {
        // ------------------------------------------------------ MMA issuer
        uint32_t s = 0, phase = 0, i = 0;
        bool ok = true;
        constexpr uint32_t kDescWide = instr_desc(kTile, A_MN, B_MN);
        const uint32_t desc_narrow = instr_desc(kTile / P.parts, A_MN, B_MN);
        const uint64_t desc_a0 = operand_desc<A_MN>(base), desc_b0 = operand_desc<B_MN>(base + 2 * kHalfBytes);
        constexpr uint64_t kDescStage = kStageBytes >> 4, kDescHalf = kHalfBytes >> 4;
        constexpr uint64_t kStepA = A_MN ? 2048 >> 4 : 32 >> 4, kStepB = B_MN ? 2048 >> 4 : 32 >> 4;
        for (uint32_t t = cluster; ok && t < items; t += clusters) {
            const uint32_t idesc = t < P.wide ? kDescWide : desc_narrow;
            const int b = static_cast<int>(i % kAccBufs);
            const uint32_t ub = i++ / kAccBufs;
            if (ub > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait_cluster(acc_empty(b), (ub - 1) & 1u, limit_ns))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + static_cast<uint32_t>(b * kTile);
            for (uint32_t kb = 0; kb < kblocks; ++kb) {
                if (!warp_wait(full(s), phase, limit_ns)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint64_t ad = desc_a0 + s * kDescStage, bd = desc_b0 + s * kDescStage;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint64_t aj = ad + j * kDescHalf, bj = bd + j * kDescHalf;
                        mma_bf16_pair(d, aj, bj, idesc, (kb | j) != 0 ? 1u : 0u);
                        mma_bf16_pair(d, aj + kStepA, bj + kStepB, idesc, 1u);
                        mma_bf16_pair(d, aj + 2 * kStepA, bj + 2 * kStepB, idesc, 1u);
                        mma_bf16_pair(d, aj + 3 * kStepA, bj + 3 * kStepB, idesc, 1u);
                        mma_commit_pair(empty(s, j));
                    }
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (elect_one()) mma_commit_pair(acc_full(b));
            __syncwarp();
        }
        if (elect_one())
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drained)
                         : "memory");
        __syncwarp();
        warp_wait(drained, 0, limit_ns);
    } else if (warp >= 2) {
        // ------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const uint32_t group = static_cast<uint32_t>((warp - 2) / 4);
        float *stage = reinterpret_cast<float *>(smem_raw + (bars + kBarBytes - raw) + (warp - 2) * kWarpStage);
        uint32_t i = 0;
        for (uint32_t t = cluster; t < items; t += clusters) {
            const Item it = work_item<kSym>(P, t);
            const uint32_t row = it.m0 + rank * 128 + quarter * 32 + lane;
            const uint32_t ncols = it.n0 >= P.n ? 0 : P.n - it.n0 < it.width ? P.n - it.n0 : it.width;
            const uint32_t span = it.width / (kEpi / 4), c_lo = group * span;      // this warp's columns
            const uint32_t c_hi = ncols < c_lo + span ? ncols : c_lo + span;
            constexpr bool kStored = OP == kGram || OP == kPoly || OP == kNext;
            constexpr bool kGains = OP == kNext || OP == kOut || OP == kParam;
            const bool rows_in = row - lane < P.m;          // the same for the whole warp
            const uint32_t col0 = it.n0 + c_lo, cols = c_hi > c_lo && rows_in ? c_hi - c_lo : 0;
            uint32_t prior[OP == kPoly ? kSpan / 2 : 1];
            float diagonal = 0.0f, gain[kSpan / 32];
            // what the epilogue reads from memory, before it waits for the sums
            if constexpr (OP == kPoly) {
#pragma unroll
                for (int c = 0; c < kSpan; c += kBlock)
                    if (static_cast<uint32_t>(c) < cols && row < P.m)
                        ld_global_v8(P.aux + it.z * P.stride + static_cast<uint64_t>(row) * P.ld + col0 + c, prior + c / 2);
                if (!it.mirror && row < P.m) diagonal = P.diag[it.z * P.side + row];
            }
            // P's rows' gains: it is operand A where B is stored across (its rows are the
            // output's), else B (the output's columns)
            if constexpr (kGains) {
#pragma unroll
                for (int h = 0; h < kSpan / 32; ++h) {
                    if (B_MN) gain[h] = row < P.m ? P.gain[it.z * P.side + row] : 0.0f;
                    else gain[h] = 32u * h + lane < cols ? P.gain[it.z * P.side + col0 + 32 * h + lane] : 0.0f;
                }
            }
            uint32_t p[OP == kParam ? 16 : 1];
            if constexpr (OP == kParam)
                if (cols) load_params(P, P.slot[it.z].ptr, row, col0, lane, p);
            const int b = static_cast<int>(i % kAccBufs);
            if (!__all_sync(0xFFFFFFFFu, pair_wait(acc_full(b), (i++ / kAccBufs) & 1u, limit_ns))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t tq =
                tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(b * kTile) + c_lo;
#pragma unroll (kStored ? kSpan / kBlock : 1)
            for (int c = 0; c < kSpan; c += kBlock) {
                uint32_t v[16];
                const bool have = static_cast<uint32_t>(c) < cols;
                if (have) gemm::tmem_ld16(tq + c, v);
                if (c + kBlock == kSpan) {
                    // this warp has read its part of accumulator b
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(peer_addr(acc_empty(b), 0));
                }
                if (!have) continue;
                if constexpr (kGains) {
                    const float g = c < 32 ? gain[0] : gain[1];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        v[q] = __float_as_uint(__uint_as_float(v[q]) *
                                               (B_MN ? g : __shfl_sync(0xFFFFFFFFu, g, (c & 31) + q)));
                }
                if constexpr (kStored) {
                    store_stored<OP>(P, it, row, col0 + c, v, prior + (OP == kPoly ? c / 2 : 0), diagonal, stage, lane);
                } else {
                    float x[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) x[q] = __uint_as_float(v[q]);
                    finish_block<OP>(P, it.z, row, col0 + c, x, p, nullptr, stage, lane, [&]() {
                        if constexpr (OP == kParam)
                            if (static_cast<uint32_t>(c + kBlock) < cols)
                                load_params(P, P.slot[it.z].ptr, row, col0 + c + kBlock, lane, p);
                    });
                }
            }
        }
    }
    // ------------------------------------------------------------ cleanup
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
    }
}

// ------------------------------------------------------------------ host

// Shared-memory opt-in and resident pairs, set up for every form of the kernel
// on a device's first product, so that later ones may be captured into graphs.
std::mutex g_prod_mu;
bool g_prod_ready[kMaxDevices];
int g_prod_pairs[kMaxDevices];

// Loads a kernel, so that its first launch may be in a stream capture.
template <typename K>
cudaError_t load_kernel(K kernel)
{
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel);
}

// Launches a kernel that may start before the one ahead of it on the stream has
// ended; it waits for that itself (griddepcontrol.wait).
template <typename P>
asr_status launch_early(int kind, void (*kernel)(P), dim3 grid, unsigned threads, const P &params, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(kind);
}

// Opts a kernel of this shape in to its shared memory; *pairs: how many pairs of
// CTAs of it and of those before can be resident at once.
template <typename K>
cudaError_t setup_one(K kernel, int *pairs)
{
    int dev = 0, sms = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e == cudaSuccess && (*pairs == 0 || n < *pairs)) *pairs = n;
    return e;
}

asr_status setup(int *pairs)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return ASR_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_prod_mu);
    if (!g_prod_ready[dev]) {
        int n = 0;
        e = setup_one(product_kernel<false, false, kGram>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<true, true, kGram>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<false, false, kPoly>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<false, true, kNext>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<false, false, kNext>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<false, true, kOut>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<false, false, kOut>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<false, true, kParam>, &n);
        if (e == cudaSuccess) e = setup_one(product_kernel<false, false, kParam>, &n);
        if (e != cudaSuccess) return cuda_fail(e);
        if (n < 1) return cuda_fail(cudaErrorNotSupported);
        g_prod_pairs[dev] = n;
        g_prod_ready[dev] = true;
    }
    *pairs = g_prod_pairs[dev];
    return ASR_OK;
}

// A stack of row-major f16 matrices (rows x cols, ld elements between rows,
// stride between matrices) in boxes of box_rows x 64.
asr_status make_map(CUtensorMap *map, const void *ptr, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t stride,
                    uint64_t batch, uint32_t box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    asr_status st = gemm::encoder(&enc);
    if (st != ASR_OK) return st;
    const cuuint64_t dims[3] = {cols, rows, batch};
    const cuuint64_t strides[2] = {ld * 2, stride * 2};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ASR_OK : ASR_ERR_INVALID_VALUE;
}

// One row-major f16 matrix, in boxes of box_rows x 64.
asr_status make_map_2d(CUtensorMap *map, const void *ptr, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    asr_status st = gemm::encoder(&enc);
    if (st != ASR_OK) return st;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
    const cuuint32_t box[2] = {64, box_rows}, estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ASR_OK : ASR_ERR_INVALID_VALUE;
}

// One stored stack of matrices: f16, rows a multiple of 32 bytes apart.
struct Stored {
    __half *ptr;
    uint64_t rows, cols, ld, stride;
};

// Launches the product of a (m x k, or k x m where A_MN) and b (n x k, or
// k x n where B_MN); P's sizes and schedule are filled in here.
template <bool A_MN, bool B_MN, int OP>
asr_status launch(const Stored &a, const Stored &b, Params &P, cudaStream_t stream)
{
    int pairs = 0;
    asr_status st = setup(&pairs);
    if (st != ASR_OK) return st;
    P.m = static_cast<uint32_t>(A_MN ? a.cols : a.rows);
    P.k = static_cast<uint32_t>(A_MN ? a.rows : a.cols);
    P.n = static_cast<uint32_t>(B_MN ? b.cols : b.rows);
    P.tiles_m = (P.m + kTile - 1) / kTile;
    P.tiles_n = (P.n + kTile - 1) / kTile;
    constexpr bool kSym = OP == kGram || OP == kPoly;
    const uint64_t per = kSym ? static_cast<uint64_t>(P.tiles_m) * (P.tiles_m + 1) / 2
                              : static_cast<uint64_t>(P.tiles_m) * P.tiles_n;
    const uint64_t tiles = per * P.batch;
    if (tiles >= (1ull << 30)) return ASR_ERR_INVALID_VALUE;
    P.per_matrix = static_cast<uint32_t>(per);
    // as in gemm_sr.cuh: the tiles of a last round that is at most half full go
    // as halves, of one at most a quarter full as quarters
    const uint64_t rest = tiles % static_cast<uint64_t>(pairs);
    P.parts = 4 * rest <= static_cast<uint64_t>(pairs) ? 4 : 2 * rest <= static_cast<uint64_t>(pairs) ? 2 : 1;
    P.narrow = static_cast<uint32_t>(P.parts > 1 ? P.parts * rest : 0);
    P.wide = static_cast<uint32_t>(tiles - (P.narrow ? rest : 0));
    const uint64_t items = P.wide + static_cast<uint64_t>(P.narrow);
    const unsigned clusters = static_cast<unsigned>(items < static_cast<uint64_t>(pairs) ? items : pairs);
    CUtensorMap ma, mb, mbh;
    st = make_map(&ma, a.ptr, a.rows, a.cols, a.ld, a.stride, P.batch, A_MN ? 64 : 128);
    if (st == ASR_OK) st = make_map(&mb, b.ptr, b.rows, b.cols, b.ld, b.stride, P.batch, B_MN ? 64 : 128);
    if (st == ASR_OK) st = make_map(&mbh, b.ptr, b.rows, b.cols, b.ld, b.stride, P.batch, B_MN ? 64 : 128 / P.parts);
    if (st != ASR_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const uint64_t limit = kWaitLimitNs;
    cudaError_t e = cudaLaunchKernelEx(&cfg, product_kernel<A_MN, B_MN, OP>, ma, mb, mbh, P, limit);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(ASR_KERNEL_PRODUCT);
}

}  // namespace prod
