// int8_few.cuh -- the 8-bit integer product with few rows of A (tokens): what
// bounds it is reading B (the weight) once.  Included into asr.cu (inside its
// anonymous namespace), before int8.cuh.
//
// Two kernels:
//   few_dots_kernel    up to 4 tokens: dot products of four bytes (dp4a), 16
//                      instructions for a lane's four rows of 16 bytes;
//   few_rows_kernel    up to 128 tokens a pass: tcgen05.mma with the weight as
//                      the 128 rows of A.  The weight's bytes are widened to f16
//                      in registers and stored into tensor memory, from which
//                      the product reads them: through shared memory each byte
//                      would cost four bytes' traffic, and 23 bytes a cycle
//                      arrive.  The tokens are the B operand, from shared memory.
//                      mma.sync takes 2 cycles an SM for 256 bytes and 8 tokens
//                      (measured: 1.05 ns), so beyond 16 tokens it falls behind
//                      the memory: 40 us for 58.7 MB and 33 tokens.
// At most 1,024 products are added in binary32, which is exact; int32 then.
//
// Measured on a weight of 14,336 x 4,096 (58.7 MB, 8.6 us at the copy rate), with
// the launch: 1 token 14.4 us, 4 17.5, 16 20.5, 33 23.8, 64 26, 128 39; on one
// eight times as large 1 token 87 us (5.4 TB/s), 33 tokens 92.  What is left at
// the small end is latency: launch, first weights, quantiser, last sums.

namespace int8few {

constexpr int kRows = 128;                  // rows of B a piece
constexpr int kDotTokens = 4;               // up to this many, dot products
constexpr int kMaxTokens = 128;             // of a pass over B

struct Params {
    const __half *a;                        // tokens, m x k: widened, rows a multiple of 16 values apart and zero past k
    const int8_t *b;                        // weight, n x k
    const float *row_scale, *col_scale;
    void *c;
    int32_t *sums;                          // [row block][token][128], zero at the start
    uint32_t *counts;                       // [pass][row block], zero at the start
    uint64_t lda, ldb, ldc;
    uint32_t m, n, k, tiles, pieces;        // row blocks, pieces of each
    uint32_t each;                          // tokens a pass, a multiple of 16 (tcgen05)
    uint32_t b_vec;                         // rows of B in 16-byte aligned units
    uint32_t c_dtype, rounding, step;
    RoundKeys keys;
};

// Four 8-bit integers (bytes of w) to f16, exact: 1,024 + (x + 128), less 1,152.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// `count` bytes at p, at most 16, then zeros, of the bytes [first, end): four
// words of the five around them where all lie inside, else byte by byte.  (Weight
// of 1,001 x 2,049, rows at any address, 48 tokens: 37 us byte by byte, 14 so.)
__device__ __noinline__ uint4 load16_slow(const int8_t *p, uint32_t count, const int8_t *first, const int8_t *end)
{
    uint32_t w[5] = {0, 0, 0, 0, 0};
    const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
    const int8_t *a = p - shift;
    if (count >= 16 && a >= first && a + 20 <= end) {
#pragma unroll
        for (int q = 0; q < 5; ++q) w[q] = __ldg(reinterpret_cast<const uint32_t *>(a) + q);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = __funnelshift_r(w[q], w[q + 1], 8 * shift);
    } else {
        for (uint32_t q = 0; q < 16 && q < count; ++q) {
            const uint32_t v = static_cast<uint32_t>(static_cast<uint8_t>(p[q])) << (8 * (q & 3));
            if (q < 4) w[0] |= v;
            else if (q < 8) w[1] |= v;
            else if (q < 12) w[2] |= v;
            else w[3] |= v;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Stochastic rounding of the output of element e: out of line, so that the code
// around it, which runs once or twice a CTA and mostly rounds to nearest, stays
// short (inlined for 16 tokens, fetching it cost 2 us).
__device__ __noinline__ uint32_t round_stochastic(float y, uint64_t e, uint32_t step, const RoundKeys &K)
{
    uint32_t r[4];
    philox_q(e >> 2, step, K, r);
    const uint32_t sel = static_cast<uint32_t>(e & 3u);
    return round_sr(y, sel == 0 ? r[0] : sel == 1 ? r[1] : sel == 2 ? r[2] : r[3]);
}

// The outputs of one column (of scale cs) and COUNT tokens (`live` of them, of
// scales rs) from their integer sums.
template <int COUNT, typename P_>
__device__ __forceinline__ void store_outputs(const P_ &P, uint32_t token, uint32_t col, float cs, const float *rs,
                                              const int32_t sum[COUNT], uint32_t live)
{
    float y[COUNT];
#pragma unroll
    for (int q = 0; q < COUNT; ++q) y[q] = __fmul_rn(__fmul_rn(__int2float_rn(sum[q]), rs[q]), cs);
    const uint64_t dst = token * P.ldc + col;
    if (P.c_dtype == ASR_F32) {
#pragma unroll
        for (int q = 0; q < COUNT; ++q)
            if (static_cast<uint32_t>(q) < live) static_cast<float *>(P.c)[dst + q * P.ldc] = y[q];
    } else if (P.rounding == ASR_ROUND_SR) {
        const uint64_t e = static_cast<uint64_t>(token) * P.n + col;
#pragma unroll
        for (int q = 0; q < COUNT; ++q)
            if (static_cast<uint32_t>(q) < live)
                static_cast<uint16_t *>(P.c)[dst + q * P.ldc] =
                    static_cast<uint16_t>(round_stochastic(y[q], e + static_cast<uint64_t>(q) * P.n, P.step, P.keys));
    } else {
#pragma unroll
        for (int q = 0; q < COUNT; ++q)
            if (static_cast<uint32_t>(q) < live)
                static_cast<uint16_t *>(P.c)[dst + q * P.ldc] = static_cast<uint16_t>(round_rne(y[q]));
    }
}

// ------------------------------------------------------------ dot products
//
// A cluster of up to eight CTAs takes 64 rows of the weight, each CTA a share of
// K; a CTA has eight warps, two blocks of 32 rows and four quarters of every 512
// of K.  A lane holds 16 bytes of four rows at a time, a 512 ahead.  The tokens
// lie in shared memory as integers, quantised by every CTA for itself (the
// scale needs the whole row, a few KB out of L2) while its first weights are on
// their way; so there is one launch and no workspace.  With the quantiser in a
// launch of its own and the sums of shared row blocks through memory one token of
// 14,336 x 4,096 took 17.3 us, of which 8.6 us are the weight's bytes.
constexpr int kDotThreads = 256;
constexpr uint32_t kDotRows = 64;
constexpr uint32_t kSlab = 512;                 // K a round, a quarter of it a warp
constexpr uint32_t kDotSmem = 96 * 1024;        // room for the tokens
constexpr uint32_t kDotSplit = 8;

struct DotParams {
    const void *a;                              // tokens: f32, bf16, or (with row_scale) int8
    const int8_t *b;
    const float *row_scale, *col_scale;
    void *c;
    uint64_t lda, ldb, ldc;
    uint32_t m, n, k, share;                    // share: K of a CTA, a multiple of kSlab
    uint32_t a_dtype, a_vec, b_vec;
    uint32_t c_dtype, rounding, step;
    RoundKeys keys;
};

__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t addr)
{
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <bool QUANTISE>
__global__ void __launch_bounds__(kDotThreads, 2) few_dots_kernel(const __grid_constant__ DotParams P)
{
    extern __shared__ __align__(16) int8_t xs[];                            // [token][share]
    __shared__ int32_t sums[kDotTokens * kDotRows];
    __shared__ uint32_t part[kDotTokens][kDotThreads / 32];
    __shared__ float scales[kDotTokens];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t g = lane >> 2, t = lane & 3, quarter = warp & 3, block = warp >> 2;
    const uint32_t rank = gemm::cluster_rank();
    uint32_t split;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t n0 = blockIdx.x / split * kDotRows, k0 = rank * P.share;
    const uint32_t k1 = min(P.k, k0 + P.share);                             // at or below k0: nothing to add

    // the weight's rows g, g + 8, g + 16, g + 24 of the warp's 32, two 64-wide pieces a round
    const uint32_t row = n0 + block * 32 + g;
    const int8_t *src = P.b + row * P.ldb;
    const uint64_t ldb8 = 8 * P.ldb;
    uint4 w[2][4];
    auto weight = [&](uint32_t k, int i) {
        const uint32_t at = k + quarter * (kSlab / 4) + i * 64 + t * 16;
        if (P.b_vec && n0 + kDotRows <= P.n && k + kSlab <= k1) {           // the same for the whole CTA
#pragma unroll
            for (int r = 0; r < 4; ++r) w[i][r] = __ldcs(reinterpret_cast<const uint4 *>(src + r * ldb8 + at));
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                w[i][r] = make_uint4(0, 0, 0, 0);
                if (row + 8 * r < P.n && at < k1) {
                    if (P.b_vec && at + 16 <= k1) w[i][r] = __ldcs(reinterpret_cast<const uint4 *>(src + r * ldb8 + at));
                    else w[i][r] = load16_slow(src + r * ldb8 + at, k1 - at, P.b, P.b + (P.n - 1) * P.ldb + P.k);
                }
            }
        }
    };
    if (k0 < k1) {
        weight(k0, 0);
        weight(k0, 1);
    }
    for (uint32_t i = threadIdx.x; i < kDotTokens * kDotRows; i += kDotThreads) sums[i] = 0;

    // ---- the tokens
    if (QUANTISE) {
        uint32_t top[kDotTokens] = {};
        for (uint32_t c = threadIdx.x * 8; c < P.k; c += kDotThreads * 8) {
            const int live = P.k - c < 8 ? static_cast<int>(P.k - c) : 8;
#pragma unroll
            for (int q = 0; q < kDotTokens; ++q) {
                if (q >= static_cast<int>(P.m)) break;
                float x[8];
                muon::load8(P.a, P.a_dtype, q * P.lda + c, live, P.a_vec, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) top[q] = max(top[q], int8::absbits(x[e]));
            }
        }
#pragma unroll
        for (int q = 0; q < kDotTokens; ++q) {
            top[q] = __reduce_max_sync(0xFFFFFFFFu, top[q]);
            if (lane == 0) part[q][warp] = top[q];
        }
        __syncthreads();
        for (uint32_t q = 0; q < P.m; ++q) {
            uint32_t most = part[q][0];
#pragma unroll
            for (int e = 1; e < kDotThreads / 32; ++e) most = max(most, part[q][e]);
            const float amax = __uint_as_float(most);
            const int8::Levels L = int8::levels_of(amax);
            if (threadIdx.x == 0) scales[q] = __fdiv_rn(amax, 127.0f);
            for (uint32_t c = threadIdx.x * 8; c < P.share; c += kDotThreads * 8) {
                const int live = k0 + c >= P.k ? 0 : P.k - k0 - c < 8 ? static_cast<int>(P.k - k0 - c) : 8;
                float x[8];
                uint32_t e[4];
                muon::load8(P.a, P.a_dtype, q * P.lda + k0 + c, live, P.a_vec, x);
                int8::quantise8<false>(x, L, nullptr, e);
                *reinterpret_cast<uint2 *>(xs + q * P.share + c) = int8::bytes_of(e);
            }
        }
    } else {
        for (uint32_t q = 0; q < P.m; ++q) {
            const int8_t *a = static_cast<const int8_t *>(P.a) + q * P.lda + k0;
            for (uint32_t c = threadIdx.x; c < P.share; c += kDotThreads) xs[q * P.share + c] = k0 + c < P.k ? a[c] : 0;
            if (threadIdx.x == 0) scales[q] = P.row_scale[q];
        }
    }
    __syncthreads();

    int32_t dot[4][kDotTokens];                 // rows g + 8 r, this lane's part of K
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int q = 0; q < kDotTokens; ++q) dot[r][q] = 0;
    for (uint32_t k = k0; k < k1; k += kSlab) {
        const int8_t *x = xs + (k - k0) + quarter * (kSlab / 4) + t * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t v[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r][0] = w[i][r].x, v[r][1] = w[i][r].y, v[r][2] = w[i][r].z, v[r][3] = w[i][r].w;
            if (k + kSlab < k1) weight(k + kSlab, i);
#pragma unroll
            for (int q = 0; q < kDotTokens; ++q) {
                if (q > 0 && q >= static_cast<int>(P.m)) break;
                const int4 b = *reinterpret_cast<const int4 *>(x + q * P.share + i * 64);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dot[r][q] = __dp4a(static_cast<int>(v[r][0]), b.x, dot[r][q]);
                    dot[r][q] = __dp4a(static_cast<int>(v[r][1]), b.y, dot[r][q]);
                    dot[r][q] = __dp4a(static_cast<int>(v[r][2]), b.z, dot[r][q]);
                    dot[r][q] = __dp4a(static_cast<int>(v[r][3]), b.w, dot[r][q]);
                }
            }
        }
    }
    // the warps' sums, then the cluster's
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int q = 0; q < kDotTokens; ++q) {
            int32_t v = dot[r][q];
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
            if (t == static_cast<uint32_t>(q)) atomicAdd(sums + q * kDotRows + block * 32 + r * 8 + g, v);
        }
    gemm::cluster_sync();
    // each CTA finishes its share of the outputs: rows of the weight by rank
    const uint32_t each = kDotRows / split;
    for (uint32_t o = threadIdx.x; o < each * P.m; o += kDotThreads) {
        const uint32_t token = o / each, r = rank * each + o % each, col = n0 + r;
        int32_t sum = 0;
        for (uint32_t p = 0; p < split; ++p)
            sum += ld_cluster_s32(gemm::peer_addr(smem_addr(sums + token * kDotRows + r), p));
        if (col < P.n) store_outputs<1>(P, token, col, __ldg(P.col_scale + col), scales + token, &sum, 1);
    }
    gemm::cluster_sync();                       // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------------ tcgen05
//
// The work is cut into pieces, 128 rows of B by 128 of K, and every CTA (one on
// each SM) takes the same number of consecutive ones, across row blocks where
// they end: all SMs read the same share of the weight, whatever its shape.  The
// int32 sums of a row block that several CTAs share are added up in the
// workspace, and the CTA that completes the block's count of pieces writes its
// outputs.  Integer sums are the same in every order, and nobody waits for
// anybody.
//
// Warp 0 brings the tokens (two boxes of 64
// of K, 128-byte swizzle), warp 14 the weight's bytes (one box of 128 x 128,
// likewise), warp 1 issues the products, warps 2 to 5 read the sums (after 1,024
// of K or at the end of a row block) and finish them, warps 6 to 13 widen the
// weight: four of them, one for each quarter of the tensor memory's lanes, take
// every other piece.  A lane is a row: 128 bytes of it a piece, which become 64
// columns.  (Loading a lane's row straight into its registers, 32 rows a load
// instruction, left the memory at 4.2 TB/s, and at less with more loads in
// flight: a line's four sectors came in four requests.)
constexpr int kPiece = 128;
constexpr int kSets = 2;                        // of four widening warps
constexpr int kWidener = 6;                     // first widening warp
constexpr int kFewThreads = 32 * (kWidener + 4 * kSets + 1);
constexpr uint32_t kRing = 4;                   // pieces in tensor memory
constexpr uint32_t kRun = 1024 / kPiece;        // pieces added up in binary32
constexpr uint32_t kAccAt = kRing * kPiece / 2; // columns: the weight, then two accumulators
constexpr uint32_t kFewSmem = 226 * 1024;      // of the 227 KB, some static
constexpr uint32_t kMaxRing = 8;                // stages of a ring in shared memory
constexpr uint32_t kPieceBytes = kRows * kPiece;
constexpr int kBars = 4 * kMaxRing + 2 * kRing + 4 + 3;

// Shared memory for a pass of `each` tokens: rings of the tokens and of the
// weight's bytes, and the sums of a part longer than 1,024 of K.
struct FewShape {
    uint32_t x_ring, w_ring, x_bytes, sums_at, w_at, scales_at, bars_at, bytes;
};

__host__ __device__ constexpr FewShape few_shape(uint32_t each)
{
    FewShape f{};
    f.x_bytes = each * kPiece * 2;
    f.x_ring = each <= 64 ? 4 : 2;
    f.w_at = f.x_ring * f.x_bytes;              // 1,024-byte multiples: each is a multiple of 16
    const uint32_t left = kFewSmem - 16 - 1024 - f.w_at - each * (kRows + 4) * 4 - kBars * 8;
    f.w_ring = left / kPieceBytes < kMaxRing ? left / kPieceBytes : kMaxRing;
    f.sums_at = f.w_at + f.w_ring * kPieceBytes;
    f.scales_at = f.sums_at + each * kRows * 4;
    f.bars_at = f.scales_at + each * 4 * 4;
    f.bytes = 1024 + f.bars_at + kBars * 8 + 16;
    return f;
}

__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t v[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Where piece `at` of a CTA's stretch ends a run (its sums are read) and a part
// (of a row block); the same for every role.
struct Place {
    uint32_t tile, s, run, part;
    __device__ Place(uint32_t at, uint32_t pieces) : tile(at / pieces), s(at % pieces), run(0), part(0) {}
    __device__ bool ends_part(uint32_t at, uint32_t end, uint32_t pieces) const { return at + 1 == end || s + 1 == pieces; }
    __device__ bool ends_run(uint32_t at, uint32_t end, uint32_t pieces) const
    {
        return run + 1 == kRun || ends_part(at, end, pieces);
    }
    __device__ void next(uint32_t at, uint32_t end, uint32_t pieces)
    {
        const bool p = ends_part(at, end, pieces), r = ends_run(at, end, pieces);
        run = r ? 0 : run + 1;
        part = p ? 0 : part + 1;
        if (++s == pieces) {
            s = 0;
            ++tile;
        }
    }
};

__global__ void __launch_bounds__(kFewThreads, 1)
few_rows_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ Params P, uint64_t limit_ns)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ uint32_t done;
    const FewShape F = few_shape(P.each);
    const uint32_t raw = smem_addr(smem_raw), xs = (raw + 1023u) & ~1023u, ws = xs + F.w_at;
    const uint32_t each = P.each, box = each * 128;
    int32_t *sums = reinterpret_cast<int32_t *>(smem_raw + (xs - raw) + F.sums_at);     // [token][row]
    const uint32_t bars = xs + F.bars_at;
    auto full_x = [&](uint32_t i) { return bars + 8u * i; };
    auto empty_x = [&](uint32_t i) { return bars + 8u * (kMaxRing + i); };
    auto full_w = [&](uint32_t i) { return bars + 8u * (2 * kMaxRing + i); };
    auto empty_w = [&](uint32_t i) { return bars + 8u * (3 * kMaxRing + i); };
    auto full_a = [&](uint32_t i) { return bars + 8u * (4 * kMaxRing + i); };
    auto empty_a = [&](uint32_t i) { return bars + 8u * (4 * kMaxRing + kRing + i); };
    auto acc_full = [&](uint32_t i) { return bars + 8u * (4 * kMaxRing + 2 * kRing + i); };
    auto acc_empty = [&](uint32_t i) { return bars + 8u * (4 * kMaxRing + 2 * kRing + 2 + i); };
    const uint32_t added = bars + 8u * (kBars - 3), counted = added + 8u, drained = added + 16u, tmem_slot = drained + 8u;

    const int warp = prod::warp_index(), lane = threadIdx.x & 31;
    const uint32_t token0 = blockIdx.y * each, tokens = min(each, P.m - token0);
    const uint32_t total = P.tiles * P.pieces;
    const uint32_t first = static_cast<uint32_t>(static_cast<uint64_t>(total) * blockIdx.x / gridDim.x);
    const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(total) * (blockIdx.x + 1) / gridDim.x);

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kMaxRing; ++i) {
            mbar_init(full_x(i), 1);
            mbar_init(empty_x(i), 1);
            mbar_init(full_w(i), 1);
            mbar_init(empty_w(i), 4);
        }
        for (uint32_t i = 0; i < kRing; ++i) {
            mbar_init(full_a(i), 4);
            mbar_init(empty_a(i), 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_empty(i), 4);
        }
        mbar_init(added, 4);
        mbar_init(counted, 1);
        mbar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<const uint32_t *>(smem_raw + (tmem_slot - raw)), 0);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ------------------------------------------------------- tokens
        asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t s = first % P.pieces, i = 0;
        for (uint32_t at = first; at < end; ++at, ++i) {
            const uint32_t st = i % F.x_ring, use = i / F.x_ring;
            if (use > 0 && !prod::warp_wait(empty_x(st), (use - 1) & 1u, limit_ns)) break;
            const uint32_t dst = xs + st * F.x_bytes;
            if (prod::elect_one()) {
                mbar_arrive_expect_tx(full_x(st), F.x_bytes);
                gemm::tma_load_2d(dst, &map_x, static_cast<int32_t>(s * kPiece), static_cast<int32_t>(token0), full_x(st));
                gemm::tma_load_2d(dst + box, &map_x, static_cast<int32_t>(s * kPiece + 64), static_cast<int32_t>(token0),
                                  full_x(st));
            }
            __syncwarp();
            s = s + 1 == P.pieces ? 0 : s + 1;
        }
        for (uint32_t q = 0; q < F.x_ring && q < i; ++q) mbar_wait(full_x(q), ((i - 1 - q) / F.x_ring) & 1u, limit_ns);
    } else if (warp == kWidener + 4 * kSets) {
        // ------------------------------------------------------- weight
        // older than the previous kernel on the stream, so nothing to wait for
        if (P.b_vec) {
            uint32_t tile = first / P.pieces, s = first % P.pieces, i = 0;
            for (uint32_t at = first; at < end; ++at, ++i) {
                const uint32_t st = i % F.w_ring, use = i / F.w_ring;
                if (use > 0 && !prod::warp_wait(empty_w(st), (use - 1) & 1u, limit_ns)) break;
                if (prod::elect_one()) {
                    mbar_arrive_expect_tx(full_w(st), kPieceBytes);
                    gemm::tma_load_2d(ws + st * kPieceBytes, &map_w, static_cast<int32_t>(s * kPiece),
                                      static_cast<int32_t>(tile * kRows), full_w(st));
                }
                __syncwarp();
                if (++s == P.pieces) {
                    s = 0;
                    ++tile;
                }
            }
            for (uint32_t q = 0; q < F.w_ring && q < i; ++q)
                mbar_wait(full_w(q), ((i - 1 - q) / F.w_ring) & 1u, limit_ns);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- products
        const uint32_t idesc = (1u << 4) | ((each >> 3) << 17) | ((128u >> 4) << 24);
        Place pl(first, P.pieces);
        uint32_t i = 0, r = 0;
        bool ok = true;
        for (uint32_t at = first; ok && at < end; ++at, ++i) {
            const uint32_t st = i % kRing, sx = i % F.x_ring, b = r & 1u;
            if (pl.run == 0 && r >= 2) ok = prod::warp_wait(acc_empty(b), ((r >> 1) - 1) & 1u, limit_ns);
            ok = ok && prod::warp_wait(full_x(sx), (i / F.x_ring) & 1u, limit_ns) &&
                 prod::warp_wait(full_a(st), (i / kRing) & 1u, limit_ns);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + kAccAt + b * kMaxTokens, a = tmem + st * (kPiece / 2);
            const uint64_t x = gemm::smem_desc(xs + sx * F.x_bytes), x2 = gemm::smem_desc(xs + sx * F.x_bytes + box);
            const bool ends = pl.ends_run(at, end, P.pieces);
            if (prod::elect_one()) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    mma_from_tmem(d, a + q * 8, (q < 4 ? x : x2) + (q & 3) * 2, idesc, pl.run != 0 || q != 0);
                gemm::mma_commit(empty_a(st));
                gemm::mma_commit(empty_x(sx));
                if (ends) gemm::mma_commit(acc_full(b));
            }
            __syncwarp();
            if (ends) ++r;
            pl.next(at, end, P.pieces);
        }
        if (prod::elect_one()) gemm::mma_commit(drained);
        __syncwarp();
        prod::warp_wait(drained, 0, limit_ns);
    } else if (warp >= 2 && warp < 6) {
        // ------------------------------------------------------- sums
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const uint32_t quarter = warp & 3u, row = quarter * 32 + lane;
        // the tokens' scales at hand (each warp writes and reads its own copy), zero past the last
        float *rs = reinterpret_cast<float *>(smem_raw + (xs - raw) + F.scales_at) + quarter * each;
        for (uint32_t q = lane; q < each; q += 32) rs[q] = q < tokens ? P.row_scale[token0 + q] : 0.0f;
        __syncwarp();
        Place pl(first, P.pieces);
        uint32_t r = 0, shares = 0;
        bool held = false;                              // sums of this part in shared memory already
        for (uint32_t at = first; at < end; ++at) {
            if (pl.ends_run(at, end, P.pieces)) {
                const uint32_t b = r & 1u, out = pl.tile * kRows + row;
                const float cs = out < P.n ? __ldg(P.col_scale + out) : 0.0f;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_full(b), (r >> 1) & 1u, limit_ns))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const bool last = pl.ends_part(at, end, P.pieces), whole = last && pl.part + 1 == P.pieces;
                const uint32_t tq = tmem + ((quarter * 32) << 16) + kAccAt + b * kMaxTokens, col = out;
                int32_t *shared = P.sums + (static_cast<uint64_t>(pl.tile) * P.m + token0) * kRows + row;
#pragma unroll 1
                for (uint32_t c = 0; c < tokens; c += 16) {
                    uint32_t v[16];
                    int32_t sum[16];
                    gemm::tmem_ld16(tq + c, v);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        sum[q] = __float2int_rn(__uint_as_float(v[q]));
                        if (held) sum[q] += sums[(c + q) * kRows + row];
                    }
                    if (!last) {
#pragma unroll
                        for (int q = 0; q < 16; ++q) sums[(c + q) * kRows + row] = sum[q];
                    } else if (!whole) {
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (c + q < tokens) atomicAdd(shared + (c + q) * kRows, sum[q]);
                    } else if (col < P.n) {
                        store_outputs<16>(P, token0 + c, col, cs, rs + c, sum, tokens - c);
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty(b));
                held = !last;
                if (last && !whole) {
                    // the last CTA to add its part finishes the row block
                    __threadfence();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(added);
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(added, shares & 1u, limit_ns))) break;
                    if (threadIdx.x == 64) {
                        const uint32_t run = pl.part + 1;
                        done = atomicAdd(P.counts + blockIdx.y * P.tiles + pl.tile, run) + run;
                        mbar_arrive(counted);
                    }
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(counted, shares & 1u, limit_ns))) break;
                    ++shares;
                    if (done == P.pieces) {
                        __threadfence();
                        // 64 tokens' loads at a time in flight
#pragma unroll 1
                        for (uint32_t c = 0; c < tokens && col < P.n; c += 64) {
                            int32_t sum[64];
#pragma unroll
                            for (int h = 0; h < 4; ++h)
                                if (c + 16 * h < tokens) {
#pragma unroll
                                    for (int q = 0; q < 16; ++q)
                                        sum[16 * h + q] = __ldcg(shared + min(c + 16 * h + q, tokens - 1) * kRows);
                                }
#pragma unroll
                            for (int h = 0; h < 4; ++h)
                                if (c + 16 * h < tokens)
                                    store_outputs<16>(P, token0 + c + 16 * h, col, cs, rs + c + 16 * h, sum + 16 * h,
                                                      tokens - c - 16 * h);
                        }
                    }
                }
                ++r;
            }
            pl.next(at, end, P.pieces);
        }
    } else if (warp >= kWidener && warp < kWidener + 4 * kSets) {
        // ------------------------------------------------------- widening
        const uint32_t quarter = warp & 3u, row = quarter * 32 + lane;
        const unsigned char *mine = smem_raw + (ws - raw) + row * kPiece;
        uint32_t i = (warp - kWidener) >> 2;
        for (uint32_t at = first + i; at < end; at += kSets, i += kSets) {
            uint4 w[8];
            if (P.b_vec) {
                const uint32_t sw = i % F.w_ring;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(full_w(sw), (i / F.w_ring) & 1u, limit_ns))) break;
                // 16-byte unit q of a row lies at q ^ (row & 7) of its 128 bytes
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    w[q] = *reinterpret_cast<const uint4 *>(mine + sw * kPieceBytes + ((q ^ (row & 7)) << 4));
            } else {
                const uint32_t n = at / P.pieces * kRows + row, k = at % P.pieces * kPiece;
                for (int q = 0; q < 8; ++q)
                    w[q] = n < P.n && k + 16 * q < P.k
                               ? load16_slow(P.b + n * P.ldb + k + 16 * q, P.k - k - 16 * q, P.b,
                                             P.b + (P.n - 1) * P.ldb + P.k)
                               : make_uint4(0, 0, 0, 0);
            }
            const uint32_t st = i % kRing, use = i / kRing;
            if (use > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(empty_a(st), (use - 1) & 1u, limit_ns))) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t dst = tmem + ((quarter * 32) << 16) + st * (kPiece / 2);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t f[16];
                const uint32_t u[8] = {w[2 * h].x, w[2 * h].y, w[2 * h].z, w[2 * h].w,
                                       w[2 * h + 1].x, w[2 * h + 1].y, w[2 * h + 1].z, w[2 * h + 1].w};
#pragma unroll
                for (int q = 0; q < 8; ++q) widen4(u[q], f[2 * q], f[2 * q + 1]);
                tmem_st16(dst + 16 * h, f);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full_a(st));
                if (P.b_vec) mbar_arrive(empty_w(i % F.w_ring));
            }
        }
    }
    // ------------------------------------------------------------ cleanup
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ------------------------------------------------------------------ host

std::mutex g_few_mu;
int g_few_sms[kMaxDevices];

asr_status setup(int *sms)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return ASR_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_few_mu);
    if (!g_few_sms[dev]) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(few_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(few_dots_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDotSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(few_dots_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDotSmem);
        if (e != cudaSuccess) return cuda_fail(e);
        g_few_sms[dev] = n;
    }
    *sms = g_few_sms[dev];
    return ASR_OK;
}

// A row-major matrix of bytes in boxes of 128 x 128.
asr_status make_map_int8(CUtensorMap *map, const int8_t *ptr, uint64_t rows, uint64_t cols, uint64_t ld)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    const asr_status st = gemm::encoder(&enc);
    if (st != ASR_OK) return st;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld};
    const cuuint32_t box[2] = {kPiece, kRows}, estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(ptr), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ASR_OK : ASR_ERR_INVALID_VALUE;
}

// CTAs that share a row block's K: enough to give every SM one, none of them
// less than a round.
uint32_t dot_split(uint64_t n, uint64_t k)
{
    const uint64_t tiles = (n + kDotRows - 1) / kDotRows, rounds = (k + kSlab - 1) / kSlab;
    uint32_t split = 1;
    while (split < kDotSplit && 2 * split <= rounds && tiles * split < 152) split *= 2;
    return split;
}

uint64_t dot_share(uint64_t n, uint64_t k)
{
    const uint32_t split = dot_split(n, k);
    return ((k + kSlab - 1) / kSlab + split - 1) / split * kSlab;
}

// Whether the dot products' kernel takes m tokens: their shares have to fit its shared memory.
bool dots(uint64_t m, uint64_t n, uint64_t k) { return m <= kDotTokens && m * dot_share(n, k) <= kDotSmem; }

asr_status run_dots(DotParams &P, bool quantise, cudaStream_t stream)
{
    int sms = 0;
    const asr_status st = setup(&sms);
    if (st != ASR_OK) return st;
    const uint32_t split = dot_split(P.n, P.k);
    P.share = static_cast<uint32_t>(dot_share(P.n, P.k));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((P.n + kDotRows - 1) / kDotRows * split, 1, 1);
    cfg.blockDim = dim3(kDotThreads, 1, 1);
    cfg.dynamicSmemBytes = P.m * P.share;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = quantise ? cudaLaunchKernelEx(&cfg, few_dots_kernel<true>, P)
                                   : cudaLaunchKernelEx(&cfg, few_dots_kernel<false>, P);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(ASR_KERNEL_INT8_FEW_ROWS);
}

uint32_t passes(uint64_t m) { return static_cast<uint32_t>((m + kMaxTokens - 1) / kMaxTokens); }

// P.m tokens in passes of equal size, at most kMaxTokens each.
asr_status run(Params &P, cudaStream_t stream)
{
    int sms = 0;
    asr_status st = setup(&sms);
    if (st != ASR_OK) return st;
    P.tiles = (P.n + kRows - 1) / kRows;
    P.pieces = (P.k + kPiece - 1) / kPiece;
    const uint64_t total = static_cast<uint64_t>(P.tiles) * P.pieces;
    if (total >= (1ull << 31)) return ASR_ERR_INVALID_VALUE;
    const uint32_t p = passes(P.m);
    P.each = ((P.m + p - 1) / p + 15) / 16 * 16;
    CUtensorMap map, map_w;
    st = prod::make_map_2d(&map, P.a, P.m, P.k, P.lda, P.each);
    if (st == ASR_OK && P.b_vec) st = make_map_int8(&map_w, P.b, P.n, P.k, P.ldb);
    if (st != ASR_OK) return st;
    if (!P.b_vec) map_w = map;                  // not read
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(total < static_cast<uint64_t>(sms) ? static_cast<uint32_t>(total) : static_cast<uint32_t>(sms),
                       (P.m + P.each - 1) / P.each, 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = few_shape(P.each).bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const uint64_t limit = kWaitLimitNs;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, few_rows_kernel, map, map_w, P, limit);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(ASR_KERNEL_INT8_FEW_ROWS);
}

}  // namespace int8few
