// skinny.cuh -- the whole Newton-Schulz iteration (or Muon step) of matrices
// whose smaller side is at most 128 in one launch, with X in shared memory from
// the gradient to the result.  Included into asr.cu (inside its anonymous
// namespace), in muon.cuh's namespace muon, before its host side.
//
// A cluster of C CTAs holds a matrix, X with its smaller side as rows (a tall
// matrix is turned as it is loaded): each CTA 128 rows (zeros past m) of up to
// 512 columns, f16, in blocks of 64 columns whose 128-byte rows are swizzled as
// the tensor cores read them -- the same bytes serve as K-major operands of
// X X^T and as the MN-major operand of P X.  A step:
//   - the CTA's part of S = X X^T in tensor memory (binary32); with C > 1 the
//     parts meet in distributed shared memory: each CTA adds up 128 / C rows and
//     writes them, f16, into every CTA's S;
//   - S S and P = a I + b S + c S S in every CTA (8 products of 128 x 128 x 16);
//   - X' = P X over X.
// Number format, formulas and order of the epilogue's operations are those of
// the products in memory (muon.cuh).  Those take three launches a step of 4.5 us
// each however small the matrix is: 70 us for 96 x 160, against 28 us here (both
// with the host's part).
// What bounds it is latency: a chain of MMA, tensor memory read and shared memory
// write three times a step.

constexpr int kSkinnyThreads = 256;
constexpr uint32_t kSkinnyRows = 128;
constexpr uint32_t kSkinnyCols = 512;           // of a CTA
constexpr uint32_t kSkinnyClusters = 8;         // CTAs of a cluster, at most
constexpr uint32_t kColBlock = kSkinnyRows * 128;   // bytes of 64 columns
constexpr uint32_t kSkinnyX = kSkinnyCols / 64 * kColBlock;
constexpr uint32_t kSkinnyS = 2 * kColBlock;
// X, S, P and, from P on, the CTA's part of S in binary32 (P is dead then)
constexpr uint32_t kSkinnySmem = 1024 + kSkinnyX + kSkinnyS + kSkinnyRows * kSkinnyRows * 4;

bool skinny_fits(uint64_t rows, uint64_t cols)
{
    const uint64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    return m <= kSkinnyRows && n <= static_cast<uint64_t>(kSkinnyCols) * kSkinnyClusters;
}

struct SkinnyParams {
    PrepParams in;                              // partial, count, out unused
    prod::Params out;                           // the caller's output
    uint32_t m, n, tall, share;                 // smaller and larger side; columns of X a CTA
    uint32_t steps;
    float a, b, c;
};

// Byte offset of X, S or P's row r, column c.
__device__ __forceinline__ uint32_t tile_at(uint32_t r, uint32_t c)
{
    return (c >> 6) * kColBlock + r * 128 + ((((c >> 3) & 7u) ^ (r & 7u)) << 4) + (c & 7u) * 2;
}

// Word offset of 16 bytes (columns 4 q on) of row r of a part of S.
__device__ __forceinline__ uint32_t part_at(uint32_t r, uint32_t q) { return r * 128 + ((q ^ (r & 31u)) << 2); }

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float pick_word(const uint32_t v[16], uint32_t i)
{
    float x[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) x[q] = __uint_as_float(v[q]);
    return prod::pick(x, i);
}

// Descriptor of 64-column blocks read across (their rows are the contraction).
__device__ __forceinline__ uint64_t across_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(kColBlock >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

template <bool MUON>
__global__ void __launch_bounds__(kSkinnyThreads, 1)
skinny_kernel(const __grid_constant__ SkinnyParams P, uint64_t limit_ns)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bar_mem;
    __shared__ uint32_t tmem_slot;
    __shared__ Squares squares[8], total;
    __shared__ float diagonal[kSkinnyRows], gain[kSkinnyRows];      // S's before its rounding; of P's rows
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char *xs = smem_raw + (base - raw), *ss = xs + kSkinnyX, *ps = ss + kSkinnyS;
    float *part = reinterpret_cast<float *>(ps);
    const uint32_t xa = base, sa = base + kSkinnyX, pa = sa + kSkinnyS, bar = smem_addr(&bar_mem);

    const int warp = prod::warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = gemm::cluster_rank(), quarter = warp & 3, half = warp >> 2;
    uint32_t ctas;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const uint32_t z = blockIdx.x / ctas, col0 = rank * P.share;
    const uint32_t cols = P.n > col0 ? min(P.share, P.n - col0) : 0;        // this CTA's columns of X
    const Matrix M = P.in.m[z];

    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    for (uint32_t i = threadIdx.x; i < P.share / 64 * kColBlock / 16; i += kSkinnyThreads)
        reinterpret_cast<uint4 *>(xs)[i] = make_uint4(0, 0, 0, 0);

    // ---- the gradient, eight elements of a row of it at a time: the part that
    // becomes this CTA's columns (rows, of a tall matrix)
    const uint32_t lines = P.tall ? cols : P.m, first = P.tall ? col0 : 0;          // rows of the source
    const uint32_t from = P.tall ? 0 : col0, width = P.tall ? P.m : cols, units = (width + 7) / 8;
    auto visit = [&](auto f) {
        for (uint32_t u = threadIdx.x; u < lines * units; u += kSkinnyThreads) {
            const uint32_t line = u / units, c = (u - line * units) * 8;
            const int live = width - c < 8 ? static_cast<int>(width - c) : 8;
            const uint64_t row = first + line, col = from + c;
            float x[8];
            load8(M.src, P.in.src_dtype, row * P.in.src_ld + col, live, P.in.vec, x);
            f(line, c, live, row * P.in.cols + col, x);
        }
    };
    Squares sum = {0.0f, 0.0f};
    visit([&](uint32_t, uint32_t, int live, uint64_t at, float x[8]) {
        if (MUON) {
            float m[8];
            load8(M.momentum, ASR_F32, at, live, P.in.vec, m);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                m[q] = __fadd_rn(m[q], __fmul_rn(P.in.omu, __fsub_rn(x[q], m[q])));
                x[q] = update_of(P.in, x[q], m[q]);
            }
            if (P.in.vec && live == 8) {
                reinterpret_cast<float4 *>(M.momentum + at)[0] = make_float4(m[0], m[1], m[2], m[3]);
                reinterpret_cast<float4 *>(M.momentum + at)[1] = make_float4(m[4], m[5], m[6], m[7]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < live) M.momentum[at + q] = m[q];
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) add_square(sum, x[q]);
    });
    add_warp(sum);
    if (lane == 0) squares[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) add_squares(sum, squares[w].plain, squares[w].raised);
        total = sum;
    }
    gemm::cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_slot, 0);
    sum = {0.0f, 0.0f};
    for (uint32_t r = 0; r < ctas; ++r) {
        float v, w;
        const uint32_t at = gemm::peer_addr(smem_addr(&total), r);
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(at + 4) : "memory");
        add_squares(sum, v, w);
    }
    const float f = factor_of(sum, P.in.eps);
    visit([&](uint32_t line, uint32_t c, int live, uint64_t at, float x[8]) {
        if (MUON) {
            float m[8];
            load8(M.momentum, ASR_F32, at, live, P.in.vec, m);
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = update_of(P.in, x[q], m[q]);
        }
        if (P.tall) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < live) *reinterpret_cast<__half *>(xs + tile_at(c + q, line)) = __float2half_rn(x[q] * f);
        } else {
            *reinterpret_cast<uint4 *>(xs + tile_at(line, c)) =
                make_uint4(prod::pack_f16(x[0] * f, x[1] * f), prod::pack_f16(x[2] * f, x[3] * f),
                           prod::pack_f16(x[4] * f, x[5] * f), prod::pack_f16(x[6] * f, x[7] * f));
        }
    });
    asm volatile("fence.proxy.async;" ::: "memory");
    __syncthreads();

    // ---- the iteration
    constexpr float kDown = 1.0f / kStore;
    constexpr uint32_t kDesc128 = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t row = quarter * 32 + lane, tq = tmem + ((quarter * 32) << 16);
    uint32_t phase = 0;
    // the sums are in tensor memory (a wait that gives up has raised the error bit, and the kernel runs on)
    auto done = [&]() {
        mbar_wait(bar, phase, limit_ns);
        __syncwarp();
        phase ^= 1u;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    };
    // what was written to shared memory and read from tensor memory, before the next products
    auto settle = [&](bool cluster) {
        asm volatile("fence.proxy.async;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        if (cluster) gemm::cluster_sync();
        else __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    };
    for (uint32_t step = 0; step < P.steps; ++step) {
        const bool last = step + 1 == P.steps;
        // S, this CTA's part
        if (warp == 0) {
            if (prod::elect_one()) {
                for (uint32_t b = 0; b < P.share / 64; ++b) {
                    const uint64_t d = gemm::smem_desc(xa + b * kColBlock);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f16(tmem, d + 2 * k, d + 2 * k, kDesc128, (b | k) != 0);
                }
                gemm::mma_commit(bar);
            }
            __syncwarp();
        }
        done();
#pragma unroll 1
        for (uint32_t c = half * 64; c < half * 64 + 64; c += 16) {
            uint32_t v[16];
            gemm::tmem_ld16(tq + c, v);
            if (ctas == 1) {
                uint32_t w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    w[q] = prod::pack_f16(kDown * __uint_as_float(v[2 * q]), kDown * __uint_as_float(v[2 * q + 1]));
                *reinterpret_cast<uint4 *>(ss + tile_at(row, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(ss + tile_at(row, c + 8)) = make_uint4(w[4], w[5], w[6], w[7]);
                if (row - c < 16u) diagonal[row] = kDown * pick_word(v, row - c);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4 *>(part + part_at(row, c / 4 + q)) =
                        make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
        }
        if (ctas > 1) {
            settle(true);
            const uint32_t rows = kSkinnyRows / ctas;
            for (uint32_t i = threadIdx.x; i < rows * 32; i += kSkinnyThreads) {
                const uint32_t r = rank * rows + i / 32, q = i % 32, at = pa + part_at(r, q) * 4;
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (uint32_t p = 0; p < ctas; ++p) {
                    const float4 v = ld_cluster_f4(gemm::peer_addr(at, p));
                    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                }
                const uint32_t lo = prod::pack_f16(kDown * s.x, kDown * s.y), hi = prod::pack_f16(kDown * s.z, kDown * s.w);
                for (uint32_t p = 0; p < ctas; ++p) st_cluster_v2(gemm::peer_addr(sa + tile_at(r, 4 * q), p), lo, hi);
                if (r / 4 == q) {
                    const float d = kDown * ((r & 3) == 0 ? s.x : (r & 3) == 1 ? s.y : (r & 3) == 2 ? s.z : s.w);
                    for (uint32_t p = 0; p < ctas; ++p) st_cluster_f32(gemm::peer_addr(smem_addr(diagonal + r), p), d);
                }
            }
            settle(true);
        } else {
            settle(false);
        }
        // S S
        if (warp == 0) {
            if (prod::elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t d = gemm::smem_desc(sa + (k >> 2) * kColBlock) + 2 * (k & 3);
                    mma_f16(tmem, d, d, kDesc128, k != 0);
                }
                gemm::mma_commit(bar);
            }
            __syncwarp();
        }
        // P's diagonal but for c S S
        const float t = __half2float(*reinterpret_cast<const __half *>(ss + tile_at(row, row)));
        const float rest = prod::with_diagonal(fmaf(P.b, t, P.a * kStore), t, diagonal[row], P.c * kDown, P.b);
        done();
#pragma unroll 1
        for (uint32_t c = half * 64; c < half * 64 + 64; c += 16) {
            uint32_t v[16], w[8];
            gemm::tmem_ld16(tq + c, v);
            const uint4 lo = *reinterpret_cast<const uint4 *>(ss + tile_at(row, c));
            const uint4 hi = *reinterpret_cast<const uint4 *>(ss + tile_at(row, c + 8));
            const uint32_t s[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float2 t = prod::unpack_f16(s[q]);
                const float x = fmaf(P.c * kDown, __uint_as_float(v[2 * q]), P.b * t.x);
                const float y = fmaf(P.c * kDown, __uint_as_float(v[2 * q + 1]), P.b * t.y);
                w[q] = prod::pack_f16(x, y);
            }
            *reinterpret_cast<uint4 *>(ps + tile_at(row, c)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(ps + tile_at(row, c + 8)) = make_uint4(w[4], w[5], w[6], w[7]);
            if (row - c < 16u) {
                const float x = fmaf(P.c * kDown, pick_word(v, row - c), rest);
                *reinterpret_cast<__half *>(ps + tile_at(row, row)) = __float2half_rn(x);
                gain[row] = prod::gain_of(x);
            }
        }
        settle(false);
        const float down = kDown * gain[row];
        // P X, 256 columns an instruction
        if (warp == 0) {
            if (prod::elect_one()) {
                for (uint32_t c = 0; c < P.share; c += 256) {
                    const uint32_t wide = P.share - c < 256 ? P.share - c : 256;
                    const uint32_t idesc = (1u << 4) | (1u << 16) | ((wide >> 3) << 17) | ((128u >> 4) << 24);
                    const uint64_t bd = across_desc(xa + c / 64 * kColBlock);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16(tmem + c, gemm::smem_desc(pa + (k >> 2) * kColBlock) + 2 * (k & 3), bd + k * (2048 >> 4),
                                idesc, k != 0);
                }
                gemm::mma_commit(bar);
            }
            __syncwarp();
        }
        done();
        if (!last) {
#pragma unroll 1
            for (uint32_t c = half * 16; c < P.share; c += 32) {
                uint32_t v[16], w[8];
                gemm::tmem_ld16(tq + c, v);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    w[q] = prod::pack_f16(down * __uint_as_float(v[2 * q]), down * __uint_as_float(v[2 * q + 1]));
                *reinterpret_cast<uint4 *>(xs + tile_at(row, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(xs + tile_at(row, c + 8)) = make_uint4(w[4], w[5], w[6], w[7]);
            }
            settle(false);
        }
    }

    // ---- the result, from tensor memory
    constexpr int OP = MUON ? prod::kParam : prod::kOut;
    float *stage = reinterpret_cast<float *>(ss) + warp * (prod::kWarpStage / 4);       // S is dead
#pragma unroll 1
    for (uint32_t c = half * 16; c < cols; c += 32) {
        uint32_t v[16], p[16];
        float x[16];
        gemm::tmem_ld16(tq + c, v);
#pragma unroll
        for (int q = 0; q < 16; ++q) x[q] = __uint_as_float(v[q]) * gain[row];
        if (!P.tall) {
            if (row - lane < P.m) {
                if (MUON) prod::load_params(P.out, P.out.slot[z].ptr, row, col0 + c, lane, p);
                prod::finish_block<OP>(P.out, z, row, col0 + c, x, p, nullptr, stage, lane, []() {});
            }
        } else if (row < P.m) {
            // column `row` of the caller's matrix, a warp 32 of them: rows c .. c+15 of this CTA's
            const prod::Slot S = P.out.slot[z];
#pragma unroll 1
            for (uint32_t q = 0; q < 16 && c + q < cols; ++q) {
                float y = 0.0f;
#pragma unroll
                for (uint32_t e = 0; e < 16; ++e) y = e == q ? x[e] : y;
                const uint64_t r = col0 + c + q, at = r * P.out.out_ld + row;
                uint16_t *p16 = static_cast<uint16_t *>(S.ptr) + at;
                float *p32 = static_cast<float *>(S.ptr) + at;
                const bool bf16 = P.out.out_dtype == ASR_BF16;
                if (MUON) y = __fsub_rn(__fmul_rn(bf16 ? bf16_lo(*p16) : *p32, P.out.beta), __fmul_rn(P.out.alpha, y));
                else y *= P.out.alpha;
                if (!bf16) {
                    *p32 = y;
                } else if (P.out.rounding == ASR_ROUND_SR) {
                    const uint64_t e = S.base + r * P.in.cols + row;
                    uint32_t w[4];
                    philox_q(e >> 2, P.out.step, P.out.keys, w);
                    const uint32_t sel = static_cast<uint32_t>(e & 3u);
                    *p16 = static_cast<uint16_t>(round_sr(y, sel == 0 ? w[0] : sel == 1 ? w[1] : sel == 2 ? w[2] : w[3]));
                } else {
                    *p16 = static_cast<uint16_t>(round_rne(y));
                }
            }
        }
        __syncwarp();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}
