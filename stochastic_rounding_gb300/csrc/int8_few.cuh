// int8_few.cuh -- the 8-bit integer product with few rows of A (tokens): what
// bounds it is reading B (the weight) once.  Included into asr.cu (inside its
// anonymous namespace), before int8.cuh.
//
// A CTA takes 128 rows of B and a share of K; the CTAs of a cluster hold the
// shares of one 128-row block and add their int32 sums through distributed
// shared memory, so that a weight of few rows still occupies the GPU.  Eight
// warps: four blocks of 32 rows, two halves of every 512-wide slab of K.  A
// warp streams its rows from global memory straight into registers, 16 bytes a
// lane and row, four 64-wide pieces (8 KB) ahead, and widens them to f16 there.
// Tokens are widened into shared memory, a slab ahead.
//
// The products are mma.sync m16n8k16 (f16, binary32 sums): B's rows are the 16,
// tokens the 8.  At up to 64 tokens the tensor work stays below the time that
// the weight's bytes take (64 tokens: 128 operations a byte, 0.87 PFLOP/s at
// the measured copy rate), and with operands in registers the weight never
// passes through shared memory, which tcgen05 would need.  The order of K
// inside a product is free, so a lane's 16 contiguous bytes serve as its
// fragments of four consecutive steps.  Sums of at most 1,024 products are
// exact in binary32 and go to int32 then.

namespace int8few {

constexpr int kThreads = 256;
constexpr int kRows = 128;                  // rows of B a CTA
constexpr int kSlab = 512;                  // K a slab, half of it a warp
constexpr int kPitch = kSlab * 2 + 16;      // bytes between tokens in shared memory: 8 lanes' 16 bytes never collide
constexpr int kMaxTokens = 64;
constexpr int kFlush = 1024 / (kSlab / 2);  // slabs between flushes to int32

struct Params {
    const int8_t *a, *b;                    // tokens (m x k), weight (n x k)
    const float *row_scale, *col_scale;
    void *c;
    uint64_t lda, ldb, ldc;
    uint32_t m, n, k, slabs;                // slabs: of one CTA's share
    uint32_t a_vec, b_vec;                  // 16-byte units aligned
    uint32_t c_dtype, rounding, step;
    uint32_t early;                         // B may be read before the previous kernel has finished
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

// 16 bytes of a row from column k on, zeros past its end.
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const int8_t *row, uint32_t k, uint32_t end, bool vec)
{
    if (vec && k + 16 <= end) {
        if (STREAM) return __ldcs(reinterpret_cast<const uint4 *>(row + k));
        return *reinterpret_cast<const uint4 *>(row + k);
    }
    uint32_t w[4] = {0, 0, 0, 0};
    if (k < end) {
#pragma unroll 1
        for (uint32_t q = 0; q < 16 && k + q < end; ++q) {
            const uint32_t v = static_cast<uint32_t>(static_cast<uint8_t>(row[k + q])) << (8 * (q & 3));
            if (q < 4) w[0] |= v;
            else if (q < 8) w[1] |= v;
            else if (q < 12) w[2] |= v;
            else w[3] |= v;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma16816(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t addr)
{
    int32_t v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <int NB>
constexpr int smem_bytes()
{
    return 2 * 8 * NB * kPitch + 2 * 8 * NB * kRows * 4;
}

template <int NB>
__global__ void __launch_bounds__(kThreads, NB <= 2 ? 2 : 1) few_rows_kernel(const __grid_constant__ Params P)
{
    constexpr int kTokens = 8 * NB;
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char *xs = smem;                                               // [2][kTokens][kPitch], f16
    int32_t *part = reinterpret_cast<int32_t *>(smem + 2 * kTokens * kPitch);   // [2][kTokens][kRows]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3, half = warp & 1, wr = warp >> 1;
    const uint32_t rank = gemm::cluster_rank();
    uint32_t split;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t n0 = (blockIdx.x / split) * kRows;
    const uint32_t k_first = rank * P.slabs * kSlab;
    const uint32_t k_last = min(P.k, k_first + P.slabs * kSlab);            // at or below k_first: nothing to add
    const uint32_t slabs = k_last > k_first ? (k_last - k_first + kSlab - 1) / kSlab : 0;

    const int8_t *rows[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t row = min(n0 + wr * 32 + r * 8 + g, P.n - 1);        // a row past the end: its sums are not stored
        rows[r] = P.b + static_cast<uint64_t>(row) * P.ldb;
    }
    if (!P.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t kw = k_first + half * (kSlab / 2) + 16 * t;
    uint4 w[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) w[i][r] = load16<true>(rows[r], kw + i * 64, k_last, P.b_vec);
    if (P.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    uint4 xr[NB];
    auto fetch = [&](uint32_t s) {
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int u = q * kThreads + threadIdx.x, token = u >> 5;
            const uint32_t k = k_first + s * kSlab + (u & 31) * 16;
            xr[q] = static_cast<uint32_t>(token) < P.m
                        ? load16<false>(P.a + static_cast<uint64_t>(token) * P.lda, k, k_last, P.a_vec)
                        : make_uint4(0, 0, 0, 0);
        }
    };
    auto place = [&](uint32_t s) {
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            const int u = q * kThreads + threadIdx.x;
            uint32_t h[8];
            widen4(xr[q].x, h[0], h[1]);
            widen4(xr[q].y, h[2], h[3]);
            widen4(xr[q].z, h[4], h[5]);
            widen4(xr[q].w, h[6], h[7]);
            uint4 *dst = reinterpret_cast<uint4 *>(xs + ((s & 1) * kTokens + (u >> 5)) * kPitch + (u & 31) * 32);
            dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
            dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
        }
    };

    float acc[2][NB][4];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[mb][nb][q] = 0.0f;
    bool flushed = false;
    // this warp's sums so far to its own half's int32 sums
    auto flush = [&]() {
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int token = nb * 8 + 2 * t + (q & 1), row = wr * 32 + mb * 16 + g + (q >> 1) * 8;
                    int32_t *p = part + (half * kTokens + token) * kRows + row;
                    const int32_t v = __float2int_rn(acc[mb][nb][q]);
                    *p = flushed ? *p + v : v;
                    acc[mb][nb][q] = 0.0f;
                }
        flushed = true;
    };

    if (slabs) {
        fetch(0);
        place(0);
    }
    __syncthreads();
    for (uint32_t s = 0; s < slabs; ++s) {
        const bool more = s + 1 < slabs;
        if (more) fetch(s + 1);
        const unsigned char *x = xs + ((s & 1) * kTokens + g) * kPitch + half * kSlab + t * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[4][2][4];                 // [step][row block][fragment]
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t v[4] = {w[i][r].x, w[i][r].y, w[i][r].z, w[i][r].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) widen4(v[q], a[q][r >> 1][r & 1], a[q][r >> 1][(r & 1) + 2]);
                if (more) w[i][r] = load16<true>(rows[r], kw + (s + 1) * kSlab + i * 64, k_last, P.b_vec);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint4 *p = reinterpret_cast<const uint4 *>(x + nb * 8 * kPitch + i * 128);
                const uint4 lo = p[0], hi = p[1];
                const uint32_t b[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mma16816(acc[0][nb], a[q][0], b[2 * q], b[2 * q + 1]);
                    mma16816(acc[1][nb], a[q][1], b[2 * q], b[2 * q + 1]);
                }
            }
        }
        if (more) place(s + 1);
        if ((s + 1) % kFlush == 0) flush();
        __syncthreads();
    }
    if (!flushed || slabs % kFlush) flush();
    gemm::cluster_sync();

    // the cluster's sums: each CTA finishes its share of the outputs
    const uint32_t outs = kTokens * kRows;
    for (uint32_t o = rank * kThreads + threadIdx.x; o < outs; o += split * kThreads) {
        const uint32_t token = o / kRows, col = n0 + o % kRows;
        if (token >= P.m || col >= P.n) continue;
        int32_t sum = 0;
        const uint32_t at = smem_addr(part + o);
        for (uint32_t r = 0; r < split; ++r) {
            const uint32_t p = gemm::peer_addr(at, r);
            sum += ld_cluster_s32(p) + ld_cluster_s32(p + outs * 4);
        }
        const float y = __fmul_rn(__fmul_rn(__int2float_rn(sum), P.row_scale[token]), P.col_scale[col]);
        const uint64_t dst = token * P.ldc + col;
        if (P.c_dtype == ASR_F32) {
            static_cast<float *>(P.c)[dst] = y;
        } else {
            uint32_t h;
            if (P.rounding == ASR_ROUND_SR) {
                const uint64_t e = static_cast<uint64_t>(token) * P.n + col;
                uint32_t r[4];
                philox_q(e >> 2, P.step, P.keys, r);
                const uint32_t sel = static_cast<uint32_t>(e & 3u);
                h = round_sr(y, sel == 0 ? r[0] : sel == 1 ? r[1] : sel == 2 ? r[2] : r[3]);
            } else {
                h = round_rne(y);
            }
            static_cast<uint16_t *>(P.c)[dst] = static_cast<uint16_t>(h);
        }
    }
    gemm::cluster_sync();                        // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------------ host

std::mutex g_few_mu;
int g_few_sms[kMaxDevices];

template <int NB>
cudaError_t opt_in()
{
    return cudaFuncSetAttribute(few_rows_kernel<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NB>());
}

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
        if (e == cudaSuccess) e = opt_in<1>();
        if (e == cudaSuccess) e = opt_in<2>();
        if (e == cudaSuccess) e = opt_in<4>();
        if (e == cudaSuccess) e = opt_in<6>();
        if (e == cudaSuccess) e = opt_in<8>();
        if (e != cudaSuccess) return cuda_fail(e);
        g_few_sms[dev] = n;
    }
    *sms = g_few_sms[dev];
    return ASR_OK;
}

#ifndef ASR_FEW_CTAS
#define ASR_FEW_CTAS 4                      // CTAs wanted for each SM
#endif

template <int NB>
asr_status launch_few(Params &P, int sms, cudaStream_t stream)
{
    const uint32_t tiles = (P.n + kRows - 1) / kRows, all = (P.k + kSlab - 1) / kSlab;
    // shares of K: enough CTAs to fill the GPU, none below one slab, at most the portable cluster size
    uint32_t split = 1;
    while (split < 8 && split * 2 <= all && tiles * split < static_cast<uint32_t>(ASR_FEW_CTAS * sms)) split *= 2;
    P.slabs = (all + split - 1) / split;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(tiles * split, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<NB>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, few_rows_kernel<NB>, P);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(ASR_KERNEL_INT8_FEW_ROWS);
}

asr_status run(Params &P, cudaStream_t stream)
{
    int sms = 0;
    const asr_status st = setup(&sms);
    if (st != ASR_OK) return st;
    if (P.m <= 8) return launch_few<1>(P, sms, stream);
    if (P.m <= 16) return launch_few<2>(P, sms, stream);
    if (P.m <= 32) return launch_few<4>(P, sms, stream);
    if (P.m <= 48) return launch_few<6>(P, sms, stream);
    return launch_few<8>(P, sms, stream);
}

}  // namespace int8few
