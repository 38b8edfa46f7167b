// int8_product.cuh -- the products of 8-bit integers held in f16 (int8.cuh), one
// or two in a launch.  Included into asr.cu (inside its anonymous namespace),
// after product.cuh, whose tiles, roles and barriers it keeps.
//
// The sum over K is cut into chunks of 1,024, each accumulated on its own in
// tensor memory -- exact in binary32 -- and added up by the epilogue warps in
// int32 registers; the next chunk's products go into the other accumulator
// meanwhile.  Sums of more than 131,071 products (gradients over as many tokens
// or outputs), which int32 need not hold, are added up in int64 by a form of the
// kernel of its own (LONG), whose running sums do not fit the registers (dw of
// 1,024 x 2,048 over 131,071 tokens 962 us, over 131,072 974 us).
//
// The two products of a backward pass (dx and dw) go as one list of tiles, those
// of the longer sum first: in a launch each, both leave their last round of tiles
// part empty, and small ones pay for two launches (4,096 tokens, 8,192 x 2,048: the
// call 295 us with two, 273 with one; 1,111 tokens, 515 x 1,365: 49.3 and 46.6).  How
// an operand is stored is a field of its product here, the same for all lanes.
//
// What bounds it: the tensor cores, at 1,590 to 1,660 TFLOP/s for the first of
// these (166 to 173 us) and 1,820 for 8,192 x 14,336 x 4,096 alone (528 us), less
// where calls follow one another and the power limit lowers the clock; small ones
// the chain of copies, sums and epilogue (20 us for 777 x 1,001 x 2,049).  The
// running sums take 64 of an epilogue thread's 96 registers: 248 bytes of a
// thread's other values are spilled, once a tile.

namespace prod {

constexpr uint32_t kMaxIntSum = 131071;         // 128^2 of each product: below 2^31

struct Int8Product {
    Params P;                       // sizes, output, scales; parts of its tiles in the last round
    uint32_t a_mn, b_mn;            // stored across the contraction
};

struct Int8Products {
    CUtensorMap map[6];             // of each product: A, B, B for parts of tiles
    Int8Product p[2];
    uint32_t count, tiles0;         // tiles of the first product
    // Work items: whole tiles up to `wide`; parts of the first product's tiles up
    // to `mid`, of the second's up to `items`.  From `last` on they are a round that
    // does not fill the clusters.
    uint32_t wide, mid, items, last;
    uint32_t chunk;                 // K slices per accumulation
};

struct Int8Item {
    uint32_t which;
    Item it;
};

__device__ __forceinline__ Int8Item int8_item(const Int8Products &L, uint32_t t, uint32_t clusters)
{
    Int8Item I;
    // the clusters that had shorter tiles before take what is left
    if (t >= L.last) t = L.last + clusters - 1 - (t - L.last);
    uint32_t tile = t, part = 0;
    I.it.width = kTile;
    if (t >= L.wide) {
        const bool second = t >= L.mid;
        const uint32_t parts = L.p[second ? 1 : 0].P.parts, first = second ? L.mid : L.wide;
        tile = (second ? max(L.tiles0, L.wide) : L.wide) + (t - first) / parts;
        part = (t - first) & (parts - 1);
        I.it.width = kTile / parts;
    }
    I.which = tile >= L.tiles0 ? 1 : 0;
    const Params &P = L.p[I.which].P;
    uint32_t mt, nt;
    tile_coords(I.which ? tile - L.tiles0 : tile, P.tiles_m, P.tiles_n, mt, nt, kGroupM);
    I.it.z = 0;
    I.it.m0 = mt * kTile;
    I.it.n0 = nt * kTile + part * I.it.width;
    I.it.mirror = false;
    return I;
}

// Persistent over work items: cluster c takes items c, c + clusters, ...
template <bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
int8_product_kernel(const __grid_constant__ Int8Products L, uint64_t limit_ns)
{
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
    // this cluster's items: t = cluster, cluster + clusters, ... below `end`
    const uint32_t end = L.items - L.last > clusters - 1 - cluster ? L.last + clusters : L.last;

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
        for (uint32_t t = cluster; ok && t < end; t += clusters) {
            const Int8Item I = int8_item(L, t, clusters);
            const Item &it = I.it;
            const Params &P = L.p[I.which].P;
            const bool narrow = it.width != kTile, a_mn = L.p[I.which].a_mn != 0, b_mn = L.p[I.which].b_mn != 0;
            const CUtensorMap *map_a = &L.map[3 * I.which], *map_b = &L.map[3 * I.which + (narrow ? 2 : 1)];
            const uint32_t kblocks = (P.k + kBK - 1) / kBK;
            uint32_t ra = it.m0 + rank * 128, rb = it.n0 + rank * (it.width / 2);
            // rows wholly past the matrix: any rows do, their sums are not stored
            const bool a2 = ra + 64 < P.m, b2 = rb + 64 < P.n;
            if (ra >= P.m) ra = 0;
            if (rb >= P.n) rb = 0;
            // B in this CTA: half of the item's columns, or (stored across) blocks of 64 of them
            const uint32_t bytes_b = !narrow ? kHalfBytes : b_mn ? kHalfBytes / 2 : kHalfBytes / P.parts;
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
                    if (a_mn) {
                        tma_load_3d_pair(da, map_a, static_cast<int32_t>(ra), k0, z, bar);
                        tma_load_3d_pair(da + 8192, map_a, static_cast<int32_t>(a2 ? ra + 64 : ra), k0, z, bar);
                    } else {
                        tma_load_3d_pair(da, map_a, k0, static_cast<int32_t>(ra), z, bar);
                    }
                    if (b_mn) {
                        tma_load_3d_pair(db, map_b, static_cast<int32_t>(rb), k0, z, bar);
                        if (!narrow)
                            tma_load_3d_pair(db + 8192, map_b, static_cast<int32_t>(b2 ? rb + 64 : rb), k0, z, bar);
                    } else {
                        tma_load_3d_pair(db, map_b, k0, static_cast<int32_t>(rb), z, bar);
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
        constexpr uint64_t kDescStage = kStageBytes >> 4, kDescHalf = kHalfBytes >> 4;
        for (uint32_t t = cluster; ok && t < end; t += clusters) {
            const Int8Item I = int8_item(L, t, clusters);
            const bool a_mn = L.p[I.which].a_mn != 0, b_mn = L.p[I.which].b_mn != 0;
            const uint32_t idesc = instr_desc(I.it.width, a_mn, b_mn), kblocks = (L.p[I.which].P.k + kBK - 1) / kBK;
            const uint64_t desc_a0 = a_mn ? operand_desc<true>(base) : operand_desc<false>(base);
            const uint64_t desc_b0 = b_mn ? operand_desc<true>(base + 2 * kHalfBytes)
                                          : operand_desc<false>(base + 2 * kHalfBytes);
            const uint64_t step_a = a_mn ? 2048 >> 4 : 32 >> 4, step_b = b_mn ? 2048 >> 4 : 32 >> 4;
            for (uint32_t kc = 0; ok && kc < kblocks; kc += L.chunk, ++i) {
                const int b = static_cast<int>(i % kAccBufs);
                const uint32_t ub = i / kAccBufs;
                if (ub > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait_cluster(acc_empty(b), (ub - 1) & 1u, limit_ns))) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + static_cast<uint32_t>(b * kTile);
                const uint32_t kend = kblocks - kc < L.chunk ? kblocks : kc + L.chunk;
                for (uint32_t kb = kc; kb < kend; ++kb) {
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
                            mma_bf16_pair(d, aj, bj, idesc, (kb != kc || j != 0) ? 1u : 0u);
                            mma_bf16_pair(d, aj + step_a, bj + step_b, idesc, 1u);
                            mma_bf16_pair(d, aj + 2 * step_a, bj + 2 * step_b, idesc, 1u);
                            mma_bf16_pair(d, aj + 3 * step_a, bj + 3 * step_b, idesc, 1u);
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
        bool ok = true;
        for (uint32_t t = cluster; ok && t < end; t += clusters) {
            const Int8Item I = int8_item(L, t, clusters);
            const Item &it = I.it;
            const Params &P = L.p[I.which].P;
            const uint32_t kblocks = (P.k + kBK - 1) / kBK;
            const uint32_t row = it.m0 + rank * 128 + quarter * 32 + lane;
            const uint32_t ncols = it.n0 >= P.n ? 0 : P.n - it.n0 < it.width ? P.n - it.n0 : it.width;
            const uint32_t span = it.width / (kEpi / 4), c_lo = group * span;      // this warp's columns
            const uint32_t c_hi = ncols < c_lo + span ? ncols : c_lo + span;
            const uint32_t col0 = it.n0 + c_lo, cols = c_hi > c_lo && row - lane < P.m ? c_hi - c_lo : 0;
            std::conditional_t<LONG, int64_t, int32_t> acc[kSpan];
            // the scales, before the wait for the sums; ordinary loads, as the kernel
            // that wrote them may have been running when this one started
            float scale[kSpan / 32];
#pragma unroll
            for (int h = 0; h < kSpan / 32; ++h)
                scale[h] = 32u * h + lane < cols ? P.col_scale[col0 + 32 * h + lane] : 0.0f;
            for (uint32_t kc = 0; kc < kblocks; kc += L.chunk, ++i) {
                const int b = static_cast<int>(i % kAccBufs);
                if (!__all_sync(0xFFFFFFFFu, pair_wait(acc_full(b), (i / kAccBufs) & 1u, limit_ns))) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t tq =
                    tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(b * kTile) + c_lo;
#pragma unroll
                for (int c = 0; c < kSpan; c += kBlock) {
                    if (static_cast<uint32_t>(c) >= span) continue;
                    uint32_t v[16];
                    gemm::tmem_ld16(tq + c, v);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const int32_t a = __float2int_rn(__uint_as_float(v[q]));
                        acc[c + q] = kc == 0 ? a : acc[c + q] + a;
                    }
                }
                // this warp has read its part of accumulator b
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(peer_addr(acc_empty(b), 0));
            }
            if (ok) {
                // one copy of the finishing code for the warp's blocks
#pragma unroll 1
                for (int c = 0; static_cast<uint32_t>(c) < cols; c += kBlock) {
                    float x[16], cs[16];
#pragma unroll
                    for (int d = 0; d < kSpan; d += kBlock) {
                        if (c != d) continue;
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            x[q] = LONG ? __ll2float_rn(acc[d + q]) : __int2float_rn(static_cast<int32_t>(acc[d + q]));
                            cs[q] = __shfl_sync(0xFFFFFFFFu, scale[d / 32], (d & 31) + q);
                        }
                    }
                    finish_block<kScaled>(P, 0, row, col0 + c, x, nullptr, cs, stage, lane, []() {});
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

bool g_int8_ready[kMaxDevices];
int g_int8_pairs[kMaxDevices];

asr_status int8_setup(int *pairs)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return ASR_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lk(g_prod_mu);
    if (!g_int8_ready[dev]) {
        int n = 0;
        e = setup_one(int8_product_kernel<false>, &n);
        if (e == cudaSuccess) e = setup_one(int8_product_kernel<true>, &n);
        if (e != cudaSuccess) return cuda_fail(e);
        if (n < 1) return cuda_fail(cudaErrorNotSupported);
        g_int8_pairs[dev] = n;
        g_int8_ready[dev] = true;
    }
    *pairs = g_int8_pairs[dev];
    return ASR_OK;
}

// Adds the product of a (m x k, or k x m where a_mn) and b (n x k, or k x n
// where b_mn) to a launch; P holds the output's fields.
void int8_add(Int8Products &L, Stored operands[4], const Stored &a, bool a_mn, const Stored &b, bool b_mn,
              const Params &P)
{
    operands[2 * L.count] = a;
    operands[2 * L.count + 1] = b;
    Int8Product &Q = L.p[L.count++];
    Q.P = P;
    Q.a_mn = a_mn;
    Q.b_mn = b_mn;
    Q.P.m = static_cast<uint32_t>(a_mn ? a.cols : a.rows);
    Q.P.k = static_cast<uint32_t>(a_mn ? a.rows : a.cols);
    Q.P.n = static_cast<uint32_t>(b_mn ? b.cols : b.rows);
    Q.P.tiles_m = (Q.P.m + kTile - 1) / kTile;
    Q.P.tiles_n = (Q.P.n + kTile - 1) / kTile;
}

asr_status int8_launch(Int8Products &L, Stored operands[4], uint32_t chunk, cudaStream_t stream)
{
    int pairs = 0;
    asr_status st = int8_setup(&pairs);
    if (st != ASR_OK) return st;
    L.chunk = chunk;
    if (L.count == 2 && L.p[0].P.k < L.p[1].P.k) {          // the longer sums first
        std::swap(L.p[0], L.p[1]);
        std::swap(operands[0], operands[2]);
        std::swap(operands[1], operands[3]);
    }
    uint64_t tiles = static_cast<uint64_t>(L.p[0].P.tiles_m) * L.p[0].P.tiles_n;
    if (tiles >= (1ull << 30)) return ASR_ERR_INVALID_VALUE;
    L.tiles0 = static_cast<uint32_t>(tiles);
    if (L.count == 2) tiles += static_cast<uint64_t>(L.p[1].P.tiles_m) * L.p[1].P.tiles_n;
    if (tiles >= (1ull << 30)) return ASR_ERR_INVALID_VALUE;
    // The tiles of a last round that leaves clusters idle go in parts, of the two
    // products' such as make the longest of them shortest.
    const uint64_t slots = static_cast<uint64_t>(pairs), rest = tiles % slots, whole = tiles - rest;
    const uint64_t rest0 = whole < L.tiles0 ? L.tiles0 - whole : 0, rest1 = rest - rest0;
    uint64_t best = ~0ull;
    for (uint32_t p0 = 4; p0; p0 /= 2)
        for (uint32_t p1 = 4; p1; p1 /= 2) {
            if (rest0 * p0 + rest1 * p1 > slots) continue;
            const uint64_t k0 = rest0 ? 4 / p0 * static_cast<uint64_t>(L.p[0].P.k) : 0;
            const uint64_t k1 = rest1 ? 4 / p1 * static_cast<uint64_t>(L.p[1].P.k) : 0;
            if ((k0 > k1 ? k0 : k1) > best) continue;
            best = k0 > k1 ? k0 : k1;
            L.p[0].P.parts = p0;
            L.p[1].P.parts = p1;
        }
    L.wide = static_cast<uint32_t>(whole);
    L.mid = static_cast<uint32_t>(whole + rest0 * L.p[0].P.parts);
    L.items = static_cast<uint32_t>(L.mid + rest1 * L.p[1].P.parts);
    const unsigned clusters = L.items < slots ? L.items : static_cast<unsigned>(pairs);
    L.last = L.items - L.items % clusters;
    for (uint32_t i = 0; i < L.count; ++i) {
        const Int8Product &Q = L.p[i];
        const Stored &a = operands[2 * i], &b = operands[2 * i + 1];
        st = make_map(&L.map[3 * i], a.ptr, a.rows, a.cols, a.ld, a.stride, 1, Q.a_mn ? 64 : 128);
        if (st == ASR_OK) st = make_map(&L.map[3 * i + 1], b.ptr, b.rows, b.cols, b.ld, b.stride, 1, Q.b_mn ? 64 : 128);
        if (st == ASR_OK)
            st = make_map(&L.map[3 * i + 2], b.ptr, b.rows, b.cols, b.ld, b.stride, 1, Q.b_mn ? 64 : 128 / Q.P.parts);
        if (st != ASR_OK) return st;
    }
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
    const bool wide_sums = L.p[0].P.k > kMaxIntSum || L.p[1].P.k > kMaxIntSum;
    const cudaError_t e = wide_sums ? cudaLaunchKernelEx(&cfg, int8_product_kernel<true>, L, limit)
                                    : cudaLaunchKernelEx(&cfg, int8_product_kernel<false>, L, limit);
    if (e != cudaSuccess) return cuda_fail(e);
    return launched(ASR_KERNEL_PRODUCT);
}

}  // namespace prod
