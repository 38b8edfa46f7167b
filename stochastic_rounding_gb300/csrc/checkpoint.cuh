// checkpoint.cuh -- what a layer keeps of its input for the backward pass, in 8
// bits: making it and reading it, as kernels of their own and as what the
// activation's (activation.cuh) and the norm's (norm.cuh) kernels do on the way.
// Included into asr.cu (inside its anonymous namespace), after int8.cuh.
//
//   32 values of a row share a power of two, 2^e, the least (at least 2^-127)
//   with max |x| <= 127 2^e;   y = x 2^-e, exact;
//   q = rint(y)                              (nearest)
//     = floor(y) + [65536 (y - floor(y)) > r]  (stochastic)
//
// A power of two, and not max / 127, because everything about it is then exact --
// y, which neighbour a value goes to, the value that is read back, in bf16 too --
// at one byte for 32 values.  It costs up to a bit where the largest value is just
// above 127 2^e; 32 values rather than a row keep a strong channel from costing the
// others theirs.
//
// Bound by bytes, but for the stochastic form of bf16, which is by its instructions, twice
// the other's (8,192 x 14,336 bf16, one launch after another, at 6,697 GB/s 53 us: pack
// 56, stochastic 75, restore 59): no pipe is full (multiplications 48 %, logic 57, issue
// 59), but warps come to Philox's multiplications together and wait for that pipe.  Pairs
// of values go through the conversions together (fma.f32x2; pack, stochastic, 82 without).
//
// Random bits: eight values to a Philox counter, sixteen bits each, where the
// optimizers take four: the generator is a third of the stochastic form's
// instructions, and the third counter word sets these numbers apart from theirs.

namespace kept {

constexpr int kThreads = 256;
constexpr int kGroup = 32;
constexpr uint32_t kStream = 1;                 // last counter word

struct Store {                                  // where it goes
    int8_t *q;
    uint8_t *power;                             // e + 127; 255: the group holds an infinity or a NaN
    uint32_t q_ld, power_ld;
    uint64_t base;                              // first counter
    uint32_t across;                            // counters a row
    uint32_t vec;                               // codes of 16 values (2) or 8 (1) are aligned to their size
    uint32_t step;
    RoundKeys keys;
};

struct Source {
    const int8_t *q;
    const uint8_t *power;
    uint32_t q_ld, power_ld;
    uint32_t vec;
};

// How many of a unit's values, `most` at most, a row of `cols` has from `col` on.  Kernels
// have a form, FULL, that does not ask: for matrices of whole spans whose units are all
// aligned, as the widths of layers are, without the tests and the element by element
// accesses.  Only for bf16, whose kernels are bound by their instructions (pack,
// stochastic: 8,192 x 14,336 75 us, 8,192 x 14,352 without FULL 84; the gated activation's
// backward pass from codes at 0.96 of the copy rate, 0.88 without at 8,192 x 11,008);
// f32's are bound by bytes.
__device__ __forceinline__ int live_of(uint32_t cols, uint32_t col, uint32_t most = 8)
{
    return col >= cols ? 0 : static_cast<int>(cols - col < most ? cols - col : most);
}

// A matrix of f32 or bf16 values, rows `ld` apart.
struct Matrix {
    const void *p;
    uint32_t ld;
    uint32_t vec;                               // rows begin on 16 bytes (1), 32 bytes (2), or not (0)
};

struct Out {
    void *p;
    uint32_t ld;
    uint32_t vec;
};

// A unit of f32 in one access, where a lane's two of 16 bytes would each leave half of
// the sectors to the other (4,096 x 14,336: unpack 70 -> 53 us).
__device__ __forceinline__ void load32(const void *p, uint32_t w[8])
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

// Two binary32 numbers at once, each rounded as by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d)
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)),
          "l"(reinterpret_cast<const uint64_t &>(c)));
    return reinterpret_cast<const float2 &>(d);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d)
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return reinterpret_cast<const float2 &>(d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d)
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return reinterpret_cast<const float2 &>(d);
}

// Rounded up.
__device__ __forceinline__ float2 fma2_up(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("fma.rp.f32x2 %0, %1, %2, %3;" : "=l"(d)
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)),
          "l"(reinterpret_cast<const uint64_t &>(c)));
    return reinterpret_cast<const float2 &>(d);
}

__device__ __forceinline__ float2 add2_up(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rp.f32x2 %0, %1, %2;" : "=l"(d)
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return reinterpret_cast<const float2 &>(d);
}

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

__device__ __forceinline__ uint64_t place(uint32_t row, uint32_t ld, uint32_t col)
{
    return static_cast<uint64_t>(row) * ld + col;
}

// Eight values as they lie in memory, so that they can be fetched ahead of their use
// in as few registers as they take there.
template <int DT>
struct Raw {
    uint32_t w[DT == ASR_BF16 ? 4 : 8];
};

template <int DT, bool FULL = false>
__device__ __forceinline__ Raw<DT> fetch(const Matrix &M, uint32_t row, uint32_t col, int live, uint32_t vec)
{
    Raw<DT> r;
    const char *src = static_cast<const char *>(M.p) + place(row, M.ld, col) * (DT == ASR_BF16 ? 2 : 4);
    if constexpr (DT == ASR_F32) {
        if (vec == 2 && live == 8) {
            load32(src, r.w);
            return r;
        }
    }
    if (FULL || (vec && live == 8)) {
        const uint4 *p = reinterpret_cast<const uint4 *>(src);
        const uint4 a = p[0];
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        if (DT == ASR_F32) {
            const uint4 b = p[1];
            r.w[DT == ASR_F32 ? 4 : 0] = b.x, r.w[DT == ASR_F32 ? 5 : 0] = b.y;
            r.w[DT == ASR_F32 ? 6 : 0] = b.z, r.w[DT == ASR_F32 ? 7 : 0] = b.w;
        }
    } else if (DT == ASR_BF16) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = (2 * i < live ? p[2 * i] : 0u) | (2 * i + 1 < live ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
    } else {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(src);
#pragma unroll
        for (int i = 0; i < (DT == ASR_F32 ? 8 : 0); ++i) r.w[i] = i < live ? p[i] : 0u;
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void values(const Raw<DT> &r, float x[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = DT == ASR_F32 ? __uint_as_float(r.w[DT == ASR_F32 ? i : 0])
                             : (i & 1) ? bf16_hi(r.w[DT == ASR_F32 ? 0 : i >> 1]) : bf16_lo(r.w[DT == ASR_F32 ? 0 : i >> 1]);
}

// Sixteen values of a lane: two units side by side, of a warp 512 columns.
template <int DT>
struct Pair {
    Raw<DT> h[2];
};

__device__ __forceinline__ int half_of(int live, int h) { return live - 8 * h < 0 ? 0 : live - 8 * h < 8 ? live - 8 * h : 8; }

// Rows that begin off alignment come and go value by value, a warp's side by side, and
// change hands in shared memory: units of such rows, taken lane by lane, would touch
// every sector once for each of its values (8,192 x 14,335 bf16: unpack 86 us, 679
// lane by lane).
struct Stage {
    uint4 w[128];                               // a warp's 512 values
};

template <int DT>
struct WordOf {
    using type = uint32_t;
};
template <>
struct WordOf<ASR_BF16> {
    using type = uint16_t;
};

// COUNT values a lane, in the order of `place_of`: where value e of the warp lies, or
// null where there is none.
template <int DT, int COUNT, typename F>
__device__ __forceinline__ void stage_in(Stage &S, F place_of)
{
    using Word = typename WordOf<DT>::type;
    const uint32_t lane = threadIdx.x & 31;
    Word v[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        const Word *p = static_cast<const Word *>(place_of(32 * i + lane));
        v[i] = p ? *p : static_cast<Word>(0);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < COUNT; ++i) reinterpret_cast<Word *>(S.w)[32 * i + lane] = v[i];
    __syncwarp();
}

template <int DT, int COUNT, typename F>
__device__ __forceinline__ void stage_out(const Stage &S, F place_of)
{
    using Word = typename WordOf<DT>::type;
    const uint32_t lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        Word *p = static_cast<Word *>(place_of(32 * i + lane));
        if (p) *p = reinterpret_cast<const Word *>(S.w)[32 * i + lane];
    }
    __syncwarp();
}

template <int DT>
__device__ __forceinline__ Raw<DT> staged(const Stage &S, uint32_t unit)
{
    Raw<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == ASR_BF16 ? 1 : 2); ++i) {
        const uint4 v = S.w[unit * (DT == ASR_BF16 ? 1 : 2) + i];
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
    return r;
}

// A lane's sixteen from column `col` on, the row ending at `end`; all lanes of a warp together.
template <int DT, bool FULL>
__device__ __forceinline__ Pair<DT> fetch16(const Matrix &M, uint32_t row, uint32_t col, uint32_t end, uint32_t vec, Stage &S)
{
    Pair<DT> p;
    const int live = FULL ? 16 : live_of(end, col, 16);
    if (!FULL && vec == 0) {
        const uint32_t first = col - (threadIdx.x & 31) * 16;
        stage_in<DT, 16>(S, [&](uint32_t e) -> const void * {
            return first + e < end ? static_cast<const char *>(M.p) + place(row, M.ld, first + e) * sizeof(typename WordOf<DT>::type)
                                   : nullptr;
        });
#pragma unroll
        for (int h = 0; h < 2; ++h) p.h[h] = staged<DT>(S, (threadIdx.x & 31) * 2 + h);
    } else if (DT == ASR_BF16 && (FULL || (vec == 2 && live == 16))) {
        uint32_t w[8];
        load32(static_cast<const char *>(M.p) + place(row, M.ld, col) * 2, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) p.h[i >> 2].w[i & 3] = w[i];
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) p.h[h] = fetch<DT>(M, row, col + 8 * h, half_of(live, h), vec);
    }
    return p;
}

// A warp's way through a matrix in spans of kSpan columns: span `at` counted along
// the rows, then every `stride`-th.  Both are counts of a launch's warps.
constexpr uint32_t kSpan = 512;                 // sixteen values a lane

struct Walk {
    uint32_t row, rows, span, spans, drow, dspan;
    __device__ Walk(uint32_t rows_, uint32_t spans_)
    {
        const uint32_t at = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), stride = gridDim.x * (kThreads / 32);
        rows = rows_;
        spans = spans_;
        row = at / spans;
        span = at % spans;
        drow = stride / spans;
        dspan = stride % spans;
    }
    __device__ bool more() const { return row < rows; }
    __device__ void next()
    {
        row += drow;
        span += dspan;
        if (span >= spans) {
            span -= spans;
            ++row;
        }
    }
};

// The larger magnitude, NaN where one of them is.
__device__ __forceinline__ float most(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
    return d;
}

// Of pairs of bf16; their signs are left to be taken off.
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The bits of a group's largest magnitude, from COUNT units of each of its 4 / COUNT
// lanes.
template <int DT, int COUNT>
__device__ __forceinline__ uint32_t group_most(const Raw<DT> *r)
{
    if (DT == ASR_BF16) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
            const uint32_t u = most2(most2(r[k].w[0], r[k].w[1]), most2(r[k].w[2], r[k].w[3]));
            m = k ? most2(m, u) : u;
        }
#pragma unroll
        for (int d = 1; d < 4 / COUNT; d *= 2) m = most2(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        m &= 0x7FFF7FFFu;
        return max(m << 16, m & 0xFFFF0000u);               // as numbers: a NaN's bits are the largest
    }
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < COUNT; ++k) {
        float x[8];
        values(r[k], x);
        m = most(m, most(most(most(x[0], x[1]), most(x[2], x[3])), most(most(x[4], x[5]), most(x[6], x[7]))));
    }
#pragma unroll
    for (int d = 1; d < 4 / COUNT; d *= 2) m = most(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    return __float_as_uint(m);
}

// e + 127 for the bits of a largest value, 127 being 1.984375 * 2^6.
__device__ __forceinline__ uint32_t power_of(uint32_t top)
{
    const int b = static_cast<int>((top + 0x1FFFFu) >> 23) - 6;
    return top >= 0x7F800000u ? 255u : b > 0 ? static_cast<uint32_t>(b) : 0u;
}

__device__ __forceinline__ float scale_of(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7FC00000u : b ? b << 23 : 0x00400000u);
}

// Codes of a unit, the first value's in the lowest byte.  `up` is 2^-e; `at` the unit's
// counter.
//
// To nearest: x 2^-e + 1.5 * 2^23, rounded once, has q in its low byte.
// Stochastically: q = ceil(y - r / 65536), which is floor(y), or one more where the
// fraction is above r / 65536.  128 + r / 65536 is a binary32 number with r for its
// low bits; taken from y and rounded up, the difference keeps its ceiling, -128 away
// (whole numbers are representable), and 1.5 * 2^23 + 128 more, rounded up, is it.
template <bool SR, int DT>
__device__ __forceinline__ uint2 codes8(const Store &S, uint64_t at, float up, const Raw<DT> &raw)
{
    float x[8];
    values(raw, x);
    uint32_t c[8], w[4];
    if (SR) philox4x32_10(static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32), S.step, kStream, S.keys, w);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float2 v = make_float2(x[i], x[i + 1]);
        if (SR) {
            // less 128 + r / 65536: the sign is the highest bit of the word that r is put in
            const float2 r = make_float2(__uint_as_float(__byte_perm(w[i >> 1], 0xC3000000u, 0x7610)),
                                         __uint_as_float(__byte_perm(w[i >> 1], 0xC3000000u, 0x7632)));
            v = add2_up(fma2_up(v, both(up), r), both(12583040.0f));
        } else {
            v = fma2(v, both(up), both(12582912.0f));
        }
        c[i] = __float_as_uint(v.x), c[i + 1] = __float_as_uint(v.y);
    }
    return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

template <bool FULL>
__device__ __forceinline__ void store_codes(const Store &S, int8_t *q, int live, uint2 v)
{
    if (FULL || (live == 8 && S.vec)) {
        *reinterpret_cast<uint2 *>(q) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) q[i] = static_cast<int8_t>((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
    }
}

// Keeps a unit of a row, from `col` on, a multiple of 8, of which `live` values are the
// row's.  All lanes of a warp call this together; four in a row hold a group.
template <bool SR, int DT, bool FULL>
__device__ __forceinline__ void keep8(const Store &S, uint32_t row, uint32_t col, int live, const Raw<DT> &raw)
{
    const uint32_t b = power_of(group_most<DT, 1>(&raw));
    uint2 v = codes8<SR>(S, S.base + place(row, S.across, col >> 3), __uint_as_float((254u - b) << 23), raw);
    if (b == 255u) v = make_uint2(0, 0);
    store_codes<FULL>(S, S.q + place(row, S.q_ld, col), live, v);
    if ((FULL || live > 0) && (threadIdx.x & 3) == 0) S.power[place(row, S.power_ld, col >> 5)] = static_cast<uint8_t>(b);
}

// The same of two units side by side; two lanes hold a group.
template <bool SR, int DT, bool FULL>
__device__ __forceinline__ void keep16(const Store &S, uint32_t row, uint32_t col, int live, const Pair<DT> &raw)
{
    const uint32_t b = power_of(group_most<DT, 2>(raw.h));
    const float up = __uint_as_float((254u - b) << 23);
    const uint64_t at = S.base + place(row, S.across, col >> 3);        // even
    uint2 v = codes8<SR>(S, at, up, raw.h[0]), z = codes8<SR>(S, at | 1, up, raw.h[1]);
    if (b == 255u) v = z = make_uint2(0, 0);
    int8_t *q = S.q + place(row, S.q_ld, col);
    if (FULL || (live == 16 && S.vec == 2)) {
        *reinterpret_cast<uint4 *>(q) = make_uint4(v.x, v.y, z.x, z.y);
    } else {
        store_codes<false>(S, q, half_of(live, 0), v);
        store_codes<false>(S, q + 8, half_of(live, 1), z);
    }
    if ((FULL || live > 0) && (threadIdx.x & 1) == 0) S.power[place(row, S.power_ld, col >> 5)] = static_cast<uint8_t>(b);
}

// Codes and power of eight values, to be fetched ahead of their use.
struct Codes {
    uint2 v;
    uint32_t b;
};

template <bool FULL = false>
__device__ __forceinline__ Codes fetch_codes(const Source &S, uint32_t row, uint32_t col, int live)
{
    Codes c{make_uint2(0, 0), 0};
    if (!FULL && live <= 0) return c;
    const int8_t *q = S.q + place(row, S.q_ld, col);
    if (FULL || (live == 8 && S.vec)) {
        c.v = *reinterpret_cast<const uint2 *>(q);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) (i < 4 ? c.v.x : c.v.y) |= static_cast<uint32_t>(static_cast<uint8_t>(q[i])) << (8 * (i & 3));
    }
    c.b = S.power[place(row, S.power_ld, col >> 5)];
    return c;
}

struct Codes16 {
    uint2 h[2];
    uint32_t b;
};

template <bool FULL>
__device__ __forceinline__ Codes16 fetch_codes16(const Source &S, uint32_t row, uint32_t col, int live)
{
    Codes16 c;
    if (FULL || (live == 16 && S.vec == 2)) {
        const uint4 v = *reinterpret_cast<const uint4 *>(S.q + place(row, S.q_ld, col));
        c.h[0] = make_uint2(v.x, v.y), c.h[1] = make_uint2(v.z, v.w);
        c.b = S.power[place(row, S.power_ld, col >> 5)];
        return c;
    }
    const Codes a = fetch_codes(S, row, col, half_of(live, 0)), b = fetch_codes(S, row, col + 8, half_of(live, 1));
    c.h[0] = a.v, c.h[1] = b.v, c.b = a.b;
    return c;
}

// 2^7 + (128 + q) 2^-16 has a code for its low byte: times 2^16 2^e, less a constant
// times that, it is q 2^e, exactly.  The constant's product leaves binary32 above
// e = 104, where values are that large a number of times 2^7.
__device__ __forceinline__ void values(const Codes &c, float x[8])
{
    const uint32_t lo = c.v.x ^ 0x80808080u, hi = c.v.y ^ 0x80808080u;
    const float scale = scale_of(c.b);
    const bool large = c.b > 220u && c.b < 255u;
    const float by = large ? 65536.0f : __fmul_rn(scale, 65536.0f), less = __fmul_rn(-128.001953125f, by);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 v = fma2(make_float2(__uint_as_float(__byte_perm(i < 4 ? lo : hi, 0x43000000u, 0x7650 + (i & 3))),
                                          __uint_as_float(__byte_perm(i < 4 ? lo : hi, 0x43000000u, 0x7651 + (i & 3)))),
                              both(by), both(less));
        x[i] = v.x, x[i + 1] = v.y;
    }
    if (large) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], scale);
    }
}

// Codes of a lane's sixteen values from any column `col` on, and the powers of the two
// groups that they may lie in.
struct CodesAcross {
    uint4 v;
    uint32_t b[2];
    uint32_t left;                              // values in the first group
};

__device__ __forceinline__ CodesAcross fetch_across(const Source &S, uint32_t row, uint32_t col, uint32_t end, Stage &T)
{
    const uint32_t lane = threadIdx.x & 31, first = col - lane * 16;
    const int8_t *q = S.q + place(row, S.q_ld, first + lane);
    int8_t c[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) c[i] = first + 32 * i + lane < end ? q[32 * i] : 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) reinterpret_cast<int8_t *>(T.w)[32 * i + lane] = c[i];
    __syncwarp();
    CodesAcross r;
    r.v = T.w[lane];
    r.left = 32 - col % 32;
    r.b[0] = col < end ? S.power[place(row, S.power_ld, col >> 5)] : 0;
    r.b[1] = col + r.left < end ? S.power[place(row, S.power_ld, (col >> 5) + 1)] : 0;
    return r;
}

__device__ __forceinline__ void values(const CodesAcross &c, int half, float x[8])
{
    const float near = scale_of(c.b[0]), far = scale_of(c.b[1]);
    const uint32_t w[4] = {c.v.x, c.v.y, c.v.z, c.v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = 8 * half + i;
        const float q = static_cast<float>(static_cast<int8_t>(w[k >> 2] >> (8 * (k & 3))));
        x[i] = __fmul_rn(q, k < c.left ? near : far);
    }
}

// Eight values out, `live` of them, to nearest where they are bf16.
template <int DT, bool FULL = false>
__device__ __forceinline__ void store8(const Out &O, uint32_t row, uint32_t col, int live, uint32_t vec, const float v[8])
{
    char *dst = static_cast<char *>(O.p) + place(row, O.ld, col) * (DT == ASR_BF16 ? 2 : 4);
    if (DT == ASR_BF16) {
        uint16_t *p = reinterpret_cast<uint16_t *>(dst);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if (FULL || (vec && live == 8)) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < live) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
    } else {
        float *p = reinterpret_cast<float *>(dst);
        if (vec == 2 && live == 8) {
            gemm::st_global_v8(p, reinterpret_cast<const uint32_t *>(v));
        } else if (FULL || (vec && live == 8)) {
            reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < live) p[i] = v[i];
        }
    }
}

// Values as they are stored, to nearest where they are bf16.
template <int DT>
__device__ __forceinline__ Raw<DT> rounded(const float v[8])
{
    Raw<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == ASR_BF16 ? 4 : 8); ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[DT == ASR_BF16 ? 2 * i : i], v[DT == ASR_BF16 ? 2 * i + 1 : i]);
        r.w[i] = DT == ASR_BF16 ? *reinterpret_cast<const uint32_t *>(&h) : __float_as_uint(v[i]);
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void put_staged(Stage &S, uint32_t unit, const Raw<DT> &r)
{
#pragma unroll
    for (int i = 0; i < (DT == ASR_BF16 ? 1 : 2); ++i)
        S.w[unit * (DT == ASR_BF16 ? 1 : 2) + i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
}

// Sixteen out, as they come in.
template <int DT, bool FULL>
__device__ __forceinline__ void store16(const Out &O, uint32_t row, uint32_t col, uint32_t end, uint32_t vec, const float v[2][8],
                                        Stage &S)
{
    const int live = FULL ? 16 : live_of(end, col, 16);
    if (!FULL && vec == 0) {
        const uint32_t first = col - (threadIdx.x & 31) * 16;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) put_staged<DT>(S, (threadIdx.x & 31) * 2 + h, rounded<DT>(v[h]));
        stage_out<DT, 16>(S, [&](uint32_t e) -> void * {
            return first + e < end ? static_cast<char *>(O.p) + place(row, O.ld, first + e) * sizeof(typename WordOf<DT>::type)
                                   : nullptr;
        });
    } else if (DT == ASR_BF16 && (FULL || (vec == 2 && live == 16))) {
        const Raw<DT> a = rounded<DT>(v[0]), b = rounded<DT>(v[1]);
        const uint32_t w[8] = {a.w[0], a.w[1], a.w[2], a.w[3], b.w[0], b.w[1], b.w[2], b.w[3]};
        gemm::st_global_v8(static_cast<char *>(O.p) + place(row, O.ld, col) * 2, w);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) store8<DT>(O, row, col + 8 * h, half_of(live, h), vec, v[h]);
    }
}

// Where every value goes its own way, rows off alignment need no such exchange: a lane
// takes every 32nd of a span, and stores each as soon as it has it (8,192 x 14,335 bf16:
// the gated activation 153 us, its backward pass 336, exchanged 256 and 423; the backward
// pass with all of da stored before all of db 654).
constexpr int kLoose = 16;

template <int DT>
__device__ __forceinline__ void fetch_loose(const Matrix &M, uint32_t row, uint32_t first, uint32_t end, float x[kLoose])
{
    const char *p = static_cast<const char *>(M.p) + place(row, M.ld, first + (threadIdx.x & 31)) * (DT == ASR_BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kLoose; ++i) {
        x[i] = 0.0f;
        if (first + 32 * i + (threadIdx.x & 31) < end)
            x[i] = DT == ASR_F32 ? reinterpret_cast<const float *>(p)[32 * i] : bf16_lo(reinterpret_cast<const uint16_t *>(p)[32 * i]);
    }
}

// The i-th of them.
template <int DT>
__device__ __forceinline__ void store_loose1(const Out &O, uint32_t row, uint32_t first, uint32_t end, int i, float x)
{
    const uint32_t col = first + 32 * i + (threadIdx.x & 31);
    if (col >= end) return;
    if (DT == ASR_F32) static_cast<float *>(O.p)[place(row, O.ld, col)] = x;
    else static_cast<__nv_bfloat16 *>(O.p)[place(row, O.ld, col)] = __float2bfloat16_rn(x);
}

struct PackParams {
    Matrix x;
    uint32_t rows, cols;
    Store to;
};

// The next span's values are fetched before the current one's are worked on.
template <bool SR, int DT, bool FULL>
__global__ void __launch_bounds__(kThreads) pack_kernel(const __grid_constant__ PackParams P, uint32_t spans)
{
    __shared__ Stage stages[FULL ? 1 : kThreads / 32];
    Stage &stage = stages[FULL ? 0 : threadIdx.x >> 5];
    const uint32_t at = (threadIdx.x & 31) * 16;
    Pair<DT> next;
    auto load = [&](const Walk &k) {
        if (k.more()) next = fetch16<DT, FULL>(P.x, k.row, k.span * kSpan + at, P.cols, P.x.vec, stage);
    };
    Walk k(P.rows, spans);
    load(k);
    while (k.more()) {
        const Pair<DT> x = next;
        const uint32_t row = k.row, col = k.span * kSpan + at;
        k.next();
        load(k);
        keep16<SR, DT, FULL>(P.to, row, col, FULL ? 16 : live_of(P.cols, col, 16), x);
    }
}

struct UnpackParams {
    Source from;
    Out out;
    uint32_t rows, cols;
};

template <int DT, bool FULL>
__global__ void __launch_bounds__(kThreads) unpack_kernel(const __grid_constant__ UnpackParams P, uint32_t spans)
{
    __shared__ Stage stages[FULL ? 1 : kThreads / 32];
    Stage &stage = stages[FULL ? 0 : threadIdx.x >> 5];
    const uint32_t at = (threadIdx.x & 31) * 16;
    Codes16 next;
    auto load = [&](const Walk &k) {
        const uint32_t col = k.span * kSpan + at;
        if (k.more()) next = fetch_codes16<FULL>(P.from, k.row, col, FULL ? 16 : live_of(P.cols, col, 16));
    };
    Walk k(P.rows, spans);
    load(k);
    while (k.more()) {
        const Codes16 c = next;
        const uint32_t row = k.row, col = k.span * kSpan + at;
        k.next();
        load(k);
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) values(Codes{c.h[h], c.b}, v[h]);
        store16<DT, FULL>(P.out, row, col, P.cols, P.out.vec, v, stage);
    }
}

// ------------------------------------------------------------------ host

constexpr uint64_t kMaxRows = 1ull << 30, kMaxCols = 1ull << 24;
constexpr uint64_t kMaxWidth = 2 * kMaxCols;    // of a checkpoint: both halves of a gated activation's input

bool sizes_ok(uint64_t rows, uint64_t cols, uint64_t most = kMaxCols) { return rows <= kMaxRows && cols <= most; }

bool dtype_ok(int32_t dtype) { return dtype == ASR_F32 || dtype == ASR_BF16; }

bool pitch_ok(uint64_t ld, uint64_t least) { return ld >= least && ld < (1ull << 32); }

bool matrix_ok(const void *p, int32_t dtype, uint64_t ld, uint64_t cols)
{
    return p && muon::element_aligned(p, dtype) && pitch_ok(ld, cols);
}

// How every row's units begin: on 32 bytes (2: eight f32 values or sixteen bf16 ones in
// one access), on 16 bytes (1: eight bf16 values or four f32 ones), or not.
uint32_t rows_vec(const void *p, uint64_t ld, int32_t dtype)
{
    const uint64_t off = reinterpret_cast<uintptr_t>(p) | ld * (dtype == ASR_BF16 ? 2 : 4);
    return off % 32 == 0 ? 2 : off % 16 == 0 ? 1 : 0;
}

Matrix matrix(const void *p, uint64_t ld, int32_t dtype) { return Matrix{p, static_cast<uint32_t>(ld), rows_vec(p, ld, dtype)}; }

Out out(void *p, uint64_t ld, int32_t dtype) { return Out{p, static_cast<uint32_t>(ld), rows_vec(p, ld, dtype)}; }

// Codes of 16 values (2) or 8 (1) are aligned to their size.
uint32_t codes_vec(const void *p, uint64_t ld)
{
    const uint64_t off = reinterpret_cast<uintptr_t>(p) | ld;
    return off % 16 == 0 ? 2 : off % 8 == 0 ? 1 : 0;
}

// Whether a row's powers are aligned words of four.
bool powers_whole(const asr_checkpoint &c, uint64_t cols)
{
    return ((reinterpret_cast<uintptr_t>(c.power) | c.power_ld) & 3u) == 0 && cols % (4 * kGroup) == 0;
}

uint64_t groups(uint64_t cols) { return (cols + kGroup - 1) / kGroup; }

// Whether a checkpoint of rows x cols can be read.
asr_status readable(const asr_checkpoint &c, uint64_t cols)
{
    return c.q && c.power && pitch_ok(c.q_ld, cols) && pitch_ok(c.power_ld, groups(cols))
               ? ASR_OK : ASR_ERR_INVALID_VALUE;
}

// And written, its random bits with it.
asr_status writable(const asr_checkpoint &c, uint64_t rows, uint64_t cols)
{
    if (c.rounding != ASR_ROUND_SR && c.rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (c.base_index % kGroup || c.base_index > UINT64_MAX - rows * groups(cols) * kGroup) return ASR_ERR_INVALID_VALUE;
    return readable(c, cols);
}

Source source(const asr_checkpoint &c)
{
    return Source{c.q, c.power, static_cast<uint32_t>(c.q_ld), static_cast<uint32_t>(c.power_ld),
                  codes_vec(c.q, c.q_ld)};
}

Store store(const asr_checkpoint &c, uint64_t cols)
{
    Store S;
    S.q = c.q;
    S.power = c.power;
    S.q_ld = static_cast<uint32_t>(c.q_ld);
    S.power_ld = static_cast<uint32_t>(c.power_ld);
    S.base = c.base_index / 8;
    S.across = static_cast<uint32_t>(groups(cols) * (kGroup / 8));
    S.vec = codes_vec(c.q, c.q_ld);
    S.step = c.step;
    S.keys = make_keys(c.seed);
    return S;
}

// Loads every kernel of a list on the current device once, so that any later call
// of them may be captured into a graph.
template <typename... K>
asr_status load_once(std::atomic<uint64_t> &ready, K... kernels)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (ready.load(std::memory_order_acquire) & bit)) return ASR_OK;
    (void)std::initializer_list<int>{(e = e == cudaSuccess ? prod::load_kernel(kernels) : e, 0)...};
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit, std::memory_order_release);
    return ASR_OK;
}

// How many blocks of a kernel the current device holds at once, `limit` an SM at most.
// A kernel and its threads settle the limit and the shared memory, if it has any in this
// call.
template <typename K>
asr_status resident(K kernel, int threads, size_t smem, int *blocks, int limit = 32)
{
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const uint64_t key = (static_cast<uint64_t>(dev) << 48) ^ reinterpret_cast<uintptr_t>(kernel) ^
                         (static_cast<uint64_t>(threads / 32) << 54) ^ (static_cast<uint64_t>(smem != 0) << 60);
    std::lock_guard<std::mutex> lk(g_grid_mu);
    auto it = g_grid_cache.find(key);
    if (it != g_grid_cache.end()) {
        *blocks = it->second;
        return ASR_OK;
    }
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e != cudaSuccess) return cuda_fail(e);
    *blocks = sms * (per_sm < 1 ? 1 : per_sm < limit ? per_sm : limit);
    g_grid_cache[key] = *blocks;
    return ASR_OK;
}

// A launch of blocks of eight warps that walk over the spans of a matrix, `limit` an SM at
// most: several streams are faster where fewer warps are at them at once than there is
// room for (by measurement; rows of memory that are closed before they are done would
// explain it).
template <typename K, typename P>
asr_status walk(int kind, K kernel, const P &params, uint64_t rows, uint64_t cols, uint64_t span, cudaStream_t stream,
                int limit = 32)
{
    int most = 0;
    const asr_status st = resident(kernel, kThreads, 0, &most, limit);
    if (st != ASR_OK) return st;
    const uint64_t spans = (cols + span - 1) / span;
    kernel<<<int8::blocks_for(rows * spans, kThreads / 32, static_cast<uint64_t>(most)), kThreads, 0, stream>>>(
        params, static_cast<uint32_t>(spans));
    return launched(kind);
}

asr_status setup()
{
    static std::atomic<uint64_t> ready{0};
    return load_once(ready, pack_kernel<false, ASR_F32, false>, pack_kernel<false, ASR_BF16, false>,
                     pack_kernel<false, ASR_BF16, true>, pack_kernel<true, ASR_F32, false>,
                     pack_kernel<true, ASR_BF16, false>, pack_kernel<true, ASR_BF16, true>, unpack_kernel<ASR_F32, false>,
                     unpack_kernel<ASR_BF16, false>, unpack_kernel<ASR_BF16, true>);
}

asr_status pack(const void *x, int32_t dtype, uint64_t rows, uint64_t cols, uint64_t x_ld, const asr_checkpoint *to,
                cudaStream_t stream)
{
    if (!dtype_ok(dtype)) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (!to) return ASR_ERR_INVALID_VALUE;
    if (to->rounding != ASR_ROUND_SR && to->rounding != ASR_ROUND_RNE) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (rows == 0 || cols == 0) return ASR_OK;
    if (!sizes_ok(rows, cols, kMaxWidth) || !matrix_ok(x, dtype, x_ld, cols)) return ASR_ERR_INVALID_VALUE;
    asr_status st = writable(*to, rows, cols);
    if (st == ASR_OK) st = setup();
    if (st != ASR_OK) return st;
    PackParams P;
    P.x = matrix(x, x_ld, dtype);
    P.rows = static_cast<uint32_t>(rows);
    P.cols = static_cast<uint32_t>(cols);
    P.to = store(*to, cols);
    const bool sr = to->rounding == ASR_ROUND_SR, full = cols % kSpan == 0 && P.x.vec == 2 && P.to.vec == 2;
    auto kernel = sr ? pack_kernel<true, ASR_F32, false> : pack_kernel<false, ASR_F32, false>;
    if (dtype == ASR_BF16)
        kernel = full ? (sr ? pack_kernel<true, ASR_BF16, true> : pack_kernel<false, ASR_BF16, true>)
                      : (sr ? pack_kernel<true, ASR_BF16, false> : pack_kernel<false, ASR_BF16, false>);
    // bf16, 8,192 rows of 4,096, 8,192, 11,008, 14,336, us: six blocks 18.6, 34.0, 45.2, 55.9, four 20.5, 36.3, 48.1, 59.4, as many
    // as fit 18.5, 34.1, 45.2, 57.2; stochastic the same from four on
    return walk(ASR_KERNEL_CHECKPOINT, kernel, P, rows, cols, kSpan, stream, 6);
}

asr_status unpack(const asr_checkpoint *from, uint64_t rows, uint64_t cols, void *dst, int32_t dtype, uint64_t ld,
                  cudaStream_t stream)
{
    if (!dtype_ok(dtype)) return ASR_ERR_UNSUPPORTED_DTYPE;
    if (!from) return ASR_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0) return ASR_OK;
    if (!sizes_ok(rows, cols, kMaxWidth) || !matrix_ok(dst, dtype, ld, cols)) return ASR_ERR_INVALID_VALUE;
    asr_status st = readable(*from, cols);
    if (st == ASR_OK) st = setup();
    if (st != ASR_OK) return st;
    UnpackParams P;
    P.from = source(*from);
    P.out = out(dst, ld, dtype);
    P.rows = static_cast<uint32_t>(rows);
    P.cols = static_cast<uint32_t>(cols);
    const bool full = cols % kSpan == 0 && P.from.vec == 2 && P.out.vec == 2;
    auto kernel = dtype != ASR_BF16 ? unpack_kernel<ASR_F32, false> : full ? unpack_kernel<ASR_BF16, true>
                                                                           : unpack_kernel<ASR_BF16, false>;
    // 8,192 rows of 4,096, 8,192, 11,008, 14,336, us; bf16: five blocks 20.5, 35.1, 46.8, 58.6, as many as fit 19.2, 37.1, 46.2,
    // 63.5, four 20.7, 36.9, 49.2, 61.4; f32: three 30.5, 55.2, 71.9, 92.8, as many as fit 30.3, 61.2, 82.6, 104
    return walk(ASR_KERNEL_CHECKPOINT, kernel, P, rows, cols, kSpan, stream, dtype == ASR_BF16 ? 5 : 3);
}

}  // namespace kept
