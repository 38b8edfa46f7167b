// int8_levels.cuh -- values to 8-bit integers of a given scale: what the
// quantising kernels (int8.cuh) and the product with few rows (int8_few.cuh)
// share.  Included into asr.cu (inside its anonymous namespace), after muon.cuh.

namespace int8 {

// How a row's values become integers: y = (x * pre) * inv.  A row whose largest
// value is so small that 127 / max would overflow is raised by 2^64 first (exact);
// a row that holds an infinity or a NaN gives zeros, and its scale, not finite,
// marks every product of the row.  Both are rare, and `odd` sets them apart.
struct Levels {
    float pre, inv;
    bool odd;
};

__device__ __forceinline__ Levels levels_of(float top)
{
    Levels L;
    L.pre = top < 0x1p-64f ? 0x1p64f : 1.0f;
    L.inv = top > 0.0f && top <= 3.402823466e38f ? __fdiv_rn(127.0f, __fmul_rn(top, L.pre)) : 0.0f;
    L.odd = L.inv == 0.0f || L.pre != 1.0f;
    return L;
}

__device__ __forceinline__ float regular(float x, const Levels &L) { return L.inv == 0.0f ? 0.0f : __fmul_rn(x, L.pre); }

// Integers come in pairs, as 0x6480 + q in each half of a word: as f16 that is
// 1,152 + q.
//
// To nearest: |y| <= 127 (1 + 2^-23), so that the nearest is at most 127, and
// the sum with 1.5 * 2^23 + 0x6480 has it in its low half.
__device__ __forceinline__ uint32_t nearest2(float x, float y, float inv_x, float inv_y)
{
    constexpr float kMagic = 12582912.0f + 25728.0f;
    return __byte_perm(__float_as_uint(__fadd_rn(__fmul_rn(x, inv_x), kMagic)),
                       __float_as_uint(__fadd_rn(__fmul_rn(y, inv_y), kMagic)), 0x5410);
}

// Stochastically: floor(y) + [65536 (y - floor(y)) > r] for whole r in [0, 65535]
// is floor((ceil(65536 y) + 65535 - r) / 65536), the sum's high half.  The scales
// come times 65536 (exact); not_r is 65535 - r.  |65536 y| <= 127 * 65536 (1 + 2^-24)
// before its rounding, in steps of 1/2, so at most 127 * 65536 + 1/2: the sum can
// come to 128 but not below -127.  The minimum is taken as of f16 numbers, whose
// order is that of these patterns.
__device__ __forceinline__ uint32_t random2(float x, float y, float inv_x, float inv_y, uint32_t not_r, uint32_t not_s)
{
    const uint32_t a = static_cast<uint32_t>(__float2int_ru(__fmul_rn(x, inv_x))) + not_r + 0x64800000u;
    const uint32_t b = static_cast<uint32_t>(__float2int_ru(__fmul_rn(y, inv_y))) + not_s + 0x64800000u;
    const uint32_t v = __byte_perm(a, b, 0x7632);
    const __half2 most = __halves2half2(__ushort_as_half(0x64FF), __ushort_as_half(0x64FF));
    const __half2 m = __hmin2(*reinterpret_cast<const __half2 *>(&v), most);
    return *reinterpret_cast<const uint32_t *>(&m);
}

// Eight of them as f16, or as bytes.
__device__ __forceinline__ uint4 halves_of(const uint32_t e[4])
{
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&e[i]), bias);
        h[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

__device__ __forceinline__ uint2 bytes_of(const uint32_t e[4])
{
    return make_uint2(__byte_perm(e[0], e[1], 0x6420) ^ 0x80808080u, __byte_perm(e[2], e[3], 0x6420) ^ 0x80808080u);
}

__device__ __forceinline__ void store_int8(int8_t *dst, const uint32_t e[4], int live)
{
    const uint2 w = bytes_of(e);
    if (live == 8 && (reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
        *reinterpret_cast<uint2 *>(dst) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) dst[i] = static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
}

// Eight values of one scale.
template <bool SR>
__device__ __forceinline__ void quantise8(const float x[8], const Levels &L, const uint32_t not_r[8], uint32_t e[4])
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i];
    if (L.odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = regular(x[i], L);
    }
    const float inv = SR ? __fmul_rn(L.inv, 65536.0f) : L.inv;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        e[i] = SR ? random2(v[2 * i], v[2 * i + 1], inv, inv, not_r[2 * i], not_r[2 * i + 1])
                  : nearest2(v[2 * i], v[2 * i + 1], inv, inv);
}

__device__ __forceinline__ uint32_t absbits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

}  // namespace int8
