// Microscaled storage (gfx950): 32 values along a row share a power of two.
//
//   v = q 2^(b - 127),  b one byte per block;  q: SPEC_MX_INT8 i / 64, |i| <= 127
//                                              SPEC_MX_FP4  +-{0, .5, 1, 1.5, 2, 3, 4, 6}
//
// b is the smallest at which the block's largest magnitude m 2^(E - 127), 1 <= m < 2,
// does not round past the largest q: a value is then off by half a step at most.
// INT8: 64 m < 127.5, so b = E, or E + 1 from m = 1.9921875 on.  FP4: 4 m < 7, so
// b = E - 2, or E - 1 from m = 1.75 on.  b stops at 254 and 252, where the largest q
// would leave the range of f32 (the largest values there are cut to it), and at 0.
// Byte 255 marks a block that held NaN or an infinity: all of it reads as NaN.
// Every step is exact (comparisons, powers of two, one rounding to nearest even).
//
// Four lanes hold a block, eight values each: the largest is found by two
// exchanges between neighbouring lanes.
#pragma once

#include "internal.h"
#include "mm.h"

constexpr int MX_NAN = 255;

// bytes of the codes of a block of 32
constexpr int mx_block_bytes(int fmt) { return fmt == SPEC_MX_INT8 ? 32 : 16; }
// rows of codes and of scales as spec_mx_quantize lays them out
inline int64_t mx_code_row(int fmt, int64_t cols) { return (cols + 31) / 32 * mx_block_bytes(fmt); }
inline int64_t mx_scale_row(int64_t cols) { return ((cols + 31) / 32 + 15) / 16 * 16; }

// ------------------------------------------------------------------ eight values of a row

// Eight consecutive elements as they lie in memory.  Rows need only their
// elements' alignment: the hardware splits a 16-byte access that crosses a line.
template <typename E>
struct Raw8 {
    static constexpr int N = 2 * (int)sizeof(typename E::st);
    uint32_t w[N];
    SPEC_DEVICE float get(int e) const
    {
        if constexpr (N == 8) return __uint_as_float(w[e]);
        return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    }
    SPEC_DEVICE void set(const float (&v)[8])
    {
        if constexpr (N == 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = (uint32_t)E::round(v[2 * e]) | (uint32_t)E::round(v[2 * e + 1]) << 16;
        }
    }
};
template <typename S>
struct __attribute__((packed, aligned(alignof(S)))) Bytes16 {
    uint32_t w[4];
};

// Elements c .. c + 7 of a row of d >= 8, those past d zero, in two parts.  The first
// only loads, without a branch, so that the loads of several rows can be on their
// way at once: where d ends before c + 8, the row's last eight.  The second, once
// they are there, moves them to their places.
template <typename E>
SPEC_DEVICE Raw8<E> load8_start(const typename E::st *__restrict__ row, int c, int d)
{
    Raw8<E> r;
    const typename E::st *p = row + min(c, d - 8);
#pragma unroll
    for (int i = 0; i < Raw8<E>::N / 4; ++i) {
        const Bytes16<typename E::st> b = reinterpret_cast<const Bytes16<typename E::st> *>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[4 * i + j] = b.w[j];
    }
    return r;
}

template <typename E>
SPEC_DEVICE void load8_end(Raw8<E> &r, int c, int d)
{
    constexpr int N = Raw8<E>::N, ONE = N / 4;  // words; words of two elements
    const int by = c + 8 - d;
    if (d % 8 != 0) {  // (the same in all lanes)
        const int down = by > 0 ? by : 0;
#pragma unroll
        for (int k = 2; k >= 1; --k)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t up = i + k * ONE < N ? r.w[i + k * ONE < N ? i + k * ONE : 0] : 0;
                r.w[i] = down & 2 * k ? up : r.w[i];
            }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t up = i + 1 < N ? r.w[i + 1 < N ? i + 1 : 0] : 0;
            r.w[i] = !(down & 1) ? r.w[i] : N == 8 ? up : __builtin_amdgcn_alignbit(up, r.w[i], 16);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = by < 8 ? r.w[i] : 0;
}

// the same of a row of d < 8: element by element
template <typename E>
SPEC_DEVICE Raw8<E> load8_tiny(const typename E::st *__restrict__ row, int c, int d)
{
    Raw8<E> r;
#pragma unroll
    for (int i = 0; i < Raw8<E>::N; ++i) r.w[i] = 0;
#pragma unroll
    for (int e = 0; e < 7; ++e) {
        if (c != 0 || e >= d) continue;
        if constexpr (Raw8<E>::N == 8)
            r.w[e] = __float_as_uint(row[e]);
        else
            r.w[e >> 1] |= (uint32_t)row[e] << 16 * (e & 1);
    }
    return r;
}

template <typename E>
SPEC_DEVICE Raw8<E> load8(const typename E::st *__restrict__ row, int c, int d)
{
    if (d < 8) return load8_tiny<E>(row, c, d);
    Raw8<E> r = load8_start<E>(row, c, d);
    load8_end<E>(r, c, d);
    return r;
}

template <typename E>
SPEC_DEVICE void store8(typename E::st *__restrict__ row, int64_t c, int64_t d, const Raw8<E> &r)
{
    using st = typename E::st;
    if (c + 8 <= d) {
#pragma unroll
        for (int i = 0; i < Raw8<E>::N / 4; ++i) {
            Bytes16<st> b;
#pragma unroll
            for (int j = 0; j < 4; ++j) b.w[j] = r.w[4 * i + j];
            reinterpret_cast<Bytes16<st> *>(row + c)[i] = b;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < d) {
                if constexpr (sizeof(st) == 4)
                    row[c + e] = __uint_as_float(r.w[e]);
                else
                    row[c + e] = (st)(r.w[e >> 1] >> 16 * (e & 1));
            }
    }
}

// ------------------------------------------------------------------ scales

// The block's byte from the bits of the magnitudes of this lane's eight values
// (their maximum); the same in the block's four lanes.
template <int FMT>
SPEC_DEVICE int mx_scale(uint32_t top)
{
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));  // lane ^ 1
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, false));  // lane ^ 2
    const int e = (int)(top >> 23);
    if (e == 255) return MX_NAN;
    const uint32_t m = top & 0x7FFFFFu;
    // (a subnormal magnitude is m 2^-149, without the leading one)
    return FMT == SPEC_MX_INT8 ? min(e + (m >= (e > 0 ? 0x7F0000u : 0x7F8000u)), 254) : min(max(e - 2 + (m >= 0x600000u), 0), 252);
}

// the largest magnitude's bits of eight values
template <typename E>
SPEC_DEVICE uint32_t mx_top(const Raw8<E> &r)
{
    if constexpr (Raw8<E>::N == 8) {
        uint32_t t = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) t = max(t, r.w[e] & 0x7FFFFFFFu);
        return t;
    } else {
        typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
        u16x2_t t = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2_t, r.w[i] & 0x7FFF7FFFu));
        return (uint32_t)max(t[0], t[1]) << 16;
    }
}

// ------------------------------------------------------------------ codes

// eight codes, one byte each
template <typename E>
SPEC_DEVICE uint2 mx_encode_int8(const Raw8<E> &r, int b)
{
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = __builtin_amdgcn_fmed3f(__builtin_ldexpf(r.get(e), 133 - b), -127.f, 127.f);
        c[e] = __float_as_uint(a + 0x1.8p23f);  // the nearest integer, ties to even, in the low byte
    }
    uint2 q;
    q.x = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u), __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), 0x05040100u);
    q.y = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[7], c[6], 0x0C0C0400u), __builtin_amdgcn_perm(c[5], c[4], 0x0C0C0400u), 0x05040100u);
    if (b == MX_NAN) q = make_uint2(0, 0);
    return q;
}

// eight codes, the even one of two in the low half of a byte; the conversion
// rounds to nearest even and cuts off at 6
template <typename E>
SPEC_DEVICE uint32_t mx_encode_fp4(const Raw8<E> &r, int b)
{
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = __builtin_ldexpf(r.get(e), 127 - b);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a[0], a[1], 1.f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a[2], a[3], 1.f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a[4], a[5], 1.f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a[6], a[7], 1.f, 3);
    return b == MX_NAN ? 0 : q;
}

// 2^(b - 133), the worth of an INT8 code's unit; NaN for 255
SPEC_DEVICE float mx_unit_int8(int b)
{
    return b == MX_NAN ? __builtin_nanf("") : __int_as_float(b >= 7 ? (b - 6) << 23 : 1 << (b + 16));
}

SPEC_DEVICE void mx_decode_int8(uint32_t q0, uint32_t q1, float unit, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)((e < 4 ? q0 : q1) >> 8 * (e & 3)) * unit;
}

// The conversions from FP4 take b as the exponent bits of an f32: bytes 0 (2^-127) to
// 254 and NaN for 255, exact as far as f32 (bf16) holds the values.
SPEC_DEVICE float mx_factor(int b) { return __int_as_float(b << 23); }

typedef float f32x2_t __attribute__((ext_vector_type(2)));

SPEC_DEVICE void mx_decode_fp4(uint32_t q, float f, float (&v)[8])
{
    f32x2_t p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 3);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e >> 1][e & 1];
}

// the same as eight bf16
SPEC_DEVICE bf16x8_t mx_decode_fp4_bf16(uint32_t q, float f)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, f, 3);
    return __builtin_shufflevector(__builtin_shufflevector(a, b, 0, 1, 2, 3), __builtin_shufflevector(c, d, 0, 1, 2, 3), 0, 1, 2,
                                   3, 4, 5, 6, 7);
}

// values exact in type E (eight bits or fewer) without rounding: bf16 takes the upper halves
template <typename E>
SPEC_DEVICE Raw8<E> mx_raw(const float (&v)[8])
{
    Raw8<E> r;
    if constexpr (Raw8<E>::N == 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r.w[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1]), __float_as_uint(v[2 * i]), 0x07060302u);
    }
    return r;
}
