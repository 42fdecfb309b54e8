// Products with microscaled matrices, gfx950 (the format: mx.h; the tiles: mm.h).
//
//   linear   Y[t][n] = sum_k X[t][k] W[n][k]       W in FP4, X bf16 or f32
//   product  the same, X in FP4 too
//   wgrad    dW[n][k] = beta dW[n][k] + sum_t dY[t][n] X[t][k]     X in INT8, dY bf16 or f32
//
// product: both operands go to the scaled MFMA as they lie in memory, 32 codes and
// their byte per lane (k_mx_fp4).  8192 x 14336 x 4096 takes 299 us, 3.2 PFLOP/s, in seven
// rounds of 256 tiles.  From k = 4096 on every step of 256 k adds 1.9 us to a tile (the bf16
// core's step of 64 k, as many bytes and MFMA cycles, 1.6); the 16 steps here are 30 of a tile's
// 41 us.  The other 11 are its first copies and its results, which nothing overlaps with one
// workgroup to a CU: the share that the bf16 core spreads over four times as many steps.
// The MFMAs are busy for 0.37 of the cycles (bf16 0.62), at 2.0 GHz (1.9).  32768 k reach
// 4.4 PFLOP/s.  Unpacked to bf16 first it took 749 us.
//
// linear, few rows of X (a decode step): bound by reading W and by X's fragments, which
// every workgroup reads from the L2 (k_mx_few).  1, 8, 16, 32 and 64 x 4096 x 4096 bf16 take
// 7.1, 7.0, 7.7, 11.9 and 20.4 us with W taken in turn from 600 MB of matrices, as the layers
// of a model are, and 4.3, 5.6, 6.9, 10.7 and 19.2 us where the same W stays in the caches;
// 8 x 14336 x 4096 13.2 us, 2.4 TB/s of W, and 11.0; f32 26.0 and 24.6.  Requesting W or X a
// step ahead, X in whole 64-byte pieces turned between lanes, and 4 or 16 waves instead of 8
// changed these by less than 5 %.
//
// linear of more rows, and wgrad: a microscaled value has at most seven significant
// bits and a power of two, so it is exact in bf16.  The packed operand is unpacked into
// the workspace (26 and 33 us for 14336 x 4096 FP4, 16384 x 4096 int8) and the products are
// those of mm.h, bf16 or f32 MFMA with f32 sums: 2047 x 4096 x 14336 197 us, 1220 TFLOP/s (one
// round of 256 tiles, k in two shares, and 14 us to join them; unsplit 192 x 192 tiles
// took 244), 224 us the whole call; 16384 x 4096 x 4096 468 us, 1170 TFLOP/s, 474 us the whole
// call.  (Kernels: medians of a trace, whose passes lie apart; calls: among others.)
//
//   k_mx_pack   X or dY with 16-byte rows (only where they have none)
//   k_mx_mm     bf16 or f32 tiles
//   k_mx_fp4    FP4 tiles
//   k_mx_few    few rows of X
//   k_mx_join   the sums of shares of k
#include <algorithm>

#include "mx.h"

namespace {

inline int64_t cdiv_h(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up_h(int64_t a, int64_t b) { return cdiv_h(a, b) * b; }

// rows of c elements to rows of 16-byte multiples, zero past c
template <typename E>
__global__ __launch_bounds__(256) void k_mx_pack(const typename E::st *__restrict__ X, int64_t rows, int64_t c,
                                                 int64_t ldx, int64_t eights, typename E::st *__restrict__ P)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * eights; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / eights, e = 8 * (i % eights);
        store8<E>(P + r * eights * 8, e, eights * 8, load8<E>(X + r * ldx, (int)e, (int)c));
    }
}

// What a product writes: O[q][p] (+ beta O), or for one of several shares of k its sums.
struct MmOut {
    void *out;
    int64_t ldo;
    float beta;
    float *part;  // [share][rows][ldpart]
    int64_t ldpart, rows;
    int ways;
};

template <typename E>
SPEC_DEVICE void put4(typename E::st *o, const float (&v)[4], float beta, int left, bool vec)
{
    if (vec && left >= 4) {
        Vec4<E> r;
        if (beta != 0.f) r = *reinterpret_cast<const Vec4<E> *>(o);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.v[e] = E::round(beta != 0.f ? v[e] + beta * E::wide(r.v[e]) : v[e]);
        *reinterpret_cast<Vec4<E> *>(o) = r;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) o[e] = E::round(beta != 0.f ? v[e] + beta * E::wide(o[e]) : v[e]);
    }
}

// the tile at (p0, q0), of which plim x qlim lie inside: to the output, or to the share's sums
template <typename EO, typename M, typename L>
SPEC_DEVICE void put_tile(M &mm, const L &lds, const MmOut &o, int64_t p0, int64_t q0, int plim, int qlim, int share, int vec)
{
    if (o.ways > 1) {
        float *part = o.part + (share * o.rows + q0) * o.ldpart + p0;
        mm.each4(lds, [&](int p, int q, float (&v)[4]) {
            if (q < qlim && p < plim)  // (ldpart is a multiple of 4: a group of four lies in its row)
                *reinterpret_cast<float4 *>(part + q * o.ldpart + p) = make_float4(v[0], v[1], v[2], v[3]);
        });
    } else {
        typename EO::st *out = (typename EO::st *)o.out + q0 * o.ldo + p0;
        mm.each4(lds, [&](int p, int q, float (&v)[4]) {
            if (q < qlim && p < plim) put4<EO>(out + q * o.ldo + p, v, o.beta, plim - p, vec != 0);
        });
    }
}

// acc[q][p] = sum over k of P(p, k) Q(q, k), both operands with k contiguous (S false) or slow
template <typename E, typename C, bool S>
__global__ MM_BOUNDS(C) void k_mx_mm(const typename E::st *__restrict__ P, int64_t ldp, int64_t np,
                                     const typename E::st *__restrict__ Q, int64_t ldq, int64_t nq, int64_t K,
                                     int tp_n, int tq_n, MmOut o, int vec)
{
    using M = Mm<E, C, S, S>;
    MM_STAGES(M);
    const int tiles = tp_n * tq_n, share = (int)(blockIdx.x / (unsigned)tiles);
    int tp, tq;
    mm_tile(blockIdx.x % (unsigned)tiles, tp_n, tq_n, tp, tq);
    const int64_t p0 = (int64_t)tp * C::BP, q0 = (int64_t)tq * C::BQ;
    const int64_t per = round_up((K + o.ways - 1) / o.ways, 64), kb = share * per, ke = min(K, kb + per);
    const int64_t kp = S ? ke : min(round_up(K, M::EPC), round_up(ke, M::EPC));
    const MmSrc sp{(const char *)(S ? P + p0 : P + p0 * ldp), ldp * M::SZ, (int)min<int64_t>(C::BP, np - p0), kp};
    const MmSrc sq{(const char *)(S ? Q + q0 : Q + q0 * ldq), ldq * M::SZ, (int)min<int64_t>(C::BQ, nq - q0), kp};
    M mm;
    mm.run(sp, sq, kb, ke, lds);
    put_tile<E>(mm, lds, o, p0, q0, sp.lim, sq.lim, share, vec);
}

// ------------------------------------------------------------------ both operands in FP4
//
// A K-step is 128 bytes of codes of every row, 256 values; a lane's 16-byte chunk of
// a fragment is one block of 32, so the MFMA's scale of a lane is that block's byte.
// Codes are staged as bytes by the tiles of mm.h.  Scales, 8 bytes per row and step, come
// with them: a turn of the stages takes at most one 16-byte copy per thread (two steps
// of one row), into one of two buffers, requested a turn ahead.

struct ElByte {
    using st = uint8_t;
};
struct MxTile64 {
    static constexpr int BP = 64, BQ = 64, WP = 1, WQ = 1, WK = 4, STAGES = 2, NT = 256;
};
struct MxTile32 {
    static constexpr int BP = 32, BQ = 32, WP = 1, WQ = 1, WK = 4, STAGES = 4, NT = 256;
};

struct MxSrc {
    MmSrc codes;      // K in bytes
    const char *s;    // scales of its first row
    int64_t lds;
    int row_bytes;    // of scales, a multiple of 16
};

template <typename C>
struct MmFp4 : Mm<ElByte, C, false, false> {
    using M = Mm<ElByte, C, false, false>;
    static constexpr int S = C::STAGES, BK = M::BK, KW = M::KW, WK = C::WK, MI = M::MI, NI = M::NI;
    static constexpr int CPR = S / 2;  // 16-byte chunks of scales per row and turn
    static constexpr int CHUNKS = C::BP * CPR;  // of each operand
    static_assert(C::BP == C::BQ && 2 * CHUNKS <= C::NT && CHUNKS % 64 == 0, "one chunk per thread, whole waves");
    static constexpr int SCALE_BYTES = C::NT * 16;
    typedef int i32x8_t __attribute__((ext_vector_type(8)));

    // of the rows of a fragment in one step: byte 0 for the first of two quarters of
    // the step, byte 2 for the second (WK > 1: the wave's quarter in byte 0)
    struct Scales {
        uint32_t a[MI][WK > 1 ? 1 : 2], b[NI][WK > 1 ? 1 : 2];
    };
    static SPEC_DEVICE void scales_of(const char *sc, int row, int step, int kw, int lane, uint32_t (&o)[WK > 1 ? 1 : 2])
    {
        const char *p = sc + ((row + (lane & 31)) * CPR + step / 2) * 16 + step % 2 * 8;
        const int h = lane >> 5;
        if constexpr (WK > 1) {
            o[0] = *reinterpret_cast<const uint8_t *>(p + 2 * kw + h);
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            o[0] = v.x >> 8 * h;
            o[1] = v.y >> 8 * h;
        }
    }
    static SPEC_DEVICE void scales(Scales &o, const char *sc, int p0, int q0, int step, int kw, int lane)
    {
#pragma unroll
        for (int m = 0; m < MI; ++m) scales_of(sc, p0 + 32 * m, step, kw, lane, o.a[m]);
#pragma unroll
        for (int n = 0; n < NI; ++n) scales_of(sc, C::BP + q0 + 32 * n, step, kw, lane, o.b[n]);
    }
    template <int KK>
    SPEC_DEVICE void multiply(const typename M::Frags &f, const Scales &sc)
    {
        constexpr int R = WK > 1 ? 0 : KK >> 1, SEL = WK > 1 ? 0 : 2 * (KK & 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                const f32x4_t a = f.a[m].x, b = f.b[n].x;
                i32x8_t x{}, y{};
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __float_as_int(a[i]), y[i] = __float_as_int(b[i]);
                this->acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, this->acc[m][n], 4, 4, SEL,
                                                                                 (int)sc.a[m][R], SEL, (int)sc.b[n][R]);
            }
        __builtin_amdgcn_sched_barrier(0);
    }

    // acc = sum over the codes' bytes [kb, K) (kb a multiple of two steps)
    SPEC_DEVICE void run(const MxSrc &P, const MxSrc &Q, int64_t kb, int64_t K, const typename M::Lds &s, char *sc0, char *sc1)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int p0 = M::wave_p0(wave), q0 = M::wave_q0(wave), kw = wave / (C::WP * C::WQ) * KW;
        uint32_t vp[M::PL], vq[M::QL];
        int kp, kq;
        M::template offsets<C::BP, false>(P.codes, vp, kp);
        M::template offsets<C::BQ, false>(Q.codes, vq, kq);
        // this thread's chunk of scales: the first waves P's rows, then Q's (and none for what is left)
        const MxSrc &X = __builtin_amdgcn_readfirstlane(wave) < CHUNKS / 64 ? P : Q;
        const int at = (int)threadIdx.x % CHUNKS, row = at / CPR, chunk = at % CPR * 16;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void *)X.s, 0, 0x7FFFFFF0, 0x00020000);
        const uint32_t vs = row < X.codes.lim && (int)threadIdx.x < 2 * CHUNKS ? (uint32_t)(row * (int)X.lds + chunk) : M::OUT;
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) this->acc[m][n][e] = 0.f;
        if (kb < K) {
            auto request = [&](int64_t k, int i) {
                M::template stage<false>(P.codes, vp, kp, k, s.p[i]);
                M::template stage<false>(Q.codes, vq, kq, k, s.q[i]);
            };
            // of the turn whose first step is at byte k: a scale byte stands for 16 of codes
            auto request_scales = [&](int64_t k, char *sc) {
                const int off = (int)(k / 16);
                const uint32_t past = off + chunk < X.row_bytes ? 0u : 0x80000000u;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)(sc + ((int)threadIdx.x & ~63) * 16), 16,
                                                         (int)(vs | past), off, 0, 0);
            };
            request_scales(kb, sc0);
            mm_for<0, S>([&](auto I) { request(kb + decltype(I)::value * BK, decltype(I)::value); });
            typename M::Frags f[2];
            Scales sc[2];
            M::template landed<(S - 1) * (M::PL + M::QL)>();
            M::fetch(f[0], s.p[0], s.q[0], p0, q0, kw, lane);
            scales(sc[0], sc0, p0, q0, 0, kw, lane);
            for (int64_t k0 = kb; k0 < K; k0 += 2 * S * BK) {
                mm_for<0, 2 * S>([&](auto I) {
                    constexpr int i = decltype(I)::value, st = i % S, j = (i + 1) % S;
                    if (MI * NI <= 4 && i > 0 && k0 + i * BK >= K) return;
                    mm_for<0, KW>([&](auto Q_) {
                        constexpr int kk = decltype(Q_)::value, cur = (i * KW + kk) & 1;
                        if constexpr (kk < KW - 1) {
                            M::fetch(f[cur ^ 1], s.p[st], s.q[st], p0, q0, kw + kk + 1, lane);
                        } else {
                            M::template landed<(S - 2) * (M::PL + M::QL)>();
                            // before its turn's first step, and so landed with it
                            if constexpr (st == 0) request_scales(k0 + (i + S) * BK, i / S ? sc0 : sc1);
                            request(k0 + (i + S) * BK, st);
                            M::fetch(f[cur ^ 1], s.p[j], s.q[j], p0, q0, kw, lane);
                            scales(sc[(i & 1) ^ 1], (i + 1) / S % 2 ? sc1 : sc0, p0, q0, j, kw, lane);
                        }
                        multiply<kk>(f[cur], sc[i & 1]);
                    });
                });
            }
            M::template landed<0>();
        }
        if constexpr (WK > 1) this->join(s);
    }
};

template <typename EO, typename C>
__global__ MM_BOUNDS(C) void k_mx_fp4(const uint8_t *__restrict__ P, const uint8_t *__restrict__ SP, int64_t ldp,
                                      int64_t ldsp, int64_t np, const uint8_t *__restrict__ Q,
                                      const uint8_t *__restrict__ SQ, int64_t ldq, int64_t ldsq, int64_t nq, int64_t K,
                                      int row_bytes, int tp_n, int tq_n, MmOut o, int vec)
{
    using X = MmFp4<C>;
    using M = typename X::M;
    MM_STAGES(M);
    __shared__ __attribute__((aligned(16))) char sc0[X::SCALE_BYTES], sc1[X::SCALE_BYTES];
    const int tiles = tp_n * tq_n, share = (int)(blockIdx.x / (unsigned)tiles);
    int tp, tq;
    mm_tile(blockIdx.x % (unsigned)tiles, tp_n, tq_n, tp, tq);
    const int64_t p0 = (int64_t)tp * C::BP, q0 = (int64_t)tq * C::BQ;
    const int64_t per = round_up((K + o.ways - 1) / o.ways, 256), kb = share * per, ke = min(K, kb + per);
    const MxSrc sp{{(const char *)(P + p0 * ldp), ldp, (int)min<int64_t>(C::BP, np - p0), ke}, (const char *)(SP + p0 * ldsp), ldsp, row_bytes};
    const MxSrc sq{{(const char *)(Q + q0 * ldq), ldq, (int)min<int64_t>(C::BQ, nq - q0), ke}, (const char *)(SQ + q0 * ldsq), ldsq, row_bytes};
    X mm;
    mm.run(sp, sq, kb, ke, lds, sc0, sc1);
    put_tile<EO>(mm, lds, o, p0, q0, sp.codes.lim, sq.codes.lim, share, vec);
}

// ------------------------------------------------------------------ few rows of X
//
// One decode step's tokens: bound by reading W, each byte of which is used once.  A
// workgroup takes 16 RT rows of W (the MFMA's rows; the tokens are its columns, 16 TT of
// them), its waves steps of 256 k in turn, and joins their sums through LDS.  A lane
// holds blocks of W as they lie in memory (16 bytes), unpacks eight values of one to a bf16
// fragment with one conversion per two values, scale included, and takes the same eight
// k of its token from X (L2).
constexpr int FEW_WAVES = 8;

template <typename E, int RT, int TT>
__global__ __launch_bounds__(64 * FEW_WAVES) void k_mx_few(const uint8_t *__restrict__ W, const uint8_t *__restrict__ SW,
                                                           int64_t ldw, int64_t lds, int64_t N,
                                                           const typename E::st *__restrict__ X, int64_t ldx, int64_t T,
                                                           int64_t K, typename E::st *__restrict__ Y, int64_t ldy, int vec)
{
    using st = typename E::st;
    __shared__ float4 red[FEW_WAVES][RT * TT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT), blocks = (K + 31) / 32;
    const uint8_t *w[RT], *sw[RT];
    const st *x[TT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {  // rows and tokens past the end repeat the last: their sums go nowhere
        const int64_t n = min(n0 + 16 * r + (lane & 15), N - 1);
        w[r] = W + n * ldw + 16 * g;
        sw[r] = SW + n * lds;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t] = X + min<int64_t>(16 * t + (lane & 15), T - 1) * ldx;
    f32x4_t acc[RT][TT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // 256 k from k0: two blocks per lane, 4 j + g of the eight
    const auto step = [&](int64_t k0, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        uint4 q[RT][2];
        uint2 s[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            s[r] = *reinterpret_cast<const uint2 *>(sw[r] + k0 / 32);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                q[r][j] = WHOLE || k0 / 32 + 4 * j + g < blocks ? *reinterpret_cast<const uint4 *>(w[r] + k0 / 2 + 64 * j)
                                                                : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            Raw8<E> xv[TT][4];
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = (int)k0 + 128 * j + 8 * i + 32 * g;
                    xv[t][i] = WHOLE ? load8_start<E>(x[t], k, k + 8) : load8<E>(x[t], k, (int)K);
                }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                int b = (int)((j ? s[r].y : s[r].x) >> 8 * g & 255);
                if (!WHOLE && k0 / 32 + 4 * j + g >= blocks) b = 0;
                const float f = mx_factor(b);
                const uint32_t qq[4] = {q[r][j].x, q[r][j].y, q[r][j].z, q[r][j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (sizeof(st) == 2) {
                        const bf16x8_t a = mx_decode_fp4_bf16(qq[i], f);
#pragma unroll
                        for (int t = 0; t < TT; ++t) {
                            const uint4 v = make_uint4(xv[t][i].w[0], xv[t][i].w[1], xv[t][i].w[2], xv[t][i].w[3]);
                            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, v), acc[r][t], 0, 0, 0);
                        }
                    } else {
                        float a[8];
                        mx_decode_fp4(qq[i], f, a);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
#pragma unroll
                            for (int t = 0; t < TT; ++t)
                                acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], xv[t][i].get(e), acc[r][t], 0, 0, 0);
                    }
                }
            }
        }
    };
    const int64_t whole = K / 256, steps = (K + 255) / 256;
    for (int64_t u = wave; u < whole; u += FEW_WAVES) step(u * 256, std::true_type{});
    if (steps > whole && whole % FEW_WAVES == wave) step(whole * 256, std::false_type{});

#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
            red[wave][r * TT + t][lane] = make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
    __syncthreads();
    for (int i = threadIdx.x; i < RT * TT * 64; i += 64 * FEW_WAVES) {
        const int tile = i >> 6, l = i & 63;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < FEW_WAVES; ++k) {
            const float4 a = red[k][tile][l];
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        }
        const int64_t n = n0 + 16 * (tile / TT) + 4 * (l >> 4), t = 16 * (tile % TT) + (l & 15);
        if (t < T && n < N) put4<E>(Y + t * ldy + n, v, 0.f, (int)min<int64_t>(4, N - n), vec != 0);
    }
}

template <typename EO>
__global__ __launch_bounds__(256) void k_mx_join(MmOut o, int64_t np, int vec)
{
    const int64_t fours = o.ldpart / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < o.rows * fours; i += (int64_t)gridDim.x * 256) {
        const int64_t q = i / fours, p = 4 * (i % fours);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int w = 0; w < o.ways; ++w) {
            const float4 a = *reinterpret_cast<const float4 *>(o.part + (w * o.rows + q) * o.ldpart + p);
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        }
        put4<EO>((typename EO::st *)o.out + q * o.ldo + p, v, o.beta, (int)min<int64_t>(4, np - p), vec != 0);
    }
}

// ------------------------------------------------------------------ sizes

constexpr int64_t PIECE_BYTES = (int64_t)256 << 20;  // of unpacked values at most, but no less than 256 rows of them
constexpr int64_t SPLIT_BYTES = (int64_t)64 << 20;   // of the shares' sums

// The tile and the shares of k of a bf16 or f32 product that take the least time: the
// busiest of 256 CUs at the core's rate (4.7 TFLOP/s a CU in bf16, 0.6 in f32, for the
// largest tile; per: the others' time per result, as in mm.h, the smallest's more, whose
// rounds are short here), a microsecond per round, and for shares of k their
// sums written and read again (8 TB/s, through the caches) and a launch.  Shares are of
// about 256 k or more.
struct MmPlan {
    int edge, ways;
};
template <typename E>
MmPlan mm_plan(int64_t np, int64_t nq, int64_t K)
{
    constexpr bool H = sizeof(typename E::st) == 2;
    const int edge[5] = {256, 192, 128, 64, 32};
    const double per[5] = {1.0, 1.1, H ? 1.28 : 1.03, H ? 2.1 : 1.14, 2.5};
    const double rate = (H ? 4.7e6 : 0.6e6) / 2;  // products of a CU per us
    const int64_t sums = 4 * up_h(np, 4) * std::max<int64_t>(nq, 1);
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>({cdiv_h(K, 256), SPLIT_BYTES / sums, 64}));
    MmPlan best{256, 1};
    double least = 0.0;
    for (int i = 0; i < (H ? 4 : 5); ++i)  // (in 16 bits the 64 x 64 tile is never slower than the 32 x 32)
        for (int w = 1; w <= most; ++w) {
            const int64_t tiles = cdiv_h(np, edge[i]) * cdiv_h(nq, edge[i]);
            // (of the smaller shapes two workgroups share a CU, and one alone takes as long)
            const double rounds = edge[i] > 128 ? (double)cdiv_h(tiles * w, 256) : 2.0 * cdiv_h(tiles * w, 512);
            double t = rounds * edge[i] * edge[i] * per[i] * (double)cdiv_h(K, w) / rate;
            t += (double)cdiv_h(tiles * w, edge[i] > 128 ? 256 : 512);  // a round's first copies and last stores
            if (w > 1) t += 3.0 + 2.0 * w * (double)sums / 8e6;
            if ((i == 0 && w == 1) || t < least) least = t, best = {edge[i], w};
        }
    return best;
}

template <typename E, typename F>
hipError_t with_tile(int edge, F &&f)
{
    switch (edge) {
    case 256: return f(Tile256{});
    case 192: return f(Tile192{});
    case 128: return f(Tile128{});
    case 64: return f(Tile64{});
    default:
        if constexpr (sizeof(typename E::st) == 4) return f(Tile32{});
        return hipErrorInvalidValue;  // (mm_plan gives no other)
    }
}

// FP4: as many shares as give every CU a tile of 64 x 64, of about 2048 k (eight steps) or
// more.  Shorter ones cost more in the second launch than they save: 333 x 1000 x 1000
// took 9.4 us in three shares, 6.1 in one.
int ways_of_fp4(int64_t N, int64_t T, int64_t K)
{
    const int64_t tiles = cdiv_h(N, 64) * cdiv_h(std::max<int64_t>(T, 1), 64);
    int64_t w = std::min<int64_t>(cdiv_h(256, tiles), cdiv_h(K, 2048));
    w = std::min<int64_t>(w, SPLIT_BYTES / (4 * up_h(N, 4) * std::max<int64_t>(T, 1)));
    return (int)std::max<int64_t>(1, std::min<int64_t>(w, 64));
}

template <typename E, bool S>
hipError_t product(hipStream_t stream, const typename E::st *P, int64_t ldp, int64_t np, const typename E::st *Q,
                   int64_t ldq, int64_t nq, int64_t K, void *out, int64_t ldo, float beta, float *part)
{
    using st = typename E::st;
    const int vec = (uintptr_t)out % (4 * sizeof(st)) == 0 && ldo % 4 == 0;
    const MmPlan plan = mm_plan<E>(np, nq, K);
    MmOut o{out, ldo, beta, part, up_h(np, 4), nq, plan.ways};
    const hipError_t e = with_tile<E>(plan.edge, [&](auto c) {
        using C = decltype(c);
        const int tp = (int)cdiv_h(np, C::BP), tq = (int)cdiv_h(nq, C::BQ);
        hipLaunchKernelGGL((k_mx_mm<E, C, S>), dim3((unsigned)((int64_t)tp * tq * o.ways)), dim3(C::NT), 0, stream, P,
                           ldp, np, Q, ldq, nq, K, tp, tq, o, vec);
        return hipGetLastError();
    });
    if (e != hipSuccess || o.ways == 1) return e;
    hipLaunchKernelGGL(k_mx_join<E>, dim3((unsigned)std::min<int64_t>(cdiv_h(o.rows * o.ldpart / 4, 256), 4096)), dim3(256),
                       0, stream, o, np, vec);
    return hipGetLastError();
}

// Packed matrices are unpacked a piece of rows (linear) or of columns (wgrad, whose rows
// are the sums' k) at a time; rows of up_h(c, 32) values.
int64_t piece_rows(int64_t rows, int64_t row_bytes)
{
    return std::min(rows, std::max<int64_t>(256, PIECE_BYTES / row_bytes / 256 * 256));
}

template <typename E>
bool direct(const void *X, int64_t ldx, int64_t c)
{
    const int64_t es = sizeof(typename E::st);
    return (uintptr_t)X % 16 == 0 && ldx * es % 16 == 0 && c * es % 16 == 0;
}

template <typename E>
hipError_t pack(hipStream_t stream, const typename E::st *X, int64_t rows, int64_t c, int64_t ldx, typename E::st *P)
{
    const int64_t eights = up_h(c, 32) / 8;
    hipLaunchKernelGGL(k_mx_pack<E>, dim3((unsigned)std::min<int64_t>(cdiv_h(rows * eights, 256), 1 << 16)), dim3(256), 0,
                       stream, X, rows, c, ldx, eights, P);
    return hipGetLastError();
}

spec_mx rows_from(const spec_mx *m, int64_t row)
{
    spec_mx r = *m;
    r.q = (uint8_t *)m->q + row * m->ldq;
    r.s = (uint8_t *)m->s + row * m->lds;
    return r;
}

// X of up to this many rows goes by k_mx_few: 64 rows of 8192 x 8192 bf16 take 40 us, 65 by
// the unpacked product 59; of 2048 x 2048 f32 18 and 32.
constexpr int64_t FEW_ROWS = 64;

constexpr int64_t MOST_T = 65536;  // rows of X per launch

struct LinearPlan {
    int64_t kp, wrows, w, x, part, total;  // bytes into the workspace
};
LinearPlan linear_plan(int64_t T, int64_t N, int64_t K, int64_t es)
{
    LinearPlan p{};
    if (T <= FEW_ROWS) {
        p.total = 256;
        return p;
    }
    p.kp = up_h(K, 32);
    p.wrows = piece_rows(N, p.kp * es);
    const int64_t t = std::min(T, MOST_T);
    p.w = 0;
    p.x = up_h(p.wrows * p.kp * es, 256);
    p.part = p.x + up_h(std::max<int64_t>(t, 1) * p.kp * es, 256);
    p.total = p.part + SPLIT_BYTES;
    return p;
}

template <typename E>
hipError_t linear(hipStream_t stream, const void *X, int64_t ldx, int64_t T, int64_t N, int64_t K, const spec_mx *W, void *Y,
                  int64_t ldy, char *ws)
{
    using st = typename E::st;
    constexpr int t = sizeof(st) == 2 ? SPEC_BF16 : SPEC_F32;
    const LinearPlan p = linear_plan(T, N, K, sizeof(st));
    st *const wv = (st *)(ws + p.w), *const xv = (st *)(ws + p.x);
    const bool in_place = direct<E>(X, ldx, K);
    for (int64_t n = 0; n < N; n += p.wrows) {
        const int64_t nn = std::min(p.wrows, N - n);
        const spec_mx wn = rows_from(W, n);
        hipError_t e = launch_mx_dequantize(stream, &wn, nn, K, p.kp, wv, t, p.kp);
        for (int64_t t0 = 0; t0 < T && e == hipSuccess; t0 += MOST_T) {
            const int64_t tn = std::min(MOST_T, T - t0);
            const st *x = (const st *)X + t0 * ldx;
            if (!in_place) e = pack<E>(stream, x, tn, K, ldx, xv);
            if (e == hipSuccess)
                e = product<E, false>(stream, wv, p.kp, nn, in_place ? x : xv, in_place ? ldx : p.kp, tn, K,
                                         (st *)Y + t0 * ldy + n, ldy, 0.f, (float *)(ws + p.part));
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

struct WgradPlan {
    int64_t cols, np, x, dy, part, total;
};
WgradPlan wgrad_plan(int64_t T, int64_t N, int64_t K, int64_t es)
{
    WgradPlan p{};
    const int64_t Tn = std::max<int64_t>(T, 1);
    p.cols = std::min<int64_t>(std::max<int64_t>(256, PIECE_BYTES / (Tn * es) / 256 * 256), MOST_T);
    p.cols = std::min(p.cols, up_h(K, 32));
    p.np = up_h(N, 32);
    p.x = 0;
    p.dy = up_h(Tn * p.cols * es, 256);
    p.part = p.dy + up_h(Tn * p.np * es, 256);
    p.total = p.part + SPLIT_BYTES;
    return p;
}

template <typename E>
hipError_t wgrad(hipStream_t stream, const void *dY, int64_t ldy, int64_t T, int64_t N, int64_t K, const spec_mx *X,
                 float beta, void *dW, int64_t lddw, char *ws)
{
    using st = typename E::st;
    constexpr int t = sizeof(st) == 2 ? SPEC_BF16 : SPEC_F32;
    const WgradPlan p = wgrad_plan(T, N, K, sizeof(st));
    st *const xv = (st *)(ws + p.x);
    const st *dy = (const st *)dY;
    hipError_t e = hipSuccess;
    if (T > 0 && !direct<E>(dY, ldy, N)) {
        e = pack<E>(stream, dy, T, N, ldy, (st *)(ws + p.dy));
        dy = (const st *)(ws + p.dy);
        ldy = p.np;
    }
    for (int64_t c = 0; c < K && e == hipSuccess; c += p.cols) {
        const int64_t cn = std::min(p.cols, K - c);
        spec_mx x = *X;
        x.q = (uint8_t *)X->q + c;
        x.s = (uint8_t *)X->s + c / 32;
        e = launch_mx_dequantize(stream, &x, T, cn, up_h(cn, 32), xv, t, p.cols);
        if (e == hipSuccess)
            e = product<E, true>(stream, xv, p.cols, cn, dy, ldy, N, T, (st *)dW + c, lddw, beta, (float *)(ws + p.part));
    }
    return e;
}

template <typename E>
hipError_t few(hipStream_t stream, const void *X, int64_t ldx, int64_t T, int64_t N, int64_t K, const spec_mx *W, void *Y,
               int64_t ldy)
{
    using st = typename E::st;
    const int vec = (uintptr_t)Y % (4 * sizeof(st)) == 0 && ldy % 4 == 0;
    const auto go = [&](auto rt, auto tt) {
        constexpr int RT = decltype(rt)::value, TT = decltype(tt)::value;
        hipLaunchKernelGGL((k_mx_few<E, RT, TT>), dim3((unsigned)cdiv_h(N, 16 * RT)), dim3(64 * FEW_WAVES), 0, stream,
                           (const uint8_t *)W->q, (const uint8_t *)W->s, W->ldq, W->lds, N, (const st *)X, ldx, T, K, (st *)Y,
                           ldy, vec);
        return hipGetLastError();
    };
    // Row tiles of a workgroup share the fragments of X, whose reads from the L2 cost more than
    // W's, as long as most CUs still get a workgroup: one, two and four tiles take 16.0, 12.4
    // and 11.0 us for 8 x 14336 x 4096 bf16 (896, 448 and 224 workgroups).
    const auto rows = [&](auto tt) {
        return N >= 64 * 208   ? go(std::integral_constant<int, 4>{}, tt)
               : N >= 32 * 208 ? go(std::integral_constant<int, 2>{}, tt)
                               : go(std::integral_constant<int, 1>{}, tt);
    };
    return T <= 16 ? rows(std::integral_constant<int, 1>{})
           : T <= 32 ? rows(std::integral_constant<int, 2>{})
                     : rows(std::integral_constant<int, 4>{});
}

// The tile whose busiest CU has least to do.  per: time per result against the largest
// tile's, the 16-bit core's ratios (steps are as many bytes and the rate follows the copies).
int edge_of_fp4(int64_t N, int64_t T, int ways)
{
    const int edge[4] = {256, 128, 64, 32};
    const double per[4] = {1.0, 1.3, 2.1, 6.0};
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < 4; ++i) {
        const double t = (double)cdiv_h(cdiv_h(N, edge[i]) * cdiv_h(T, edge[i]) * ways, 256) * edge[i] * edge[i] * per[i];
        if (i == 0 || t < least) least = t, best = i;
    }
    return edge[best];
}

template <typename F>
hipError_t with_tile4(int edge, F &&f)
{
    switch (edge) {
    case 256: return f(Tile256{});
    case 128: return f(Tile128{});
    case 64: return f(MxTile64{});
    default: return f(MxTile32{});
    }
}

template <typename EO>
hipError_t product4(hipStream_t stream, const spec_mx *X, const spec_mx *W, int64_t T, int64_t N, int64_t K, void *Y,
                    int64_t ldy, char *ws)
{
    using st = typename EO::st;
    const int vec = (uintptr_t)Y % (4 * sizeof(st)) == 0 && ldy % 4 == 0;
    for (int64_t t0 = 0; t0 < T; t0 += MOST_T) {
        const int64_t tn = std::min(MOST_T, T - t0);
        const spec_mx x = rows_from(X, t0);
        MmOut o{(st *)Y + t0 * ldy, ldy, 0.f, (float *)ws, up_h(N, 4), tn, ways_of_fp4(N, tn, K)};
        hipError_t e = with_tile4(edge_of_fp4(N, tn, o.ways), [&](auto c) {
            using C = decltype(c);
            const int tp = (int)cdiv_h(N, C::BP), tq = (int)cdiv_h(tn, C::BQ);
            hipLaunchKernelGGL((k_mx_fp4<EO, C>), dim3((unsigned)((int64_t)tp * tq * o.ways)), dim3(C::NT), 0, stream,
                               (const uint8_t *)W->q, (const uint8_t *)W->s, W->ldq, W->lds, N, (const uint8_t *)x.q,
                               (const uint8_t *)x.s, x.ldq, x.lds, tn, mx_code_row(SPEC_MX_FP4, K), (int)mx_scale_row(K), tp,
                               tq, o, vec);
            return hipGetLastError();
        });
        if (e == hipSuccess && o.ways > 1) {
            hipLaunchKernelGGL(k_mx_join<EO>, dim3((unsigned)std::min<int64_t>(cdiv_h(o.rows * o.ldpart / 4, 256), 4096)),
                               dim3(256), 0, stream, o, N, vec);
            e = hipGetLastError();
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename E>
void plan(int op, int64_t T, int64_t N, int64_t K, int *edge, int *shares)
{
    constexpr int64_t es = sizeof(typename E::st);
    MmPlan p;
    if (op == SPEC_MX_OP_LINEAR && T <= FEW_ROWS)
        p = {16, 1};
    else if (op == SPEC_MX_OP_LINEAR)
        p = mm_plan<E>(linear_plan(T, N, K, es).wrows, std::min(T, MOST_T), K);
    else
        p = mm_plan<E>(std::min(wgrad_plan(T, N, K, es).cols, K), N, T);
    *edge = p.edge, *shares = p.ways;
}

}  // namespace

void mx_plan(int op, int64_t T, int64_t N, int64_t K, int t, int *edge, int *shares)
{
    if (op == SPEC_MX_OP_PRODUCT) {
        const int64_t tn = std::min(T, MOST_T);
        *shares = ways_of_fp4(N, tn, K);
        *edge = edge_of_fp4(N, tn, *shares);
    } else if (t == SPEC_BF16) {
        plan<ElBF16>(op, T, N, K, edge, shares);
    } else {
        plan<ElF32>(op, T, N, K, edge, shares);
    }
}

size_t mx_linear_workspace_bytes(int64_t T, int64_t N, int64_t K, int t)
{
    return (size_t)linear_plan(T, N, K, t == SPEC_BF16 ? 2 : 4).total;
}

size_t mx_product_workspace_bytes(int64_t T, int64_t N, int64_t K)
{
    const int ways = ways_of_fp4(N, std::min(T, MOST_T), K);  // (a last, smaller piece may take more: SPLIT_BYTES)
    return T > MOST_T ? (size_t)SPLIT_BYTES : ways > 1 && T > 0 ? (size_t)ways * T * up_h(N, 4) * 4 : 256;
}

size_t mx_weight_grad_workspace_bytes(int64_t T, int64_t N, int64_t K, int t)
{
    return (size_t)wgrad_plan(T, N, K, t == SPEC_BF16 ? 2 : 4).total;
}

hipError_t launch_mx_linear(hipStream_t stream, const void *X, int t, int64_t T, int64_t N, int64_t K, int64_t ldx,
                            const spec_mx *W, void *Y, int64_t ldy, void *ws)
{
    if (T == 0) return hipSuccess;
    if (T <= FEW_ROWS)
        return t == SPEC_BF16 ? few<ElBF16>(stream, X, ldx, T, N, K, W, Y, ldy) : few<ElF32>(stream, X, ldx, T, N, K, W, Y, ldy);
    return t == SPEC_BF16 ? linear<ElBF16>(stream, X, ldx, T, N, K, W, Y, ldy, (char *)ws)
                          : linear<ElF32>(stream, X, ldx, T, N, K, W, Y, ldy, (char *)ws);
}

hipError_t launch_mx_product(hipStream_t stream, const spec_mx *X, const spec_mx *W, int64_t T, int64_t N, int64_t K,
                             void *Y, int yt, int64_t ldy, void *ws)
{
    if (T == 0) return hipSuccess;
    return yt == SPEC_BF16 ? product4<ElBF16>(stream, X, W, T, N, K, Y, ldy, (char *)ws)
                           : product4<ElF32>(stream, X, W, T, N, K, Y, ldy, (char *)ws);
}

hipError_t launch_mx_weight_grad(hipStream_t stream, const void *dY, int t, int64_t T, int64_t N, int64_t K, int64_t ldy,
                                 const spec_mx *X, float beta, void *dW, int64_t lddw, void *ws)
{
    return t == SPEC_BF16 ? wgrad<ElBF16>(stream, dY, ldy, T, N, K, X, beta, dW, lddw, (char *)ws)
                          : wgrad<ElF32>(stream, dY, ldy, T, N, K, X, beta, dW, lddw, (char *)ws);
}
