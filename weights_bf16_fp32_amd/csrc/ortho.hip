// Orthogonalisation of an update by Newton-Schulz products, gfx950.
//
//   X_0 = G / (|G|_F + eps);  A = X X^T,  X <- a X + (b A + c A^2) X  per step;  O = scale X
//
// (on the shorter side: for m > n the Gram matrix is X^T X and the factor acts
// from the right).  One step multiplies every singular value s by
// a + b s^2 + c s^4, so all of them move towards one and the singular vectors
// stay.
//
// Arithmetic for bf16 updates: f16 operands on MFMA (the iterates are bounded,
// so f16's range suffices with powers of two as scales, and its eight times
// finer rounding costs nothing), f32 accumulation.  Two things keep the
// rounding of an operand from being amplified by the later steps (a small
// singular value grows by up to a per step, and an error in its direction with
// it):
//   - X is kept as the sum of two f16 numbers (22 bits).  The products take the
//     leading one; the term a X, the only one that small singular values live
//     on, takes both.
//   - A = D + E and b A + c A^2 = D' + E' are kept as an f32 diagonal and an f16
//     off-diagonal part.  When X is nearly orthogonal A is nearly diagonal, so
//     what is rounded is small:
//       B_ij = (b + c (d_i + d_j)) E_ij + c (E E)_ij,  B_ii = b d_i + c (d_i^2 + (E E)_ii)
//       X_i <- (a + B_ii) X_i + sum_k E'_ik X_k
// f32 updates run the same products on f32 MFMA.
//
// A and B are symmetric: only tiles on and below the diagonal are computed, and
// each is written to both places.
//
// Small bf16 matrices (both sides up to 256) are bound by the number of
// dependent launches, not by their products, and take one launch per step: a
// workgroup computes 32 rows of the next X from the whole present one by
//   E_i = offdiag(X_i X^T),  R_i = E_i X,  Z_i = A_i A = d_i E_i + R_i X^T + diag,
//   X_i <- (a + b d_i + c z_ii) X_i + b R_i + c offdiag(Z_i) X
// which multiplies more (four products of 32 rows, no symmetry) but never
// waits for another workgroup's A or B.
//
// 4096 x 4096 bf16, per step: 93 us for A (253 tiles of 192 x 192, one per CU), 117 us
// for B (the same products, and A read for its epilogue), 148 us for X; the
// products' share of the time, 29 to 42 % MFMA busy, is bounded by single rounds of
// workgroups, whose first copies and last stores nothing hides, and by one wave per
// SIMD in the 192 x 192 tiles.  256 x 256: 16 us for the start and 11 to 12.5 us per step
// in one launch, of which the products are about 2: the rest is reading X, which each of
// the eight workgroups does whole on an XCD of its own, whose L2 holds little of what
// the others wrote (22 of 36 thousand requests miss).  f32 is bound by the f32 MFMA
// rate (144 of 157 TFLOP/s at 4096^3); three matrices of 333 x 1000 by the few tiles
// they have.
//
//   k_ns_norm   partial sums of squares (f64)
//   k_ns_load   X_0
//   k_ns_gram   A and its diagonal
//   k_ns_poly   B and its diagonal
//   k_ns_apply  the next X, or O
//   k_chain_load, k_chain_step   the same for small matrices
#include <algorithm>
#include <math.h>

#include "internal.h"
#include "mm.h"

namespace {

inline int64_t cdiv_h(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up_h(int64_t a, int64_t b) { return cdiv_h(a, b) * b; }

// workgroups of the norm per matrix: about 64 elements per thread
inline int norm_blocks(int64_t m, int64_t n) { return (int)std::min<int64_t>(1024, cdiv_h(m * n, 64 * 256)); }

// four consecutive elements j .. j + 3 of a row of n (zero past its end); vec:
// the row and its neighbours are aligned to four elements
template <typename G>
SPEC_DEVICE void row4(const typename G::st *x, int64_t j, int64_t n, int vec, float (&v)[4])
{
    if (vec && j + 4 <= n) {
        const Vec4<G> r = *reinterpret_cast<const Vec4<G> *>(x + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = G::wide(r.v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = j + e < n ? G::wide(x[j + e]) : 0.f;
    }
}

// grid (norm_blocks, batch): a wave per row in turn; squares and sums in f64, so
// that no G overflows
template <typename G>
__global__ __launch_bounds__(256) void k_ns_norm(const typename G::st *__restrict__ X, int64_t m, int64_t n, int64_t ld,
                                                 int64_t stride, int vec, double *__restrict__ part)
{
    __shared__ double red[4];
    const typename G::st *x = X + blockIdx.y * stride;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double s = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * 4 + wave; i < m; i += 4 * (int64_t)gridDim.x)
        for (int64_t j0 = 4 * lane; j0 < n; j0 += 8 * 256) {
            float v[8][4];
#pragma unroll
            for (int k = 0; k < 8; ++k) row4<G>(x + i * ld, min(j0 + k * 256, n), n, vec, v[k]);  // requested together
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) s += (double)v[k][e] * (double)v[k][e];
        }
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) red[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// What takes G to X: sx / (|G|_F + eps) for the sum of squares, and 0 for a zero G,
// whatever eps.  Of subnormal norms it leaves f32's range and of those above 2^126
// it loses bits there, so it is held as m p, p a power of two: x p is exact (an x
// that it takes below 2^-126 is nothing to the norm) and x p m is rounded once.
// (One product in f64 takes 14336 x 4096 elements 20 us longer.)
struct NsFactor {
    float p, m;
    SPEC_DEVICE NsFactor(double squares, double eps, float sx)
    {
        const double f = squares == 0.0 ? 0.0 : (double)sx / (sqrt(squares) + eps);
        int e;
        frexp(f, &e);
        p = __uint_as_float((uint32_t)(max(-126, min(127, e)) + 127) << 23);
        m = (float)(f / (double)p);
    }
    SPEC_DEVICE float operator()(float x) const { return x * p * m; }
};

// X as the kernels hold it: leading part and, for f16, the rest
template <typename E>
SPEC_DEVICE void put_x(typename E::st *hi, typename E::st *lo, int64_t at, const float (&v)[4])
{
    Vec4<E> h, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h.v[e] = E::round(v[e]);
        if (sizeof(typename E::st) == 2) l.v[e] = E::round(v[e] - E::wide(h.v[e]));
    }
    *reinterpret_cast<Vec4<E> *>(hi + at) = h;
    if (sizeof(typename E::st) == 2) *reinterpret_cast<Vec4<E> *>(lo + at) = l;
}

// X = G * sx / (norm + eps), padding columns zero.  grid (rows, batch)
template <typename G, typename E>
__global__ __launch_bounds__(256) void k_ns_load(const typename G::st *__restrict__ X, int64_t n, int64_t ld,
                                                 int64_t stride, int vec, const double *__restrict__ part, int nb, double eps, float sx,
                                                 typename E::st *__restrict__ hi, typename E::st *__restrict__ lo,
                                                 int64_t xp, int64_t xs)
{
    double s = 0.0;
    for (int i = threadIdx.x & 63; i < nb; i += 64) s += part[(int64_t)blockIdx.y * nb + i];
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    const NsFactor unit(s, eps, sx);
    const int64_t i = blockIdx.x;
    const typename G::st *x = X + blockIdx.y * stride + i * ld;
    for (int64_t j = 4 * threadIdx.x; j < xp; j += 1024) {
        float v[4];
        row4<G>(x, j, n, vec, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = unit(v[e]);
        put_x<E>(hi, lo, blockIdx.y * xs + i * xp + j, v);
    }
}

// One matrix of the batch: X (rows x cols at pitch xp), the r x r matrices at pitch ap.
struct NsDims {
    int64_t rows, cols, xp, xs;  // X
    int64_t r, ap, as;           // A, B
};

// stores four entries (row i, columns j..j+3) of a symmetric matrix, its diagonal
// apart in diag; on: whether the entries may lie on the diagonal
template <typename E>
SPEC_DEVICE void put_sym(typename E::st *A, float *diag, const NsDims &D, int64_t i, int64_t j, bool on,
                         const float (&v)[4], float scale)
{
    Vec4<E> o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (on && i == j + e && i < D.ap) diag[i] = v[e];  // (zero from r on)
        o.v[e] = on && i == j + e ? (typename E::st)0 : E::round(v[e] * scale);
    }
    if (i < D.r && j < D.ap) *reinterpret_cast<Vec4<E> *>(A + i * D.ap + j) = o;
}

// grid (tiles on and below the diagonal, batch).  real: 1 / sx^2
template <typename E, typename C, bool TALL>
__global__ MM_BOUNDS(C) void k_ns_gram(const typename E::st *__restrict__ X, NsDims D,
                                                                    float real, float sa,
                                                                    typename E::st *__restrict__ A,
                                                                    float *__restrict__ diag)
{
    using M = Mm<E, C, TALL, TALL>;
    MM_STAGES(M);
    int ti, tj;
    tri_tile_blocked(xcd_remap(blockIdx.x, gridDim.x), (int)((D.r + C::BP - 1) / C::BP), ti, tj);
    const int64_t i0 = (int64_t)ti * C::BQ, j0 = (int64_t)tj * C::BP;
    const typename E::st *x = X + blockIdx.y * D.xs;
    const int64_t step = TALL ? 1 : D.xp, K = TALL ? D.rows : round_up(D.cols, M::EPC);
    const MmSrc P{(const char *)(x + j0 * step), D.xp * M::SZ, (int)min<int64_t>(C::BP, D.r - j0), K};
    const MmSrc Q{(const char *)(x + i0 * step), D.xp * M::SZ, (int)min<int64_t>(C::BQ, D.r - i0), K};
    M mm;
    mm.run(P, Q, 0, K, lds);
    const auto put = [&](int64_t i, int64_t j, float (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= real;
        put_sym<E>(A + blockIdx.y * D.as, diag + blockIdx.y * D.ap, D, i, j, ti == tj, v, sa);
    };
    mm.each4(lds, [&](int p, int q, float (&v)[4]) { put(i0 + q, j0 + p, v); });
    if (ti != tj)
        mm.each4_across(lds, [](int, int) { return 0; }, [&](int p, int q, float (&v)[4], int) { put(j0 + p, i0 + q, v); });
}

// B = b A + c A^2 with A = diag(da) + E; ea = 1 / sa
template <typename E, typename C>
__global__ MM_BOUNDS(C) void k_ns_poly(const typename E::st *__restrict__ A,
                                                                    const float *__restrict__ da, NsDims D, float b,
                                                                    float c, float ea, float sb,
                                                                    typename E::st *__restrict__ B,
                                                                    float *__restrict__ diag)
{
    using M = Mm<E, C, false, false>;
    MM_STAGES(M);
    int ti, tj;
    tri_tile_blocked(xcd_remap(blockIdx.x, gridDim.x), (int)((D.r + C::BP - 1) / C::BP), ti, tj);
    const int64_t i0 = (int64_t)ti * C::BQ, j0 = (int64_t)tj * C::BP;
    const typename E::st *a = A + blockIdx.y * D.as;
    const float *d = da + blockIdx.y * D.ap;
    const int64_t K = round_up(D.r, M::EPC);
    const MmSrc P{(const char *)(a + j0 * D.ap), D.ap * M::SZ, (int)min<int64_t>(C::BP, D.r - j0), K};
    const MmSrc Q{(const char *)(a + i0 * D.ap), D.ap * M::SZ, (int)min<int64_t>(C::BQ, D.r - i0), K};
    M mm;
    mm.run(P, Q, 0, K, lds);
    struct Old {
        Vec4<E> x;
        float di;
        float4 dj;
    };
    const auto get = [&](int64_t i, int64_t j) {
        Old o{};
        if (i < D.r && j < D.ap) {
            o.x = *reinterpret_cast<const Vec4<E> *>(a + i * D.ap + j);
            o.di = d[i];
            o.dj = *reinterpret_cast<const float4 *>(d + j);
        }
        return o;
    };
    const auto put = [&](int64_t i, int64_t j, float (&v)[4], const Old &o) {
        const float dj[4] = {o.dj.x, o.dj.y, o.dj.z, o.dj.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float aa = c * (v[e] * ea * ea);
            v[e] = i == j + e ? b * o.di + (c * o.di * o.di + aa) : (b + c * (o.di + dj[e])) * (E::wide(o.x.v[e]) * ea) + aa;
        }
        put_sym<E>(B + blockIdx.y * D.as, diag + blockIdx.y * D.ap, D, i, j, ti == tj, v, sb);
    };
    mm.each4(lds, [&](int p, int q) { return get(i0 + q, j0 + p); },
             [&](int p, int q, float (&v)[4], const Old &o) { put(i0 + q, j0 + p, v, o); });
    if (ti != tj)
        mm.each4_across(lds, [&](int p, int q) { return get(j0 + p, i0 + q); },
                        [&](int p, int q, float (&v)[4], const Old &o) { put(j0 + p, i0 + q, v, o); });
}

// The next X (scaled by sx1), or O = scale X in the last step.
// ex = 1 / sx of the current X, eb = 1 / sb.
template <typename E, typename C, bool TALL, typename O, bool LAST>
__global__ MM_BOUNDS(C) void k_ns_apply(
    const typename E::st *__restrict__ hi, const typename E::st *__restrict__ lo, const typename E::st *__restrict__ B,
    const float *__restrict__ db, NsDims D, int np, int nq, float a, float ex, float eb, float sx1,
    typename E::st *__restrict__ hi1, typename E::st *__restrict__ lo1, typename O::st *__restrict__ out, int64_t ldo,
    int64_t os, int vec)
{
    using M = Mm<E, C, !TALL, false>;
    MM_STAGES(M);
    int tp, tq;
    mm_tile(blockIdx.x, np, nq, tp, tq);
    const int64_t j0 = (int64_t)tp * C::BP, i0 = (int64_t)tq * C::BQ;
    const int64_t xb = blockIdx.y * D.xs;
    const typename E::st *bm = B + blockIdx.y * D.as;
    const float *d = db + blockIdx.y * D.ap;
    const int64_t K = round_up(D.r, M::EPC);
    MmSrc P, Q;
    if (TALL) {  // rows of B (symmetric) against rows of X
        P = MmSrc{(const char *)(bm + j0 * D.ap), D.ap * M::SZ, (int)min<int64_t>(C::BP, D.r - j0), K};
        Q = MmSrc{(const char *)(hi + xb + i0 * D.xp), D.xp * M::SZ, (int)min<int64_t>(C::BQ, D.rows - i0), K};
    } else {  // columns of X against rows of B
        P = MmSrc{(const char *)(hi + xb + j0), D.xp * M::SZ, (int)min<int64_t>(C::BP, D.cols - j0), D.r};
        Q = MmSrc{(const char *)(bm + i0 * D.ap), D.ap * M::SZ, (int)min<int64_t>(C::BQ, D.r - i0), K};
    }
    M mm;
    mm.run(P, Q, 0, K, lds);
    struct Old {
        Vec4<E> h, l;
        float4 d;
    };
    const auto get = [&](int p, int q) {
        const int64_t i = i0 + q, j = j0 + p, at = xb + i * D.xp + j;
        Old o{};
        if (i < D.rows && j < D.xp) {
            o.h = *reinterpret_cast<const Vec4<E> *>(hi + at);
            if (M::SZ == 2) o.l = *reinterpret_cast<const Vec4<E> *>(lo + at);
            o.d = TALL ? *reinterpret_cast<const float4 *>(d + j) : make_float4(d[i], d[i], d[i], d[i]);
        }
        return o;
    };
    mm.each4(lds, get, [&](int p, int q, float (&v)[4], const Old &o) {
        const int64_t i = i0 + q, j = j0 + p;
        if (i >= D.rows || j >= D.xp) return;
        const float dd[4] = {o.d.x, o.d.y, o.d.z, o.d.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = E::wide(o.h.v[e]) + (M::SZ == 2 ? E::wide(o.l.v[e]) : 0.f);
            v[e] = ((a + dd[e]) * x + eb * v[e]) * ex * sx1;
        }
        if (!LAST) {
            put_x<E>(hi1, lo1, xb + i * D.xp + j, v);
        } else {
            typename O::st *o = out + blockIdx.y * os + i * ldo + j;
            if (vec && j + 4 <= D.cols) {
                Vec4<O> r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r.v[e] = O::round(v[e]);
                *reinterpret_cast<Vec4<O> *>(o) = r;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < D.cols) o[e] = O::round(v[e]);
            }
        }
    });
}

// ------------------------------------------------------------------ small matrices

// X (r x s, r <= s, whatever G's orientation; padded with zeros to rp x sp) is kept
// in `hi` and `lo`, its leading part also transposed (sp x rp) in `tr`: every
// product then reads both operands along k.  All of them, and the operands in
// LDS, lie in the order of the MFMA's fragments: blocks of 32 rows, in them groups
// of 16 k, in them 64 runs of 8 (the row, then the half of the group), so that a
// wave's fragment is 1 KB in a run.  (Row-major, a fragment met 32 cache lines for
// 32 bytes each, and reading X took 10 of a step's 17 us.)
struct ChainDims {
    int r, s, rp, sp;  // rp, sp: rounded up to 64
};
constexpr int CHAIN = 256;  // the longer side at most

// Up to here a wave holds its blocks of both operands in registers (236 of 256, and 48
// bytes of scratch per lane), and a
// matrix takes 43 us (128 x 128) to 70 us (256 x 256) against 94 to 100 us of the
// other path from 256 x 512 on; with operands read from memory 256 x 512 took 143 us.
inline bool chain_fits(int64_t m, int64_t n) { return m <= CHAIN && n <= CHAIN; }

using h8 = f16x8_t;
SPEC_DEVICE uint16_t f16_bits(float x) { return ElF16::round(x); }

// place of element (row, k) of a matrix with K columns
SPEC_DEVICE int chain_at(int row, int k, int K)
{
    return (row >> 5) * 32 * K + (k >> 4) * 512 + ((row & 31) + 32 * ((k >> 3) & 1)) * 8 + (k & 7);
}

// a block of 32 rows of a product's operand, in registers: read once, used by two products
struct ChainHeld {
    h8 a[16];
    SPEC_DEVICE ChainHeld(const uint16_t *block, int K, int lane)
    {
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = 16 * j < K ? *reinterpret_cast<const h8 *>(block + j * 512 + lane * 8) : h8{};
    }
};

SPEC_DEVICE f32x16_t chain_zero()
{
    f32x16_t z;
#pragma unroll
    for (int e = 0; e < 16; ++e) z[e] = 0.f;
    return z;
}

// 32 x 32 block sum_k P[p][k] Q[q][k] with Q's rows in LDS; the sums of even and
// odd groups of 16 apart, so that a product need not wait for the one before
SPEC_DEVICE f32x16_t chain_product(const ChainHeld &P, const uint16_t *Q, int K, int lane)
{
    f32x16_t s0 = chain_zero(), s1 = chain_zero();
    const h8 *q = reinterpret_cast<const h8 *>(Q) + lane;
#pragma unroll
    for (int j0 = 0; j0 < 16; j0 += 4)
        if (16 * j0 < K) {
            h8 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = q[(j0 + j) * 64];
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                s0 = __builtin_amdgcn_mfma_f32_32x32x16_f16(P.a[j0 + j], b[j], s0, 0, 0, 0);
                s1 = __builtin_amdgcn_mfma_f32_32x32x16_f16(P.a[j0 + j + 1], b[j + 1], s1, 0, 0, 0);
            }
        }
    return s0 + s1;
}

// grid (rp / 32, batch), 512 threads: X = G sx / (norm + eps).  Every workgroup
// sums all squares itself (at most 128 KB from the L2).
__global__ __launch_bounds__(512) void k_chain_load(const uint16_t *__restrict__ G, int m, int n, int64_t ldg, int64_t sg,
                                                    int vec, ChainDims D, double eps, float sx, uint16_t *__restrict__ hi,
                                                    uint16_t *__restrict__ lo, uint16_t *__restrict__ tr)
{
    __shared__ double red[8];
    const uint16_t *g = G + blockIdx.y * sg;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    double s = 0.0;
    // a wave per row, eight rows requested together
    for (int i = wave; i < m; i += 64)
        for (int j = 4 * lane; j < n; j += 256) {
            float v[8][4];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int ik = i + 8 * k;
                row4<ElBF16>(g + min(ik, m - 1) * ldg, ik < m ? j : n, n, vec, v[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) s += (double)v[k][e] * (double)v[k][e];
        }
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) red[wave] = s;
    __syncthreads();
    s = 0.0;
    for (int k = 0; k < 8; ++k) s += red[k];
    const NsFactor unit(s, eps, sx);
    const int i0 = blockIdx.x * 32;
    const int64_t base = (int64_t)blockIdx.y * D.rp * D.sp;
    const bool tall = m > n;
    // along G's rows: columns of X for a wide G, rows of X for a tall one
    const int q0 = tall ? lane & 31 : wave * 4, c0 = tall ? wave * 2 + (lane >> 5) : lane;
    const int qk = tall ? 0 : 1, ck = tall ? 16 : 0;
    for (int cb = 0; cb < D.sp; cb += 128) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + q0 + (k & 3) * qk, c = cb + c0 + (k & 3) * ck + 64 * (k >> 2);
            v[k] = i < D.r && c < D.s ? unit(bf16_to_f32(tall ? g[c * ldg + i] : g[i * ldg + c])) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + q0 + (k & 3) * qk, c = cb + c0 + (k & 3) * ck + 64 * (k >> 2);
            if (c >= D.sp) continue;
            const uint16_t h = f16_bits(v[k]);
            hi[base + chain_at(i, c, D.sp)] = h;
            lo[base + chain_at(i, c, D.sp)] = f16_bits(v[k] - ElF16::wide(h));
            tr[base + chain_at(c, i, D.rp)] = h;
        }
    }
}

struct ChainStep {
    float a, b, c;      // the step's polynomial
    float sx, sx1;      // scales of X and of the next one (or of O)
    float sa, sr, sz;   // of E, R and Z
};

// grid (rp / 32, batch), 512 threads: wave w has the rows j and the columns of block w
template <bool LAST>
__global__ __launch_bounds__(512, 2) void k_chain_step(const uint16_t *__restrict__ hi, const uint16_t *__restrict__ lo,
                                                    const uint16_t *__restrict__ tr, ChainDims D, ChainStep t,
                                                    uint16_t *__restrict__ hi1, uint16_t *__restrict__ lo1,
                                                    uint16_t *__restrict__ tr1, uint16_t *__restrict__ out, int64_t ldo,
                                                    int64_t so, int tall)
{
    __shared__ __attribute__((aligned(16))) uint16_t Q[32 * CHAIN], Ez[32 * CHAIN];  // Q: X_i, then R_i
    __shared__ float dd[32], zz[32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, q = lane & 31;
    const int i0 = blockIdx.x * 32;
    const int64_t base = (int64_t)blockIdx.y * D.rp * D.sp;
    hi += base, lo += base, tr += base;
    const uint16_t *own_hi = hi + i0 * D.sp, *own_lo = lo + i0 * D.sp;  // this workgroup's rows
    // X_i to LDS first, then all operands and X, requested before the first product
    uint4 mine[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (tid + 512 * k < 4 * D.sp) mine[k] = reinterpret_cast<const uint4 *>(own_hi)[tid + 512 * k];
    const bool rows = wave * 32 < D.rp, columns = wave * 32 < D.sp, own = wave == (int)blockIdx.x;
    const int c0 = wave * 32;
    const ChainHeld Pj(hi + (rows ? c0 : 0) * D.sp, D.sp, lane), Pc(tr + (columns ? c0 : 0) * D.rp, D.rp, lane);
    // place of the four elements of row q at column c0 + 8 g + 4 h in a block
    const auto place = [&](int g) { return (c0 / 16 + (g >> 1)) * 512 + (q + 32 * (g & 1)) * 8 + 4 * h; };
    Vec4<ElF16> xh[4], xl[4];
    if (columns) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            xh[g] = *reinterpret_cast<const Vec4<ElF16> *>(own_hi + place(g));
            xl[g] = *reinterpret_cast<const Vec4<ElF16> *>(own_lo + place(g));
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (tid + 512 * k < 4 * D.sp) reinterpret_cast<uint4 *>(Q)[tid + 512 * k] = mine[k];
    __syncthreads();
    const float ex = 1.f / t.sx;
    const auto four = [&](uint16_t *o, const f32x16_t &v, float scale) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            Vec4<ElF16> x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x.v[e] = f16_bits(v[4 * g + e] * scale);
            *reinterpret_cast<Vec4<ElF16> *>(o + place(g)) = x;
        }
    };
    f32x16_t E;
    if (rows) {
        E = chain_product(Pj, Q, D.sp, lane);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            E[e] *= ex * ex;
            if (own && 8 * (e >> 2) + 4 * h + (e & 3) == q) {
                dd[q] = E[e];
                E[e] = 0.f;
            }
        }
        four(Ez, E, t.sa);
    }
    __syncthreads();  // Q has been read, E and its diagonal are written
    f32x16_t R;
    if (columns) {
        R = chain_product(Pc, Ez, D.rp, lane);
#pragma unroll
        for (int e = 0; e < 16; ++e) R[e] *= ex / t.sa;
        four(Q, R, t.sr);
    }
    __syncthreads();
    if (rows) {
        const f32x16_t Z = chain_product(Pj, Q, D.sp, lane);
        const float d = dd[q];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float z = Z[e] * (ex / t.sr);
            if (own && 8 * (e >> 2) + 4 * h + (e & 3) == q) {
                zz[q] = d * d + z;
                z = 0.f;
            } else {
                z += d * E[e];
            }
            E[e] = z;
        }
        four(Ez, E, t.sz);
    }
    __syncthreads();
    if (!columns) return;
    const float f = t.a + t.b * dd[q] + t.c * zz[q];
    const int i = i0 + q;
    const f32x16_t W = chain_product(Pc, Ez, D.rp, lane);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int c = c0 + 8 * g + 4 * h;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = (ElF16::wide(xh[g].v[e]) + ElF16::wide(xl[g].v[e])) * ex;
            v[e] = (f * x + t.b * R[4 * g + e] + t.c * (W[4 * g + e] * (ex / t.sz))) * t.sx1;
        }
        if (LAST) {
            if (i < D.r) {
                uint16_t *o = out + blockIdx.y * so;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < D.s) o[tall ? (c + e) * ldo + i : i * ldo + c + e] = ElBF16::round(v[e]);
            }
        } else {
            put_x<ElF16>(hi1 + base, lo1 + base, i0 * D.sp + place(g), v);
#pragma unroll
            for (int e = 0; e < 4; ++e) tr1[base + chain_at(c + e, i, D.rp)] = f16_bits(v[e]);
        }
    }
}

struct NsPlan {
    NsDims D;
    int64_t part, da, db, a, b, x[2], xl[2], total;
};

NsPlan ns_plan(int64_t batch, int64_t m, int64_t n, int t)
{
    NsPlan p{};
    const int64_t es = t == SPEC_BF16 ? 2 : 4;
    NsDims &D = p.D;
    D.rows = m;
    D.cols = n;
    D.xp = up_h(n, 64);
    D.xs = D.rows * D.xp;
    D.r = std::min(m, n);
    D.ap = up_h(D.r, 64);
    D.as = D.r * D.ap;
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += up_h(bytes, 256);
        return at;
    };
    p.part = take(8 * batch * norm_blocks(m, n));
    p.da = take(4 * batch * D.ap);
    p.db = take(4 * batch * D.ap);
    p.a = take(es * batch * D.as);
    p.b = take(es * batch * D.as);
    for (int i = 0; i < 2; ++i) {
        p.x[i] = take(es * batch * D.xs);
        p.xl[i] = es == 2 ? take(2 * batch * D.xs) : 0;
    }
    p.total = o;
    return p;
}

struct ChainPlan {
    ChainDims D;
    int64_t hi[2], lo[2], tr[2], total;
};

ChainPlan chain_plan(int64_t batch, int64_t m, int64_t n)
{
    ChainPlan p{};
    p.D.r = (int)std::min(m, n);
    p.D.s = (int)std::max(m, n);
    p.D.rp = (int)up_h(p.D.r, 64);
    p.D.sp = (int)up_h(p.D.s, 64);
    const int64_t bytes = up_h(2 * batch * p.D.rp * p.D.sp, 256);
    for (int i = 0; i < 2; ++i) {
        p.hi[i] = (3 * i) * bytes;
        p.lo[i] = (3 * i + 1) * bytes;
        p.tr[i] = (3 * i + 2) * bytes;
    }
    p.total = 6 * bytes;
    return p;
}

// largest |s (a + b s^2 + c s^4)| over 0 <= s <= top: at the end or at a root
// of a + 3 b u + 5 c u^2, u = s^2 (the larger root's numerator without a difference,
// the other root from their product a / 5c: a small c does not cancel them)
double step_bound(const double *co, double top)
{
    const double a = co[0], b = co[1], c = co[2];
    auto f = [&](double s) { return fabs(s * (a + s * s * (b + c * s * s))); };
    double best = f(top);
    double u[2];
    int nu = 0;
    const double q = 9.0 * b * b - 20.0 * a * c;
    if (q >= 0.0) {
        const double w = -0.5 * (3.0 * b + copysign(sqrt(q), b));
        if (c != 0.0) u[nu++] = w / (5.0 * c);
        if (w != 0.0) u[nu++] = a / w;
    }
    for (int k = 0; k < nu; ++k)
        if (u[k] > 0.0 && u[k] < top * top) best = std::max(best, f(sqrt(u[k])));
    return best;
}

// the power of two that takes `bound` to at most 2^14 (f16 holds 65504), at most `most`
double scale16(double bound, double most)
{
    return std::min(most, exp2(floor(14.0 - log2(std::max(bound, 1e-300)))));
}

hipError_t chain_run(hipStream_t stream, const void *G, int64_t batch, int64_t m, int64_t n, int64_t ldg, int64_t sg,
                     const double *co, int steps, double eps, double scale, void *O, int64_t ldo, int64_t so, char *ws)
{
    const ChainPlan p = chain_plan(batch, m, n);
    const ChainDims D = p.D;
    const auto at = [&](int64_t o) { return (uint16_t *)(ws + o); };
    const double want = exp2(floor(0.5 * log2((double)m * (double)n)));
    double top = 1.0, sx = scale16(1.0, want);
    const dim3 grid((unsigned)(D.rp / 32), (unsigned)batch);
    const int vec = n % 4 == 0 && (uintptr_t)G % 8 == 0 && ldg % 4 == 0 && sg % 4 == 0;
    hipLaunchKernelGGL(k_chain_load, grid, dim3(512), 0, stream, (const uint16_t *)G, (int)m, (int)n, ldg, sg, vec, D, eps,
                       (float)sx, at(p.hi[0]), at(p.lo[0]), at(p.tr[0]));
    SPEC_LAUNCH_CHECK();
    for (int k = 0; k < steps; ++k) {
        const double *c = co + 3 * k;
        const double na = top * top, next = 1.02 * step_bound(c, top);
        const bool last = k == steps - 1;
        const ChainStep t{(float)c[0], (float)c[1], (float)c[2], (float)sx, (float)(last ? scale : scale16(next, want)),
                          (float)scale16(na, 16384.0), (float)scale16(2.0 * na * top, 16384.0),
                          (float)scale16(na * na, 16384.0)};
        const int a = k & 1, b = a ^ 1;
        const auto step = last ? k_chain_step<true> : k_chain_step<false>;
        hipLaunchKernelGGL(step, grid, dim3(512), 0, stream, at(p.hi[a]), at(p.lo[a]), at(p.tr[a]), D, t, at(p.hi[b]),
                           at(p.lo[b]), at(p.tr[b]), (uint16_t *)O, ldo, so, m > n);
        SPEC_LAUNCH_CHECK();
        top = next;
        sx = t.sx1;
    }
    return hipSuccess;
}

template <typename GT, typename E, bool TALL>
hipError_t ns_run(hipStream_t stream, const void *G, int64_t batch, int64_t m, int64_t n, int64_t ldg, int64_t sg,
                  const double *co, int steps, double eps, double scale, void *O, int64_t ldo, int64_t so, char *ws)
{
    using st = typename E::st;
    using gst = typename GT::st;
    constexpr bool F16 = sizeof(st) == 2;
    const NsPlan pl = ns_plan(batch, m, n, F16 ? SPEC_BF16 : SPEC_F32);
    const NsDims &D = pl.D;
    double *part = (double *)(ws + pl.part);
    float *da = (float *)(ws + pl.da), *db = (float *)(ws + pl.db);
    st *A = (st *)(ws + pl.a), *B = (st *)(ws + pl.b);
    // entries of X are about 1 / sqrt(m n) at first and at most the largest singular value
    const double want = exp2(floor(0.5 * log2((double)m * (double)n)));
    double top = 1.0, sx = F16 ? scale16(1.0, want) : 1.0;
    const int nb = norm_blocks(m, n);
    const int vin = (uintptr_t)G % (4 * sizeof(gst)) == 0 && ldg % 4 == 0 && sg % 4 == 0;
    hipLaunchKernelGGL(k_ns_norm<GT>, dim3((unsigned)nb, (unsigned)batch), dim3(256), 0, stream, (const gst *)G, m, n, ldg,
                       sg, vin, part);
    SPEC_LAUNCH_CHECK();
    hipLaunchKernelGGL((k_ns_load<GT, E>), dim3((unsigned)m, (unsigned)batch), dim3(256), 0, stream, (const gst *)G, n, ldg,
                       sg, vin, part, nb, eps, (float)sx, (st *)(ws + pl.x[0]), (st *)(ws + pl.xl[0]), D.xp, D.xs);
    SPEC_LAUNCH_CHECK();
    const auto tri = [&](int64_t e) { return cdiv_h(D.r, e) * (cdiv_h(D.r, e) + 1) / 2; };
    const auto rect = [&](int64_t e) { return cdiv_h(m, e) * cdiv_h(n, e); };
    const int vec = (uintptr_t)O % (4 * sizeof(gst)) == 0 && ldo % 4 == 0 && so % 4 == 0;
    for (int k = 0; k < steps; ++k) {
        const double *c = co + 3 * k;
        const double na = top * top, nb = fabs(c[1]) * na + fabs(c[2]) * na * na;
        const double sa = F16 ? scale16(na, 16384.0) : 1.0, sb = F16 ? scale16(nb, 16384.0) : 1.0;
        const double next = 1.02 * step_bound(c, top);
        const bool last = k == steps - 1;
        const double sx1 = last ? scale : (F16 ? scale16(next, want) : 1.0);
        const st *hi = (const st *)(ws + pl.x[k & 1]), *lo = (const st *)(ws + pl.xl[k & 1]);
        st *hi1 = (st *)(ws + pl.x[(k & 1) ^ 1]), *lo1 = (st *)(ws + pl.xl[(k & 1) ^ 1]);
        hipError_t e = mm_pick<E>([&](int64_t w) { return tri(w) * batch; }, [&](auto shape) {
            using C = decltype(shape);
            const dim3 grid((unsigned)tri(C::BP), (unsigned)batch);
            hipLaunchKernelGGL((k_ns_gram<E, C, TALL>), grid, dim3(C::NT), 0, stream, hi, D, (float)(1.0 / (sx * sx)),
                               (float)sa, A, da);
            SPEC_LAUNCH_CHECK();
            hipLaunchKernelGGL((k_ns_poly<E, C>), grid, dim3(C::NT), 0, stream, A, da, D, (float)c[1], (float)c[2],
                               (float)(1.0 / sa), (float)sb, B, db);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
        e = mm_pick<E>([&](int64_t w) { return rect(w) * batch; }, [&](auto shape) {
            using C = decltype(shape);
            const int np = (int)cdiv_h(n, C::BP), nq = (int)cdiv_h(m, C::BQ);
            const dim3 grid((unsigned)((int64_t)np * nq), (unsigned)batch);
            if (last)
                hipLaunchKernelGGL((k_ns_apply<E, C, TALL, GT, true>), grid, dim3(C::NT), 0, stream, hi, lo, B, db, D, np,
                                   nq, (float)c[0], (float)(1.0 / sx), (float)(1.0 / sb), (float)sx1, hi1, lo1, (gst *)O,
                                   ldo, so, vec);
            else
                hipLaunchKernelGGL((k_ns_apply<E, C, TALL, GT, false>), grid, dim3(C::NT), 0, stream, hi, lo, B, db, D, np,
                                   nq, (float)c[0], (float)(1.0 / sx), (float)(1.0 / sb), (float)sx1, hi1, lo1, (gst *)O,
                                   ldo, so, vec);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
        top = next;
        sx = sx1;
    }
    return hipSuccess;
}

}  // namespace

size_t orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n, int t)
{
    if (t == SPEC_BF16 && chain_fits(m, n)) return (size_t)chain_plan(batch, m, n).total;
    return (size_t)ns_plan(batch, m, n, t).total;
}

// whether f16 holds the iterates and the products in between
bool orthogonalize_bounded(const double *co, int steps)
{
    double top = 1.0;
    for (int k = 0; k < steps; ++k) {
        const double na = top * top;
        // A, b A + c A^2, A^2 and (A - D) X within f16's range at scale one
        if (!(na * na <= 16384.0 && 2.0 * na * top <= 16384.0 &&
              fabs(co[3 * k + 1]) * na + fabs(co[3 * k + 2]) * na * na <= 16384.0))
            return false;
        top = 1.02 * step_bound(co + 3 * k, top);
    }
    return top <= 16384.0;
}

hipError_t launch_orthogonalize(hipStream_t stream, const void *G, int t, int64_t batch, int64_t m, int64_t n,
                                int64_t ldg, int64_t sg, const double *co, int steps, double eps, double scale, void *O,
                                int64_t ldo, int64_t so, void *ws)
{
    char *w = (char *)ws;
    if (t == SPEC_BF16 && chain_fits(m, n))
        return chain_run(stream, G, batch, m, n, ldg, sg, co, steps, eps, scale, O, ldo, so, w);
    if (t == SPEC_BF16)
        return m > n ? ns_run<ElBF16, ElF16, true>(stream, G, batch, m, n, ldg, sg, co, steps, eps, scale, O, ldo, so, w)
                     : ns_run<ElBF16, ElF16, false>(stream, G, batch, m, n, ldg, sg, co, steps, eps, scale, O, ldo, so, w);
    return m > n ? ns_run<ElF32, ElF32, true>(stream, G, batch, m, n, ldg, sg, co, steps, eps, scale, O, ldo, so, w)
                 : ns_run<ElF32, ElF32, false>(stream, G, batch, m, n, ldg, sg, co, steps, eps, scale, O, ldo, so, w);
}
