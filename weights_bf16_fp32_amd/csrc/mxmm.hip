// Products with microscaled matrices, gfx950 (the format: mx.h; the tiles: mm.h).
//
//   linear   Y[t][n] = sum_k X[t][k] W[n][k]       W in FP4, X bf16 or f32
//   product  the same, X in FP4 too
//   wgrad    dW[n][k] = beta dW[n][k] + sum_t dY[t][n] X[t][k]     X in INT8, dY bf16 or f32
//
// A microscaled value has at most seven significant bits and a power of two, so it
// is exact in bf16: the packed operand is unpacked into the workspace, and the
// products are bf16 (f32) MFMA products with f32 sums.
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
        store8<E>(P + r * eights * 8, e, eights * 8, load8<E>(X + r * ldx, e, c));
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

// acc[q][p] = sum over k of P(p, k) Q(q, k), both operands with k contiguous (S false) or slow
template <typename E, typename EO, typename C, bool S>
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
    if (o.ways > 1) {
        float *part = o.part + (share * o.rows + q0) * o.ldpart + p0;
        mm.each4(lds, [&](int p, int q, float (&v)[4]) {
            if (q < sq.lim && p < sp.lim)  // (ldpart is a multiple of 4: a group of four lies in its row)
                *reinterpret_cast<float4 *>(part + q * o.ldpart + p) = make_float4(v[0], v[1], v[2], v[3]);
        });
    } else {
        typename EO::st *out = (typename EO::st *)o.out + q0 * o.ldo + p0;
        mm.each4(lds, [&](int p, int q, float (&v)[4]) {
            if (q < sq.lim && p < sp.lim) put4<EO>(out + q * o.ldo + p, v, o.beta, sp.lim - p, vec != 0);
        });
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

// shares of k of a product of np x nq results: as many as give every CU a tile,
// of 256 k at least, as far as their sums have room
int split_ways(int64_t np, int64_t nq, int64_t K)
{
    const int64_t tiles = cdiv_h(np, 128) * cdiv_h(nq, 128);
    int64_t w = std::min<int64_t>(cdiv_h(256, tiles), K / 256);
    w = std::min<int64_t>(w, SPLIT_BYTES / (4 * up_h(np, 4) * std::max<int64_t>(nq, 1)));
    return (int)std::max<int64_t>(1, std::min<int64_t>(w, 64));
}

template <typename E, typename EO, bool S>
hipError_t product(hipStream_t stream, const typename E::st *P, int64_t ldp, int64_t np, const typename E::st *Q,
                   int64_t ldq, int64_t nq, int64_t K, void *out, int64_t ldo, float beta, float *part)
{
    using st = typename EO::st;
    const int vec = (uintptr_t)out % (4 * sizeof(st)) == 0 && ldo % 4 == 0;
    MmOut o{out, ldo, beta, part, up_h(np, 4), nq, split_ways(np, nq, K)};
    const hipError_t e = mm_pick<E>([&](int64_t edge) { return cdiv_h(np, edge) * cdiv_h(nq, edge) * o.ways; }, [&](auto c) {
        using C = decltype(c);
        const int tp = (int)cdiv_h(np, C::BP), tq = (int)cdiv_h(nq, C::BQ);
        hipLaunchKernelGGL((k_mx_mm<E, EO, C, S>), dim3((unsigned)((int64_t)tp * tq * o.ways)), dim3(C::NT), 0, stream, P,
                           ldp, np, Q, ldq, nq, K, tp, tq, o, vec);
        return hipGetLastError();
    });
    if (e != hipSuccess || o.ways == 1) return e;
    hipLaunchKernelGGL(k_mx_join<EO>, dim3((unsigned)std::min<int64_t>(cdiv_h(o.rows * o.ldpart / 4, 256), 4096)), dim3(256),
                       0, stream, o, np, vec);
    return hipGetLastError();
}

// Packed matrices are unpacked a piece of rows (linear, product) or of columns
// (wgrad, whose rows are the sums' k) at a time; rows of up_h(c, 32) values.
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

constexpr int64_t MOST_T = 65536;  // rows of X per launch

struct LinearPlan {
    int64_t kp, wrows, w, x, part, total;  // bytes into the workspace
};
// X: rows of X copied or unpacked at a time (0: none)
LinearPlan linear_plan(int64_t T, int64_t N, int64_t K, int64_t es)
{
    LinearPlan p{};
    p.kp = up_h(K, 32);
    p.wrows = piece_rows(N, p.kp * es);
    const int64_t t = std::min(T, MOST_T);
    p.w = 0;
    p.x = up_h(p.wrows * p.kp * es, 256);
    p.part = p.x + up_h(std::max<int64_t>(t, 1) * p.kp * es, 256);
    const int64_t ways = split_ways(p.wrows, t, K);
    p.total = p.part + SPLIT_BYTES;
    return p;
}

template <typename E, typename EO>
hipError_t linear(hipStream_t stream, const void *X, int64_t ldx, const spec_mx *Xq, int64_t T, int64_t N, int64_t K,
                  const spec_mx *W, void *Y, int64_t ldy, char *ws)
{
    using st = typename E::st;
    constexpr int64_t es = sizeof(st), eo = sizeof(typename EO::st);
    constexpr int t = es == 2 ? SPEC_BF16 : SPEC_F32;
    const LinearPlan p = linear_plan(T, N, K, es);
    st *const wv = (st *)(ws + p.w), *const xv = (st *)(ws + p.x);
    const bool in_place = Xq == nullptr && direct<E>(X, ldx, K);
    for (int64_t n = 0; n < N; n += p.wrows) {
        const int64_t nn = std::min(p.wrows, N - n);
        const spec_mx wn = rows_from(W, n);
        hipError_t e = launch_mx_dequantize(stream, &wn, nn, K, p.kp, wv, t, p.kp);
        for (int64_t t0 = 0; t0 < T && e == hipSuccess; t0 += MOST_T) {
            const int64_t tn = std::min(MOST_T, T - t0);
            const st *x = xv;
            int64_t ld = p.kp;
            if (Xq != nullptr) {
                const spec_mx xq = rows_from(Xq, t0);
                e = launch_mx_dequantize(stream, &xq, tn, K, p.kp, xv, t, p.kp);
            } else if (in_place) {
                x = (const st *)X + t0 * ldx;
                ld = ldx;
            } else {
                e = pack<E>(stream, (const st *)X + t0 * ldx, tn, K, ldx, xv);
            }
            if (e != hipSuccess) break;
            e = product<E, EO, false>(stream, wv, p.kp, nn, x, ld, tn, K, (char *)Y + (t0 * ldy + n) * eo, ldy, 0.f,
                                      (float *)(ws + p.part));
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
            e = product<E, E, true>(stream, xv, p.cols, cn, dy, ldy, N, T, (st *)dW + c, lddw, beta, (float *)(ws + p.part));
    }
    return e;
}

}  // namespace

size_t mx_linear_workspace_bytes(int64_t T, int64_t N, int64_t K, int t)
{
    return (size_t)linear_plan(T, N, K, t == SPEC_BF16 ? 2 : 4).total;
}

size_t mx_product_workspace_bytes(int64_t T, int64_t N, int64_t K) { return (size_t)linear_plan(T, N, K, 2).total; }

size_t mx_weight_grad_workspace_bytes(int64_t T, int64_t N, int64_t K, int t)
{
    return (size_t)wgrad_plan(T, N, K, t == SPEC_BF16 ? 2 : 4).total;
}

hipError_t launch_mx_linear(hipStream_t stream, const void *X, int t, int64_t T, int64_t N, int64_t K, int64_t ldx,
                            const spec_mx *W, void *Y, int64_t ldy, void *ws)
{
    if (T == 0) return hipSuccess;
    return t == SPEC_BF16 ? linear<ElBF16, ElBF16>(stream, X, ldx, nullptr, T, N, K, W, Y, ldy, (char *)ws)
                          : linear<ElF32, ElF32>(stream, X, ldx, nullptr, T, N, K, W, Y, ldy, (char *)ws);
}

hipError_t launch_mx_product(hipStream_t stream, const spec_mx *X, const spec_mx *W, int64_t T, int64_t N, int64_t K,
                             void *Y, int yt, int64_t ldy, void *ws)
{
    if (T == 0) return hipSuccess;
    return yt == SPEC_BF16 ? linear<ElBF16, ElBF16>(stream, nullptr, 0, X, T, N, K, W, Y, ldy, (char *)ws)
                           : linear<ElBF16, ElF32>(stream, nullptr, 0, X, T, N, K, W, Y, ldy, (char *)ws);
}

hipError_t launch_mx_weight_grad(hipStream_t stream, const void *dY, int t, int64_t T, int64_t N, int64_t K, int64_t ldy,
                                 const spec_mx *X, float beta, void *dW, int64_t lddw, void *ws)
{
    return t == SPEC_BF16 ? wgrad<ElBF16>(stream, dY, ldy, T, N, K, X, beta, dW, lddw, (char *)ws)
                          : wgrad<ElF32>(stream, dY, ldy, T, N, K, X, beta, dW, lddw, (char *)ws);
}
