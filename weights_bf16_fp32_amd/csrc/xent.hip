// Softmax cross entropy of a linear head over a large vocabulary, gfx950:
//
//   z_tv = scale <h_t, w_v>,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target
//   g_tv = scale dloss_t (exp(z_tv - lse_t) - [v = target_t]),  dH = G W,  dW = beta dW + G^T H
//
// The T x V logits are never stored.  Forward: every tile of logits (256 x 256, 128 x
// 128, or 128 entries by 32 tokens) is reduced to one (maximum, sum of exponentials) per row while it is in the
// accumulators, and the tiles' pairs are joined per row.  Backward: a piece of
// the vocabulary at a time, the logits are formed again and leave as the bf16 (f32)
// gradient G of that piece, which the two gradient products read back.
//
// Rows without a target (outside [0, V)) are dropped before the products: the
// rest of H is packed, so they cost nothing, and whatever they hold (NaN
// included) reaches no output.  The number of rows left is known on the device
// only: grids are sized for all of them, and the workgroups of the first tiles
// (counted with the number left, so that they spread over the XCDs) do the work.
//
// Bound by the MFMAs (53 to 64 % busy at the clock that their power leaves): at
// 6144 targets x 131072 x 4096 bf16 the forward takes 5.5 to 5.8 ms (1140 to 1190
// TFLOP/s), the gradients 0.74 to 0.80 ms each of logits, dW and dH per piece of
// 16384 (1030 to 1110 TFLOP/s).
// Storing the logits would save the second forming of them, a quarter of the
// operations, for T x V x 4 bytes.  Eight rows of 65536 x 4096 are bound by reading W:
// 121 us, 4.4 TB/s.
//
//   k_xent_pack      positions of the rows with a target, their rows of H, packed
//   k_xent_wpack     a piece of W with 16-byte rows (only where W has none)
//   k_xent_fwd       logits tile -> (max, sum) per row, the target's logit
//   k_xent_join      lse and loss of every row
//   k_xent_g         logits tile -> G tile
//   k_xent_dw        dW of the piece
//   k_xent_dh        dH of the piece, added to the sums so far (f32)
//   k_xent_dh_out    dH from the sums, zero rows for rows without a target
#include <algorithm>

#include "internal.h"
#include "mm.h"

namespace {

inline int64_t cdiv_h(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up_h(int64_t a, int64_t b) { return cdiv_h(a, b) * b; }

SPEC_DEVICE int64_t load_id(const void *p, int is64, int64_t i)
{
    return is64 ? reinterpret_cast<const int64_t *>(p)[i] : (int64_t) reinterpret_cast<const int32_t *>(p)[i];
}

// Rows per workgroup of k_xent_pack: few, so that the copies fill the chip; more
// where many workgroups would each count the targets before theirs (the counting
// grows with the square of T).  The forward with 8 and with 64, a vocabulary of 1000:
// 8192 rows of 64 bf16 21.5 and 23.1 us, 16384 34.4 and 34.4, 32768 74 and 58, 65536
// 200 and 131; 16384 rows of 2048 93 and 98, 32768 193 and 187.
inline int pack_rows(int64_t T) { return T <= 16384 ? 8 : 64; }

// a row of d elements to one of dp, zero past d: 16 bytes at a time where both
// ends are aligned, else by element
template <typename S>
SPEC_DEVICE void copy_row(const S *__restrict__ src, S *__restrict__ dst, int64_t d, int64_t dp, bool vec, int lane)
{
    constexpr int EPC = 16 / (int)sizeof(S);
    if (vec) {
        const uint4 *s = reinterpret_cast<const uint4 *>(src);
        uint4 *o = reinterpret_cast<uint4 *>(dst);
        const int64_t n = d / EPC;
        int64_t c = lane;
        for (; c + 192 < n; c += 256) {  // four in flight per lane
            const uint4 a = s[c], b = s[c + 64], e = s[c + 128], f = s[c + 192];
            o[c] = a, o[c + 64] = b, o[c + 128] = e, o[c + 192] = f;
        }
        for (; c < dp / EPC; c += 64) o[c] = c < n ? s[c] : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll 8
        for (int64_t c = lane; c < dp; c += 64) dst[c] = c < d ? src[c] : (S)0;
    }
}

template <typename E>
__global__ __launch_bounds__(256) void k_xent_pack(const typename E::st *__restrict__ H, int64_t ldh, int64_t d,
                                                   int64_t dp, int vec, const void *__restrict__ target, int is64,
                                                   int64_t T, int64_t V, typename E::st *__restrict__ Hp,
                                                   int *__restrict__ pos, int *__restrict__ row, int *__restrict__ ptgt,
                                                   const float *__restrict__ lse, const float *__restrict__ dloss,
                                                   float *__restrict__ plse, float *__restrict__ pdl,
                                                   int *__restrict__ nvalid, int rows)
{
    __shared__ int cnt[4], where[64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * rows;
    int before = 0;  // rows with a target before this block's
    for (int64_t t = tid; t < t0; t += 256) {
        const int64_t y = load_id(target, is64, t);
        before += y >= 0 && y < V;
    }
    for (int o = 32; o > 0; o >>= 1) before += __shfl_xor(before, o);
    if (lane == 0) cnt[wave] = before;
    __syncthreads();
    before = cnt[0] + cnt[1] + cnt[2] + cnt[3];
    if (wave == 0) {
        const int64_t t = t0 + lane;
        const bool in = lane < rows && t < T;
        const int64_t y = in ? load_id(target, is64, t) : -1;
        const bool ok = y >= 0 && y < V;
        const uint64_t m = __ballot(ok);
        const int p = before + __popcll(m & ((1ull << lane) - 1));
        if (lane < rows) where[lane] = ok ? p : -1;
        if (in) pos[t] = ok ? p : -1;
        if (ok) {
            ptgt[p] = (int)y;
            row[p] = (int)t;
            if (lse != nullptr) {
                plse[p] = lse[t];
                pdl[p] = dloss[t];
            }
        }
        if (lane == 0 && t0 + rows >= T) *nvalid = before + __popcll(m);
    }
    __syncthreads();
    for (int r = wave; r < rows; r += 4) {
        const int p = where[r];
        if (p >= 0) copy_row(H + (t0 + r) * ldh, Hp + (int64_t)p * dp, d, dp, vec != 0, lane);
    }
}

template <typename E>
__global__ __launch_bounds__(256) void k_xent_wpack(const typename E::st *__restrict__ W, int64_t ldw, int64_t d,
                                                    int64_t dp, int64_t rows, typename E::st *__restrict__ Wp)
{
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r < rows) copy_row(W + r * ldw, Wp + r * dp, d, dp, false, threadIdx.x & 63);
}

// The logits of vocabulary rows [tile] (P) and packed tokens (Q).
template <typename M, typename E>
SPEC_DEVICE void logits(M &mm, const typename E::st *W, int64_t ldw, int64_t vn, const typename E::st *Hp, int64_t dp,
                        int n, int64_t d, int64_t v0, int t0, const typename M::Lds &lds, int BP, int BQ)
{
    constexpr int SZ = M::SZ;
    const MmSrc P{(const char *)(W + v0 * ldw), ldw * SZ, (int)min<int64_t>(BP, vn - v0), d};
    const MmSrc Q{(const char *)(Hp + (int64_t)t0 * dp), dp * SZ, min(BQ, n - t0), d};
    mm.run(P, Q, 0, d, lds);
}

// grid: tiles of [vn vocabulary rows] x [T tokens]; W's rows are vocabulary
// entries vbase .. vbase + vn - 1.  part[t][tile0 + tp] = (max, sum exp(z - max)).
// dk: d rounded up to 16 bytes (the padding of both operands is zero).
template <typename E, typename C>
__global__ MM_BOUNDS(C) void k_xent_fwd(const typename E::st *__restrict__ W, int64_t ldw,
                                                                  int64_t vn, int64_t vbase,
                                                                  const typename E::st *__restrict__ Hp, int64_t dp,
                                                                  int64_t dk, const int *__restrict__ nvalid, int np,
                                                                  float scale, const int *__restrict__ ptgt,
                                                                  float *__restrict__ ztgt, float2 *__restrict__ part,
                                                                  int64_t ldpart, int tile0)
{
    using M = Mm<E, C, false, false>;
    MM_STAGES(M);
    const int n = *nvalid, nq = (n + C::BQ - 1) / C::BQ;
    int tp, tq;
    if (blockIdx.x >= (unsigned)(np * nq)) return;
    mm_tile(blockIdx.x, np, nq, tp, tq);
    const int t0 = tq * C::BQ;
    const int64_t v0 = (int64_t)tp * C::BP;
    M mm;
    logits<M, E>(mm, W, ldw, vn, Hp, dp, n, dk, v0, t0, lds, C::BP, C::BQ);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wp = wave % C::WP;
    const int p0 = wp * (C::BP / C::WP) + 4 * (lane >> 5), q0 = (wave / C::WP) * (C::BQ / C::WQ) + (lane & 31);
    const int lim = (int)min<int64_t>(C::BP, vn - v0);
    float2 *red = reinterpret_cast<float2 *>(lds.p[0]);  // [wp][q] of the waves along the vocabulary
    static_assert(C::WP * C::BQ * sizeof(float2) <= M::P_BYTES, "room");
#pragma unroll
    for (int b = 0; b < M::NI; ++b) {
        const int q = q0 + 32 * b;
        const bool in = t0 + q < n;
#pragma unroll
        for (int m = 0; m < M::MI; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) mm.acc[m][b][e] *= scale;
        if (lim < C::BP) {  // the vocabulary ends in this tile
#pragma unroll
            for (int m = 0; m < M::MI; ++m)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (p0 + 32 * m + 8 * (e >> 2) + (e & 3) >= lim) mm.acc[m][b][e] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int m = 0; m < M::MI; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, mm.acc[m][b][e]);
        // few tiles hold a target of one of their rows
        const int64_t y = in ? (int64_t)ptgt[t0 + q] - vbase - v0 - p0 : -1;  // its place from this lane's first
        if (__any(y >= 0 && y < C::BP / C::WP)) {
            const int at = (int)max<int64_t>(-1, min<int64_t>(y, C::BP));
            float z = 0.f;
            bool mine = false;
#pragma unroll
            for (int m = 0; m < M::MI; ++m)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool here = at == 32 * m + 8 * (e >> 2) + (e & 3);
                    z = here ? mm.acc[m][b][e] : z;
                    mine |= here;
                }
            if (mine) ztgt[t0 + q] = z;
        }
        {
            float a = top, c = top;
            halfswap32(a, c);
            top = fmaxf(a, c);
        }
        // a tile without a finite logit sums to zero (or to NaN with NaN or +inf in it)
        const float ref = top == -INFINITY ? 0.f : top;
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < M::MI; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) s += __expf(mm.acc[m][b][e] - ref);
        s = pair32_sum(s);
        if (lane < 32) red[wp * C::BQ + q] = make_float2(top, s);
    }
    __syncthreads();
    for (int q = threadIdx.x; q < C::BQ; q += C::NT) {
        if (t0 + q >= n) break;
        float2 r = red[q];
#pragma unroll
        for (int w = 1; w < C::WP; ++w) {
            const float2 o = red[w * C::BQ + q];
            const float top = fmaxf(r.x, o.x), ref = top == -INFINITY ? 0.f : top;
            r.y = r.y * __expf(r.x - ref) + o.y * __expf(o.x - ref);
            r.x = top;
        }
        part[(int64_t)(t0 + q) * ldpart + tile0 + tp] = r;
    }
}

// one wave per row: the row's lse from its tiles' (max, sum) and its loss
__global__ __launch_bounds__(256) void k_xent_join(const float2 *__restrict__ part, int64_t ldpart, int ntile,
                                                   const int *__restrict__ pos, const float *__restrict__ ztgt,
                                                   int64_t T, float *__restrict__ loss, float *__restrict__ lse)
{
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (t >= T) return;
    const int p = pos[t];
    if (p < 0) {
        if (lane == 0) loss[t] = lse[t] = 0.f;
        return;
    }
    const float2 *r = part + (int64_t)p * ldpart;
    float top = -INFINITY, s = 0.f;
    for (int i = lane; i < ntile; i += 64) {
        const float2 o = r[i];
        const float m = fmaxf(top, o.x), ref = m == -INFINITY ? 0.f : m;
        s = s * __expf(top - ref) + o.y * __expf(o.x - ref);
        top = m;
    }
    for (int o = 32; o > 0; o >>= 1) {
        const float ot = __shfl_xor(top, o), os = __shfl_xor(s, o);
        const float m = fmaxf(top, ot), ref = m == -INFINITY ? 0.f : m;
        s = s * __expf(top - ref) + os * __expf(ot - ref);
        top = m;
    }
    if (lane == 0) {
        const float l = top == -INFINITY ? NAN : top + logf(s);  // no finite logit: as 0 / 0
        lse[t] = l;
        loss[t] = l - ztgt[p];
    }
}

// The factor that G is held without: the mantissa, in [1, 2), of the first row's
// weight.  With equal weights (the mean) the other factor is a power of two, and
// the entries near -1 of G, the targets hardly predicted, are exact in bf16; with
// the weights in it they would all be off by the same rounding of 1 / rows (0.2 %).
SPEC_DEVICE float grad_unit(const float *__restrict__ pdl, int n, float scale)
{
    const float w = n > 0 ? fabsf(pdl[0] * scale) : 0.f;
    return w > 0x1p-126f && w < INFINITY ? __uint_as_float((__float_as_uint(w) & 0x7fffffu) | 0x3f800000u) : 1.f;
}

// G[t][v - vbase], columns up to vn rounded up to 16 bytes (zero past vn)
template <typename E, typename C>
__global__ MM_BOUNDS(C) void k_xent_g(const typename E::st *__restrict__ W, int64_t ldw,
                                                                int64_t vn, int64_t vbase,
                                                                const typename E::st *__restrict__ Hp, int64_t dp,
                                                                int64_t dk, const int *__restrict__ nvalid, int np,
                                                                float scale, const int *__restrict__ ptgt,
                                                                const float *__restrict__ plse,
                                                                const float *__restrict__ pdl,
                                                                typename E::st *__restrict__ G, int64_t ldg)
{
    using M = Mm<E, C, false, false>;
    MM_STAGES(M);
    const int n = *nvalid, nq = (n + C::BQ - 1) / C::BQ;
    int tp, tq;
    if (blockIdx.x >= (unsigned)(np * nq)) return;
    mm_tile(blockIdx.x, np, nq, tp, tq);
    const int t0 = tq * C::BQ;
    const int64_t v0 = (int64_t)tp * C::BP;
    M mm;
    logits<M, E>(mm, W, ldw, vn, Hp, dp, n, dk, v0, t0, lds, C::BP, C::BQ);
    const int lim = (int)min<int64_t>(C::BP, vn - v0);
    const int lim4 = (int)min<int64_t>(C::BP, round_up(vn, M::EPC) - v0);
    struct Row {
        int y;
        float lse, w;
    };
    const float unit = grad_unit(pdl, n, scale);
    mm.each4(lds, [&](int p, int q) {
        return t0 + q < n ? Row{ptgt[t0 + q], plse[t0 + q], pdl[t0 + q] * scale / unit} : Row{};
    }, [&](int p, int q, float (&v)[4], const Row &r) {
        if (t0 + q >= n || p >= lim4) return;
        const int64_t y = r.y - vbase - v0;
        const float l = r.lse, w = r.w;
        Vec4<E> o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o.v[e] = E::round(p + e < lim ? (__expf(scale * v[e] - l) - (p + e == y ? 1.f : 0.f)) * w : 0.f);
        *reinterpret_cast<Vec4<E> *>(G + (int64_t)(t0 + q) * ldg + v0 + p) = o;
    });
}

// dW rows v (Q) by columns of d (P): sum over tokens of H[t][p] G[t][q]
template <typename E, typename C>
__global__ MM_BOUNDS(C) void k_xent_dw(const typename E::st *__restrict__ Hp, int64_t dp,
                                                                 const typename E::st *__restrict__ G, int64_t ldg,
                                                                 int64_t vn, int64_t d, const int *__restrict__ nvalid,
                                                                 int np, int nq, const float *__restrict__ pdl,
                                                                 float scale, typename E::st *__restrict__ dW,
                                                                 int64_t lddw, float beta, int vec)
{
    using M = Mm<E, C, true, true>;
    MM_STAGES(M);
    int tp, tq;
    mm_tile(blockIdx.x, np, nq, tp, tq);
    const int64_t n = *nvalid, p0 = (int64_t)tp * C::BP, v0 = (int64_t)tq * C::BQ;
    const MmSrc P{(const char *)(Hp + p0), dp * M::SZ, (int)min<int64_t>(C::BP, d - p0), n};
    const MmSrc Q{(const char *)(G + v0), ldg * M::SZ, (int)min<int64_t>(C::BQ, vn - v0), n};
    M mm;
    mm.run(P, Q, 0, n, lds);
    const float unit = grad_unit(pdl, (int)n, scale);
    mm.each4(lds, [&](int p, int q, float (&v)[4]) {
        if (q >= Q.lim || p >= P.lim) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= unit;
        typename E::st *o = dW + (v0 + q) * lddw + p0 + p;
        if (vec && p + 4 <= P.lim) {
            Vec4<E> r;
            if (beta != 0.f) r = *reinterpret_cast<const Vec4<E> *>(o);
#pragma unroll
            for (int e = 0; e < 4; ++e) r.v[e] = E::round(beta != 0.f ? v[e] + beta * E::wide(r.v[e]) : v[e]);
            *reinterpret_cast<Vec4<E> *>(o) = r;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (p + e < P.lim) o[e] = E::round(beta != 0.f ? v[e] + beta * E::wide(o[e]) : v[e]);
        }
    });
}

// How the tiles of dH are dealt out.  Rounds of `slots` workgroups (those the
// chip runs at once) take whole tiles; the tiles of a last round that leaves
// half of it or more idle are split along the vocabulary, as many ways as fill it.
struct DhPlan {
    int whole;   // tiles taken whole
    int ways;    // shares of each of the others
    int units;   // workgroups with work
};
SPEC_DEVICE DhPlan dh_plan(int tiles, int slots, int most)
{
    const int left = tiles % slots;
    const int ways = left > 0 ? max(1, min(most, slots / left)) : 1;
    const int whole = ways > 1 ? tiles - left : tiles;
    return {whole, ways, whole + (tiles - whole) * ways};
}

// part[t][p] (+)= sum over v of W[v][p] G[t][v] over the piece; the shares after
// the first of a split tile have a tile of their own in `extra`
template <typename E, typename C>
__global__ MM_BOUNDS(C) void k_xent_dh(const typename E::st *__restrict__ W, int64_t ldw,
                                       const typename E::st *__restrict__ G, int64_t ldg, int64_t vn, int64_t d,
                                       const int *__restrict__ nvalid, int np, int slots, int most,
                                       float *__restrict__ part, int64_t ldp, float *__restrict__ extra, int first)
{
    using M = Mm<E, C, true, false>;
    MM_STAGES(M);
    const int n = *nvalid, nq = (n + C::BQ - 1) / C::BQ, u = blockIdx.x;
    const DhPlan pl = dh_plan(np * nq, slots, most);
    if (u >= pl.units) return;
    int id = u, share = 0;
    int64_t kb = 0, ke = vn;
    if (u >= pl.whole && pl.ways > 1) {
        id = pl.whole + (u - pl.whole) / pl.ways;
        share = (u - pl.whole) % pl.ways;
        const int64_t per = round_up((vn + pl.ways - 1) / pl.ways, 64);
        kb = share * per;
        ke = min<int64_t>(vn, kb + per);
    }
    int tp, tq;
    mm_tile(id, np, nq, tp, tq);
    const int t0 = tq * C::BQ;
    const int64_t p0 = (int64_t)tp * C::BP;
    const MmSrc P{(const char *)(W + p0), ldw * M::SZ, (int)min<int64_t>(C::BP, d - p0), ke};
    const MmSrc Q{(const char *)(G + (int64_t)t0 * ldg), ldg * M::SZ, min(C::BQ, n - t0), round_up(ke, M::EPC)};
    M mm;
    mm.run(P, Q, kb, ke, lds);
    float *out = part + (int64_t)t0 * ldp + p0;
    if (share > 0) {
        out = extra + (int64_t)(u - pl.whole) * C::BP * C::BQ;
        ldp = C::BP;
    }
    // (ldp is a multiple of 4: a group of four lies in its row)
    const auto at = [&](int p, int q) { return reinterpret_cast<float4 *>(out + (int64_t)q * ldp + p); };
    mm.each4(lds, [&](int p, int q) {
        return first || q >= Q.lim || p >= P.lim ? make_float4(0.f, 0.f, 0.f, 0.f) : *at(p, q);
    }, [&](int p, int q, float (&v)[4], const float4 &a) {
        if (q < Q.lim && p < P.lim) *at(p, q) = make_float4(v[0] + a.x, v[1] + a.y, v[2] + a.z, v[3] + a.w);
    });
}

constexpr int OUT_ROWS = 16;  // rows of a tile per workgroup of k_xent_dh_out

// grid: tiles x (BQ / OUT_ROWS) workgroups that round the sums of their rows,
// then cdiv(T, 4) that write the rows without a target
template <typename E, typename C>
__global__ __launch_bounds__(256) void k_xent_dh_out(const float *__restrict__ part, int64_t ldp,
                                                     const float *__restrict__ extra, const int *__restrict__ nvalid,
                                                     int np, int nqmax, int slots, int most, int64_t T, int64_t d,
                                                     const int *__restrict__ pos, const int *__restrict__ row,
                                                     const float *__restrict__ pdl, float scale,
                                                     typename E::st *__restrict__ dH, int64_t lddh, int vec)
{
    constexpr int G = C::BQ / OUT_ROWS;
    const int lane = threadIdx.x & 63;
    const int64_t tileblocks = (int64_t)np * nqmax * G;
    if (blockIdx.x >= tileblocks) {
        const int64_t t = ((int64_t)blockIdx.x - tileblocks) * 4 + (threadIdx.x >> 6);
        if (t < T && pos[t] < 0)
            for (int64_t c = lane; c < d; c += 64) dH[t * lddh + c] = (typename E::st)0;
        return;
    }
    const int n = *nvalid, nq = (n + C::BQ - 1) / C::BQ;
    const DhPlan pl = dh_plan(np * nq, slots, most);
    const int id = (int)(blockIdx.x / G), r0 = (int)(blockIdx.x % G) * OUT_ROWS;
    if (id >= np * nq) return;
    int tp, tq;
    mm_tile(id, np, nq, tp, tq);
    const int64_t p0 = (int64_t)tp * C::BP;
    const int shares = id >= pl.whole ? pl.ways : 1;
    const float unit = grad_unit(pdl, n, scale);
    const float *ex = extra + (int64_t)(id - pl.whole) * pl.ways * C::BP * C::BQ;
    for (int i = threadIdx.x; i < OUT_ROWS * (C::BP / 4); i += 256) {
        const int q = r0 + i / (C::BP / 4), p = 4 * (i % (C::BP / 4)), t = tq * C::BQ + q;
        if (t >= n || p0 + p >= d) continue;
        float4 s = *reinterpret_cast<const float4 *>(part + (int64_t)t * ldp + p0 + p);
        for (int k = 1; k < shares; ++k) {
            const float4 a = *reinterpret_cast<const float4 *>(ex + ((int64_t)k * C::BQ + q) * C::BP + p);
            s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
        }
        typename E::st *o = dH + (int64_t)row[t] * lddh + p0 + p;
        const float v[4] = {s.x * unit, s.y * unit, s.z * unit, s.w * unit};
        if (vec && p0 + p + 4 <= d) {
            Vec4<E> x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x.v[e] = E::round(v[e]);
            *reinterpret_cast<Vec4<E> *>(o) = x;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (p0 + p + e < d) o[e] = E::round(v[e]);
        }
    }
}

// ------------------------------------------------------------------ sizes

// Bytes of a piece's gradient G, and of its rows of W (copied where they are not
// aligned), at most, but no fewer than 2048 entries (or V): G is larger from 65536
// bf16 rows on, 4 KB per row.  Larger pieces add into the f32 partial dH less
// often (100 MB read and written per piece at 6144 x 4096).
constexpr int64_t XENT_PIECE_BYTES = (int64_t)256 << 20;

struct XentPlan {
    int64_t dp;      // row of packed H and W: d rounded up to 64 elements
    int64_t dk;      // d rounded up to 16 bytes
    int64_t piece;   // vocabulary entries per piece
    int most;        // shares of a tile of dH at most: 512 vocabulary entries each
    bool big;        // dH in 256 x 256 tiles
    int slots;       // and how many of its workgroups run at once
    // byte offsets into the workspace
    int64_t pos, row, ptgt, plse, pdl, nvalid, hp, wp, ztgt, part, extra, g, total;
};

XentPlan xent_plan(int64_t T, int64_t V, int64_t d, int t, bool grad)
{
    XentPlan p{};
    const int64_t es = t == SPEC_BF16 ? 2 : 4;
    p.dp = up_h(d, 64);
    p.dk = up_h(d, 16 / es);
    const int64_t Tn = std::max<int64_t>(T, 1);
    p.piece = std::max<int64_t>(2048, XENT_PIECE_BYTES / (es * std::max(Tn, p.dp)) / 256 * 256);
    p.piece = std::min<int64_t>(p.piece, up_h(V, 256));
    p.most = (int)std::max<int64_t>(1, std::min<int64_t>(p.piece / 512, 64));
    p.big = cdiv_h(T, 256) * cdiv_h(d, 256) >= 128;  // fewer are split, and smaller ones split finer
    p.slots = p.big ? 256 : 512;
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += up_h(bytes, 256);
        return at;
    };
    p.nvalid = take(4);
    p.pos = take(4 * Tn);
    p.row = take(4 * Tn);
    p.ptgt = take(4 * Tn);
    p.hp = take(es * Tn * p.dp);
    p.wp = take(es * p.piece * p.dp);
    if (grad) {
        p.plse = take(4 * Tn);
        p.pdl = take(4 * Tn);
        p.g = take(es * Tn * p.piece);
        p.part = take((int64_t)4 * Tn * up_h(d, 4));
        p.extra = take((int64_t)4 * 256 * 256 * 256);
    } else {
        p.ztgt = take(4 * Tn);
        p.part = take(8 * Tn * cdiv_h(V, 128));
    }
    p.total = o;
    return p;
}

template <typename E>
hipError_t pack(hipStream_t stream, const XentPlan &pl, const void *H, int64_t ldh, const void *target, int is64,
                const float *lse, const float *dloss, int64_t T, int64_t V, int64_t d, char *ws)
{
    using st = typename E::st;
    const int vec = (uintptr_t)H % 16 == 0 && ldh * sizeof(st) % 16 == 0 && d * sizeof(st) % 16 == 0;
    hipLaunchKernelGGL(k_xent_pack<E>, dim3((unsigned)cdiv_h(T, pack_rows(T))), dim3(256), 0, stream, (const st *)H, ldh, d,
                       pl.dp, vec, target, is64, T, V, (st *)(ws + pl.hp), (int *)(ws + pl.pos), (int *)(ws + pl.row), (int *)(ws + pl.ptgt),
                       lse, dloss, (float *)(ws + pl.plse), (float *)(ws + pl.pdl), (int *)(ws + pl.nvalid), pack_rows(T));
    return hipGetLastError();
}

// W as the products can read it: itself where its rows are 16-byte aligned, else a packed piece
template <typename E>
bool direct_w(const void *W, int64_t ldw, int64_t d)
{
    const int64_t es = sizeof(typename E::st);
    return (uintptr_t)W % 16 == 0 && ldw * es % 16 == 0 && d * es % 16 == 0;
}

template <typename E>
hipError_t wpiece(hipStream_t stream, const XentPlan &pl, const typename E::st *W, int64_t &ldw, int64_t d, int64_t vn,
                  bool direct, char *ws, const typename E::st *&out)
{
    using st = typename E::st;
    out = W;
    if (direct) return hipSuccess;
    hipLaunchKernelGGL(k_xent_wpack<E>, dim3((unsigned)cdiv_h(vn, 4)), dim3(256), 0, stream, W, ldw, d, pl.dp, vn,
                       (st *)(ws + pl.wp));
    out = (const st *)(ws + pl.wp);
    ldw = pl.dp;
    return hipGetLastError();
}

// 256 x 256 tiles or 128 x 128: those with which the busiest of 256 CUs has less to
// do, a small tile's results taking 1.28 (16 bits) or 1.03 (f32) times as long.
template <typename E>
inline bool big_tiles(int64_t rows, int64_t cols)
{
    const double per = sizeof(typename E::st) == 2 ? 1.28 : 1.03;
    const auto most = [&](int64_t e) { return (double)cdiv_h(cdiv_h(rows, e) * cdiv_h(cols, e), 256) * (double)(e * e); };
    return most(256) <= per * most(128);
}

// The logits of up to this many tokens take the tile for few rows.  In f32, bound
// by the MFMAs over all of a tile's rows, it takes 207 us against 509 of the other
// tiles for 8 tokens of 65536 x 4096, 351 against 514 for 64.  In bf16, bound by W,
// 130 against 133 for 32; for 33 to 64 its two tiles per strip of W read it twice: 143
// against 134, and 38 against 32 of 50021 x 1000, but 18 against 22 of 8192 x 1024
// and 576 against 593 for the gradients of 64 tokens of 65536 x 4096.
constexpr int64_t FEW_TOKENS = 64;

template <typename E, typename C>
hipError_t fwd_piece(hipStream_t stream, const XentPlan &pl, const typename E::st *W, int64_t ldw, int64_t vn, int64_t v,
                     int64_t T, float scale, int64_t ldpart, char *ws)
{
    // (one launch unless it would have more threads than a launch holds)
    const int nq = (int)cdiv_h(T, C::BQ);
    const int64_t most = LAUNCH_THREADS / C::NT / nq * C::BP;
    for (int64_t v0 = 0; v0 < vn; v0 += most) {
        const int64_t n = std::min(most, vn - v0);
        const int np = (int)cdiv_h(n, C::BP);
        hipLaunchKernelGGL((k_xent_fwd<E, C>), dim3((unsigned)((int64_t)np * nq)), dim3(C::NT), 0, stream, W + v0 * ldw,
                           ldw, n, v + v0, (const typename E::st *)(ws + pl.hp), pl.dp, pl.dk,
                           (const int *)(ws + pl.nvalid), np, scale, (const int *)(ws + pl.ptgt), (float *)(ws + pl.ztgt),
                           (float2 *)(ws + pl.part), ldpart, (int)((v + v0) / C::BP));
        SPEC_LAUNCH_CHECK();
    }
    return hipSuccess;
}

template <typename E, typename C>
hipError_t g_piece(hipStream_t stream, const XentPlan &pl, const typename E::st *W, int64_t ldw, int64_t vn, int64_t v,
                   int64_t T, float scale, char *ws)
{
    using st = typename E::st;
    const int np = (int)cdiv_h(vn, C::BP), nq = (int)cdiv_h(T, C::BQ);
    hipLaunchKernelGGL((k_xent_g<E, C>), dim3((unsigned)((int64_t)np * nq)), dim3(C::NT), 0, stream, W, ldw, vn,
                       v, (const st *)(ws + pl.hp), pl.dp, pl.dk, (const int *)(ws + pl.nvalid), np, scale,
                       (const int *)(ws + pl.ptgt), (const float *)(ws + pl.plse), (const float *)(ws + pl.pdl),
                       (st *)(ws + pl.g), pl.piece);
    return hipGetLastError();
}

template <typename E, typename C>
hipError_t dw_piece(hipStream_t stream, const XentPlan &pl, int64_t vn, int64_t d, float scale, typename E::st *dW,
                    int64_t lddw, float beta, char *ws)
{
    using st = typename E::st;
    const int np = (int)cdiv_h(d, C::BP), nq = (int)cdiv_h(vn, C::BQ);
    const int vec = (uintptr_t)dW % (4 * sizeof(st)) == 0 && lddw % 4 == 0;
    hipLaunchKernelGGL((k_xent_dw<E, C>), dim3((unsigned)((int64_t)np * nq)), dim3(C::NT), 0, stream,
                       (const st *)(ws + pl.hp), pl.dp, (const st *)(ws + pl.g), pl.piece, vn, d,
                       (const int *)(ws + pl.nvalid), np, nq, (const float *)(ws + pl.pdl), scale, dW, lddw, beta, vec);
    return hipGetLastError();
}

template <typename E, typename C>
hipError_t dh_piece(hipStream_t stream, const XentPlan &pl, const typename E::st *W, int64_t ldw, int64_t vn, int64_t T,
                    int64_t d, bool first, char *ws)
{
    const int np = (int)cdiv_h(d, C::BP), nq = (int)cdiv_h(T, C::BQ);
    // whole tiles of every round, then at most one round of shares
    const int64_t grid = (int64_t)np * nq + pl.slots;
    hipLaunchKernelGGL((k_xent_dh<E, C>), dim3((unsigned)grid), dim3(C::NT), 0, stream, W, ldw,
                       (const typename E::st *)(ws + pl.g), pl.piece, vn, d, (const int *)(ws + pl.nvalid), np, pl.slots,
                       pl.most, (float *)(ws + pl.part), up_h(d, 4), (float *)(ws + pl.extra), first);
    return hipGetLastError();
}

template <typename E, typename C>
hipError_t dh_out(hipStream_t stream, const XentPlan &pl, int64_t T, int64_t d, float scale, void *dH, int64_t lddh,
                  char *ws)
{
    using st = typename E::st;
    const int np = (int)cdiv_h(d, C::BP), nq = (int)cdiv_h(T, C::BQ);
    const int64_t grid = (int64_t)np * nq * (C::BQ / OUT_ROWS) + cdiv_h(T, 4);
    const int vec = (uintptr_t)dH % (4 * sizeof(st)) == 0 && lddh % 4 == 0;
    hipLaunchKernelGGL((k_xent_dh_out<E, C>), dim3((unsigned)grid), dim3(256), 0, stream, (const float *)(ws + pl.part),
                       up_h(d, 4), (const float *)(ws + pl.extra), (const int *)(ws + pl.nvalid), np, nq, pl.slots,
                       pl.most, T, d, (const int *)(ws + pl.pos), (const int *)(ws + pl.row), (const float *)(ws + pl.pdl), scale, (st *)dH,
                       lddh, vec);
    return hipGetLastError();
}

template <typename E>
hipError_t xent_fwd(hipStream_t stream, const void *H, int64_t ldh, const void *W, int64_t ldw, const void *target,
                    int is64, int64_t T, int64_t V, int64_t d, float scale, float *loss, float *lse, char *ws)
{
    using st = typename E::st;
    const XentPlan pl = xent_plan(T, V, d, sizeof(st) == 2 ? SPEC_BF16 : SPEC_F32, false);
    hipError_t e = pack<E>(stream, pl, H, ldh, target, is64, nullptr, nullptr, T, V, d, ws);
    if (e != hipSuccess) return e;
    const bool direct = direct_w<E>(W, ldw, d), big = T > FEW_TOKENS && big_tiles<E>(T, V);
    const int64_t piece = direct ? V : pl.piece, ldpart = cdiv_h(V, big ? 256 : 128);
    for (int64_t v = 0; v < V; v += piece) {
        const int64_t vn = std::min(piece, V - v);
        int64_t ld = ldw;
        const st *Wv;
        e = wpiece<E>(stream, pl, (const st *)W + v * ldw, ld, d, vn, direct, ws, Wv);
        if (e != hipSuccess) return e;
        e = T <= FEW_TOKENS ? fwd_piece<E, TileRow>(stream, pl, Wv, ld, vn, v, T, scale, ldpart, ws)
            : big           ? fwd_piece<E, Tile256>(stream, pl, Wv, ld, vn, v, T, scale, ldpart, ws)
                            : fwd_piece<E, Tile128>(stream, pl, Wv, ld, vn, v, T, scale, ldpart, ws);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_xent_join, dim3((unsigned)cdiv_h(T, 4)), dim3(256), 0, stream, (const float2 *)(ws + pl.part),
                       ldpart, (int)ldpart, (const int *)(ws + pl.pos), (const float *)(ws + pl.ztgt), T, loss, lse);
    return hipGetLastError();
}

template <typename E>
hipError_t xent_grad(hipStream_t stream, const void *H, int64_t ldh, const void *W, int64_t ldw, const void *target,
                     int is64, int64_t T, int64_t V, int64_t d, float scale, const float *lse, const float *dloss,
                     void *dH, int64_t lddh, void *dW, int64_t lddw, float beta, char *ws)
{
    using st = typename E::st;
    const XentPlan pl = xent_plan(T, V, d, sizeof(st) == 2 ? SPEC_BF16 : SPEC_F32, true);
    hipError_t e = pack<E>(stream, pl, H, ldh, target, is64, lse, dloss, T, V, d, ws);
    if (e != hipSuccess) return e;
    const bool direct = direct_w<E>(W, ldw, d);
    for (int64_t v = 0; v < V; v += pl.piece) {
        const int64_t vn = std::min(pl.piece, V - v);
        int64_t ld = ldw;
        const st *Wv;
        st *dWv = (st *)dW + v * lddw;
        e = wpiece<E>(stream, pl, (const st *)W + v * ldw, ld, d, vn, direct, ws, Wv);
        if (e != hipSuccess) return e;
        e = T <= FEW_TOKENS      ? g_piece<E, TileRow>(stream, pl, Wv, ld, vn, v, T, scale, ws)
            : big_tiles<E>(T, vn) ? g_piece<E, Tile256>(stream, pl, Wv, ld, vn, v, T, scale, ws)
                                 : g_piece<E, Tile128>(stream, pl, Wv, ld, vn, v, T, scale, ws);
        if (e != hipSuccess) return e;
        e = big_tiles<E>(vn, d) ? dw_piece<E, Tile256>(stream, pl, vn, d, scale, dWv, lddw, beta, ws)
                             : dw_piece<E, Tile128>(stream, pl, vn, d, scale, dWv, lddw, beta, ws);
        if (e != hipSuccess) return e;
        e = pl.big ? dh_piece<E, Tile256>(stream, pl, Wv, ld, vn, T, d, v == 0, ws)
                   : dh_piece<E, Tile128>(stream, pl, Wv, ld, vn, T, d, v == 0, ws);
        if (e != hipSuccess) return e;
    }
    return pl.big ? dh_out<E, Tile256>(stream, pl, T, d, scale, dH, lddh, ws)
                  : dh_out<E, Tile128>(stream, pl, T, d, scale, dH, lddh, ws);
}

// dW <- beta dW where no token has a target to add
template <typename E>
__global__ __launch_bounds__(256) void k_xent_scale(typename E::st *__restrict__ dW, int64_t lddw, int64_t V, int64_t d,
                                                    float beta)
{
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {
        typename E::st *r = dW + v * lddw;
        for (int64_t c = threadIdx.x; c < d; c += 256) r[c] = E::round(beta != 0.f ? beta * E::wide(r[c]) : 0.f);
    }
}

}  // namespace

size_t linear_xent_workspace_bytes(int64_t T, int64_t V, int64_t d, int t)
{
    return (size_t)xent_plan(T, V, d, t, false).total;
}

size_t linear_xent_grad_workspace_bytes(int64_t T, int64_t V, int64_t d, int t)
{
    return (size_t)xent_plan(T, V, d, t, true).total;
}

hipError_t launch_linear_xent(hipStream_t stream, const void *H, const void *W, int t, int64_t T, int64_t V, int64_t d,
                              int64_t ldh, int64_t ldw, const void *target, int is64, float scale, float *loss,
                              float *lse, void *ws)
{
    if (T == 0) return hipSuccess;
    return t == SPEC_BF16 ? xent_fwd<ElBF16>(stream, H, ldh, W, ldw, target, is64, T, V, d, scale, loss, lse, (char *)ws)
                          : xent_fwd<ElF32>(stream, H, ldh, W, ldw, target, is64, T, V, d, scale, loss, lse, (char *)ws);
}

hipError_t launch_linear_xent_grad(hipStream_t stream, const void *H, const void *W, int t, int64_t T, int64_t V,
                                   int64_t d, int64_t ldh, int64_t ldw, const void *target, int is64, float scale,
                                   const float *lse, const float *dloss, void *dH, int64_t lddh, void *dW, int64_t lddw,
                                   float beta, void *ws)
{
    if (T == 0) {
        const dim3 grid((unsigned)std::min(V, LAUNCH_THREADS / 256));
        if (t == SPEC_BF16)
            hipLaunchKernelGGL(k_xent_scale<ElBF16>, grid, dim3(256), 0, stream, (uint16_t *)dW, lddw, V, d, beta);
        else
            hipLaunchKernelGGL(k_xent_scale<ElF32>, grid, dim3(256), 0, stream, (float *)dW, lddw, V, d, beta);
        return hipGetLastError();
    }
    return t == SPEC_BF16 ? xent_grad<ElBF16>(stream, H, ldh, W, ldw, target, is64, T, V, d, scale, lse, dloss, dH, lddh,
                                              dW, lddw, beta, (char *)ws)
                          : xent_grad<ElF32>(stream, H, ldh, W, ldw, target, is64, T, V, d, scale, lse, dloss, dH, lddh,
                                             dW, lddw, beta, (char *)ws);
}
