// The norms around a residual block, its gate and its residual sum in one pass, and
// their gradients, gfx950.  Per row (d features; f32 throughout):
//
//   n1 = y r1, r1 = (mean y^2 + eps)^(-1/2)      u = n1 w1        (or n1 = u = y, not normed)
//   h' = alpha h + beta g u
//   n2 = h' r2, r2 = (mean h'^2 + eps)^(-1/2)    x = n2 w2
//
// and backwards, from dx and dh':
//
//   a = dx w2,  m = mean(a n2),  G = dh' + r2 (a - n2 m)            dh = alpha G
//   c = beta g w1 n1,  b = beta g w1 G                          dy = r1 (b - n1 mean(b n1))  (or b)
//   dw2 = sum dx n2,  s_k = beta sum over rows of gate row k of G n1,
//   dw1 = sum over k of g_k s_k,  dg_k = w1 s_k
//
// mean(b n1) = mean(c (dh' + r2 a)) - r2 m mean(c n2), so one reduction per row
// gives all three means.
//
// Bound by memory: the forward reads y and h and writes h' and x, the gradients read
// dx, dh', y and h' and write dh and dy.  A row is held in the registers of one wave
// (short rows) or one workgroup; its threads keep their columns from row to row, so
// the weights are read once per workgroup, and the sums over rows stay in registers
// until the end of the workgroup's run of rows.  The runs' sums are joined by a
// second launch, in order: no atomics, the same result in every run.
//
// A row is requested while the one before it is worked on, by loads without branches
// (a branch around a load makes the compiler wait for it: 16384 x 4096 bf16 gradients took
// 186 us so, 157 without).  16384 x 4096 bf16, a call among others: forward 107 us, 5.0 TB/s;
// with all three matrices stored in 8 bits too 152 us, 4.9 TB/s; the norm alone 43 us, 6.2 TB/s
// (H partly from the caches); gradients from the matrices 180 us, 4.5 TB/s, from 8-bit storage 156 us,
// 4.3 TB/s, the vector work between the loads in their way, 8.5 us of each the join.
// 2047 x 1000 f32 gradients are 14.7 and 4.0 us of kernels.  One eight of a row per thread is slower
// in the forward (142 us), two are in the gradients (280 us: 256 registers).  Gradients of
// f32 rows past 4096 features and of all past 8192 spill: 8192 x 4097 f32 494 us, 1.6 TB/s,
// 4096 x 16384 bf16 490 to 540 us, 1.6 TB/s.
#include <algorithm>

#include "mx.h"

namespace {

inline int64_t cdiv_h(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up_h(int64_t a, int64_t b) { return cdiv_h(a, b) * b; }

// TPR threads hold a row, CH eights each: eight i of a thread lies at 8 (i TPR + thread).
// Rows of one wave go four to a workgroup.
// Rows of fewer than eight are TINY.
template <int TPR_, int CH_, bool TINY_ = false>
struct RowShape {
    static constexpr int TPR = TPR_, CH = CH_;
    static constexpr bool TINY = TINY_;
    static constexpr int NT = TPR == 64 ? 256 : TPR;
    static constexpr int ROWS = NT / TPR;  // workers per workgroup
    // this thread's eight i of a row: loaded, and then its elements in their places
    template <typename E>
    static SPEC_DEVICE Raw8<E> start(const typename E::st *row, int i, int d)
    {
        if constexpr (TINY) return load8_tiny<E>(row, at(i), d);
        else return load8_start<E>(row, at(i), d);
    }
    template <typename E>
    static SPEC_DEVICE void end(Raw8<E> &r, int i, int d)
    {
        if constexpr (!TINY) load8_end<E>(r, at(i), d);
    }
    static SPEC_DEVICE int at(int i) { return 8 * (i * TPR + thread()); }
    static SPEC_DEVICE int thread() { return ROWS > 1 ? threadIdx.x % TPR : threadIdx.x; }
    // the same in a wave, and known to be: its rows' addresses are scalars
    static SPEC_DEVICE int64_t worker()
    {
        return ROWS > 1 ? (int64_t)blockIdx.x * ROWS + __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR) : (int64_t)blockIdx.x;
    }
};

// The forward's: two eights per thread from 513 on, more bytes on their way per wave.
template <typename F>
inline hipError_t pick_norm(int64_t d, F &&f)
{
    if (d < 8) return f(RowShape<64, 1, true>{});
    if (d <= 512) return f(RowShape<64, 1>{});
    if (d <= 1024) return f(RowShape<64, 2>{});
    if (d <= 2048) return f(RowShape<256, 1>{});
    if (d <= 4096) return f(RowShape<256, 2>{});
    if (d <= 8192) return f(RowShape<512, 2>{});
    return f(RowShape<1024, 2>{});
}

// The gradients': one eight per thread as far as a workgroup goes: the sums then fit 128
// registers and the row's loads wait behind other waves' work.
template <typename F>
inline hipError_t pick_grad(int64_t d, F &&f)
{
    if (d < 8) return f(RowShape<64, 1, true>{});
    if (d <= 512) return f(RowShape<64, 1>{});
    if (d <= 1024) return f(RowShape<128, 1>{});
    if (d <= 2048) return f(RowShape<256, 1>{});
    if (d <= 4096) return f(RowShape<512, 1>{});
    if (d <= 8192) return f(RowShape<1024, 1>{});
    return f(RowShape<1024, 2>{});
}

// N sums over the threads of a row, the same in all of them.  LDS has two alternating
// places, so that one barrier per call suffices.
template <typename SH, int N>
struct RowSum {
    static constexpr int W = SH::TPR / 64;
    float4 part[2][W > 1 ? W : 1];
    SPEC_DEVICE void operator()(float (&v)[N], int turn)
    {
        static_assert(N <= 4 && W <= 16, "a float4 per wave");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = wave_sum<64>(v[i]);
        if constexpr (W > 1) {
            const int lane = threadIdx.x & 63;
            if (lane == 0) part[turn & 1][threadIdx.x >> 6] = make_float4(v[0], N > 1 ? v[N > 1 ? 1 : 0] : 0.f, N > 2 ? v[N > 2 ? 2 : 0] : 0.f, 0.f);
            __syncthreads();
            const float4 p = part[turn & 1][lane % W];  // every W lanes hold all waves' sums
            const float o[3] = {p.x, p.y, p.z};
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = wave_sum<W>(o[i]);
        }
    }
    // over each 2, 4, 8, 16 or all 64 lanes
    template <int L>
    static SPEC_DEVICE float wave_sum(float x)
    {
        x += dpp<0xB1>(x);
        if (L >= 4) x += dpp<0x4E>(x);
        if (L >= 8) x += dpp<0x141>(x);
        if (L >= 16) x += dpp<0x140>(x);
        if (L >= 64) {
            float y = x;
            rowswap16(x, y);
            x += y;
            y = x;
            halfswap32(x, y);
            x += y;
        }
        return x;
    }
};

// (mean of v^2 + eps)^(-1/2) from the sum of squares.  What leaves f32's range, the sum or
// the mean with eps, is formed again scaled by 2^-160 (all threads of the row agree on it).
template <typename SH, int CH8>
SPEC_DEVICE float inv_rms(const float (&v)[CH8], float inv_d, float eps, RowSum<SH, 1> &sum, int &turn)
{
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < CH8; ++i) s[0] = __builtin_fmaf(v[i], v[i], s[0]);
    sum(s, turn++);
    const float m = s[0] * inv_d + eps;
    if (m < INFINITY) return 1.f / __builtin_sqrtf(m);
    float z[1] = {0.f};
#pragma unroll
    for (int i = 0; i < CH8; ++i) {
        const float a = v[i] * 0x1p-80f;
        z[0] = __builtin_fmaf(a, a, z[0]);
    }
    sum(z, turn++);
    return 0x1p-80f / __builtin_sqrtf(z[0] * inv_d + eps * 0x1p-80f * 0x1p-80f);
}

struct BlockArgs {
    int64_t n, d;
    float alpha, beta, eps, inv_d;
    int post;
    const void *w1, *w2, *gate;
    int64_t ldg, gate_rows;
};

// a matrix of 8-bit checkpoints to write (q == nullptr: none) or to read
struct Stored {
    uint8_t *q, *s;
    int64_t ldq, lds;
};

// The eight values of one eight of a row as a checkpoint; all lanes of the row call it.
template <typename E>
SPEC_DEVICE void put_stored(const Stored &o, int64_t row, int64_t c, int64_t d, const Raw8<E> &r)
{
    const int b = mx_scale<SPEC_MX_INT8>(mx_top<E>(r));
    const int64_t blocks = (d + 31) / 32;
    if (c < blocks * 4) {
        *reinterpret_cast<uint2 *>(o.q + row * o.ldq + c * 8) = mx_encode_int8<E>(r, b);
        if ((c & 3) == 0) o.s[row * o.lds + (c >> 2)] = (uint8_t)b;
    }
}
SPEC_DEVICE void put_stored_end(const Stored &o, int64_t row, int thread, int64_t d)
{
    const int64_t blocks = (d + 31) / 32, scales = (blocks + 15) / 16 * 16;
    if (thread < scales - blocks) o.s[row * o.lds + blocks + thread] = 0;
}

// a weight's or a gate row's eight i, ones where there is none
template <typename E, typename SH>
SPEC_DEVICE Raw8<E> load_or_ones(const void *w, int i, int d)
{
    Raw8<E> r;
    if (w != nullptr) {
        r = SH::template start<E>((const typename E::st *)w, i, d);
        SH::template end<E>(r, i, d);
    } else {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 1.f;
        r.set(v);
    }
    return r;
}

// worker w of `workers` takes rows w, w + workers, ...
// (ALONE: no block, and h' is h itself.)
template <typename E, typename SH, bool ALONE>
__global__ __launch_bounds__(SH::NT) void k_block_norm(BlockArgs a, const typename E::st *Y, int64_t ldy,
                                                       const typename E::st *H, int64_t ldh, typename E::st *O, int64_t ldo,
                                                       typename E::st *X, int64_t ldx, float *__restrict__ r1,
                                                       float *__restrict__ r2, Stored yq, Stored oq, Stored xq,
                                                       int64_t workers)
{
    constexpr int CH = SH::CH;
    __shared__ RowSum<SH, 1> sum;
    const int thread = SH::thread(), d = (int)a.d;
    const int64_t w = SH::worker();
    Raw8<E> w1[CH], w2[CH], gt[CH], ny[CH], nh[CH];
    const auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if constexpr (!ALONE) ny[i] = SH::template start<E>(Y + row * ldy, i, d);
            nh[i] = SH::template start<E>(H + row * ldh, i, d);
        }
    };
    if (w < a.n) fetch(w);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        w2[i] = load_or_ones<E, SH>(a.w2, i, d);
        if constexpr (ALONE) continue;
        w1[i] = load_or_ones<E, SH>(a.w1, i, d);
        gt[i] = load_or_ones<E, SH>(nullptr, i, d);
    }
    int64_t gate_at = -1;
    int turn = 0;
    for (int64_t row = w; row < a.n; row += workers) {
        Raw8<E> y[CH], h[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) y[i] = ny[i], h[i] = nh[i];
        if (row + workers < a.n) fetch(row + workers);
        float v[8 * CH], r = 1.f;
        if constexpr (ALONE) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                SH::template end<E>(h[i], i, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * i + e] = h[i].get(e);
            }
        } else {
            if (a.gate != nullptr && row / a.gate_rows != gate_at) {
                gate_at = row / a.gate_rows;
#pragma unroll
                for (int i = 0; i < CH; ++i) gt[i] = load_or_ones<E, SH>((const typename E::st *)a.gate + gate_at * a.ldg, i, d);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                SH::template end<E>(y[i], i, d);
                SH::template end<E>(h[i], i, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * i + e] = y[i].get(e);
            }
            if (a.post) {
                r = inv_rms<SH, 8 * CH>(v, a.inv_d, a.eps, sum, turn);
                if (r1 != nullptr && thread == 0) r1[row] = r;
            }
            if (yq.q != nullptr) {
#pragma unroll
                for (int i = 0; i < CH; ++i) put_stored<E>(yq, row, i * SH::TPR + thread, a.d, y[i]);
                put_stored_end(yq, row, thread, a.d);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = v[8 * i + e] * r * w1[i].get(e) * gt[i].get(e);
                    v[8 * i + e] = __builtin_fmaf(a.beta, u, a.alpha * h[i].get(e));
                }
        }
        if (!ALONE && (O != nullptr || oq.q != nullptr)) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                Raw8<E> o;
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = v[8 * i + e];
                o.set(t);
                if (O != nullptr && SH::at(i) < d) store8<E>(O + row * ldo, SH::at(i), a.d, o);
                if (oq.q != nullptr) put_stored<E>(oq, row, i * SH::TPR + thread, a.d, o);
            }
            if (oq.q != nullptr) put_stored_end(oq, row, thread, a.d);
        }
        if (X != nullptr || xq.q != nullptr || r2 != nullptr) {
            r = inv_rms<SH, 8 * CH>(v, a.inv_d, a.eps, sum, turn);
            if (r2 != nullptr && thread == 0) r2[row] = r;
            if (X != nullptr || xq.q != nullptr) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    Raw8<E> o;
                    float t[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] = v[8 * i + e] * r * w2[i].get(e);
                    o.set(t);
                    if (X != nullptr && SH::at(i) < d) store8<E>(X + row * ldx, SH::at(i), a.d, o);
                    if (xq.q != nullptr) put_stored<E>(xq, row, i * SH::TPR + thread, a.d, o);
                }
                if (xq.q != nullptr) put_stored_end(xq, row, thread, a.d);
            }
        }
    }
}

// ------------------------------------------------------------------ gradients

// How the rows are dealt to workers, each a run of consecutive rows.
//   few gate rows (or none): `share` workers to a gate row, so that a worker has one of
//     them; it leaves a row of sums s.
//   many (share == 0): a worker has whole gate rows, writes their dg itself and
//     leaves a row of dw1.
// Either way a worker also leaves a row of dw2.
struct GradDeal {
    int64_t run, share, workers, gates;
};
struct GradPart {
    float *dw2, *rest;
    int64_t ld;  // d rounded up to 8
    GradDeal deal;
};

struct GradIo {
    const void *Y, *O, *dO, *dX;
    int64_t ldy, ldo, lddo, lddx;
    Stored yq, oq;
    const float *r1, *r2;
    void *dH, *dY;
    int64_t lddh, lddy;
    float *dgate;
    // all bits, or none where the matrix is not there (its place is taken by another)
    uint32_t keepY, keepX, keepO;
};

// An eight of a row from the matrix itself, or from its checkpoint (codes in w[0] and
// w[1], the scale in w[2]; past the row's codes those of its last eight).
template <typename E, typename SH>
SPEC_DEVICE Raw8<E> fetch8(const void *X, int64_t ld, const Stored &st, int64_t row, int i, int d)
{
    if (st.q == nullptr) return SH::template start<E>((const typename E::st *)X + row * ld, i, d);
    Raw8<E> r;
    const int c = min(SH::at(i) / 8, (d - 1) / 8);
    const uint2 q = *reinterpret_cast<const uint2 *>(st.q + row * st.ldq + c * 8);
    r.w[0] = q.x, r.w[1] = q.y, r.w[2] = st.s[row * st.lds + (c >> 2)], r.w[3] = 0;
    return r;
}

template <typename E>
SPEC_DEVICE void values8(const Raw8<E> &r, const Stored &st, float (&v)[8])
{
    if (st.q != nullptr) {
        mx_decode_int8(r.w[0], r.w[1], mx_unit_int8((int)r.w[2]), v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = r.get(e);
    }
}

// What was computed from r so far is not kept: it is formed again from these registers,
// half as many as its values in f32 would hold.
template <typename E>
SPEC_DEVICE void forget(Raw8<E> &r)
{
#pragma unroll
    for (int k = 0; k < Raw8<E>::N; ++k) asm volatile("" : "+v"(r.w[k]));
}

// one row of the gradients' inputs, zeros where there is none and past d
template <typename E, typename SH>
struct GradRow {
    static constexpr int CH = SH::CH;
    Raw8<E> y[CH], o[CH], dx[CH], dO[CH];
    float r1, r2;
    SPEC_DEVICE void fetch(const BlockArgs &a, const GradIo &io, int64_t row)
    {
        using st = typename E::st;
        const int d = (int)a.d;
        r1 = io.r1 != nullptr ? io.r1[row] : 1.f;
        r2 = io.r2 != nullptr ? io.r2[row] : 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            dx[i] = SH::template start<E>((const st *)io.dX + row * io.lddx, i, d);
            dO[i] = SH::template start<E>((const st *)io.dO + row * io.lddo, i, d);
            o[i] = fetch8<E, SH>(io.O, io.ldo, io.oq, row, i, d);
            y[i] = fetch8<E, SH>(io.Y, io.ldy, io.yq, row, i, d);
        }
    }
    SPEC_DEVICE void settle(const BlockArgs &a, const GradIo &io)
    {
        const int d = (int)a.d;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            SH::template end<E>(dx[i], i, d);
            SH::template end<E>(dO[i], i, d);
            if (io.oq.q == nullptr) SH::template end<E>(o[i], i, d);
            if (io.yq.q == nullptr) SH::template end<E>(y[i], i, d);
            const bool in = SH::at(i) < d;
#pragma unroll
            for (int k = 0; k < Raw8<E>::N; ++k) {
                dx[i].w[k] &= io.keepX;
                dO[i].w[k] &= io.keepO;
                o[i].w[k] = in ? o[i].w[k] & io.keepX : 0;
                y[i].w[k] = in ? y[i].w[k] & io.keepY : 0;
            }
        }
    }
};

template <int CH>
SPEC_DEVICE void put_sums(float *__restrict__ row, const float (&v)[8 * CH], int tpr, int thread, int64_t ld)
{
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int64_t c = 8 * (int64_t)(i * tpr + thread);
        if (c >= ld) continue;
        float4 *o = reinterpret_cast<float4 *>(row + c);
        o[0] = make_float4(v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3]);
        o[1] = make_float4(v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]);
    }
}

// The registers of a workgroup of 512 threads: 128 let two of them share a CU (bf16;
// f32 inputs alone are twice as many).
template <typename E, typename SH>
constexpr int grad_waves() { return sizeof(typename E::st) == 2 && SH::TPR == 512 ? 4 : 1; }

template <typename E, typename SH, bool MANY>
__global__ __launch_bounds__(SH::NT, (grad_waves<E, SH>())) void k_block_grad(BlockArgs a, GradIo io, GradPart part)
{
    using st = typename E::st;
    constexpr int TPR = SH::TPR, CH = SH::CH;
    // Rows of two eights per thread leave no room for the weights and the next row.
    constexpr bool KEEP = CH == 1;
    __shared__ RowSum<SH, 3> sum;
    const int thread = SH::thread();
    const int64_t worker = SH::worker();
    if (worker >= part.deal.workers) return;  // a whole row's threads
    const int64_t run = part.deal.run, share = part.deal.share;
    const int d = (int)a.d;
    const int64_t r0 = MANY ? worker * run : worker / share * a.gate_rows + worker % share * run;
    const int64_t r1 = min(a.n, MANY ? r0 + run : min(r0 + run, (worker / share + 1) * a.gate_rows));
    const auto at = [&](int i) { return SH::at(i); };
    int64_t gate_at = -1;
    const auto gate_row = [&](int i) {
        return load_or_ones<E, SH>(a.gate != nullptr && gate_at >= 0 ? (const st *)a.gate + gate_at * a.ldg : nullptr, i, d);
    };
    Raw8<E> k1[KEEP ? CH : 1], k2[KEEP ? CH : 1], kg[KEEP ? CH : 1];
    float sw2[8 * CH], ss[8 * CH], sw1[8 * CH];
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            k1[i] = load_or_ones<E, SH>(a.w1, i, d);
            k2[i] = load_or_ones<E, SH>(a.w2, i, d);
            kg[i] = gate_row(i);
        }
    }
    // the weights and the gate row's, packed (not kept as values in f32 from row to row)
    const auto w1_of = [&](int i) { if constexpr (KEEP) { forget(k1[i]); return k1[i]; } else return load_or_ones<E, SH>(a.w1, i, d); };
    const auto w2_of = [&](int i) { if constexpr (KEEP) { forget(k2[i]); return k2[i]; } else return load_or_ones<E, SH>(a.w2, i, d); };
    const auto gt_of = [&](int i) { if constexpr (KEEP) { forget(kg[i]); return kg[i]; } else return gate_row(i); };
#pragma unroll
    for (int i = 0; i < 8 * CH; ++i) sw2[i] = ss[i] = sw1[i] = 0.f;
    // the sums of gate row gate_at, which are complete: into dw1, and out
    const auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Raw8<E> w1 = w1_of(i), gt = gt_of(i);
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float &s = ss[8 * i + e];
                sw1[8 * i + e] = __builtin_fmaf(gt.get(e), s, sw1[8 * i + e]);
                t[e] = w1.get(e) * s;
                s = 0.f;
            }
            Raw8<ElF32> o;
            o.set(t);
            if (io.dgate != nullptr && at(i) < a.d) store8<ElF32>(io.dgate + gate_at * a.d, at(i), a.d, o);
        }
    };
    int turn = 0;
    GradRow<E, SH> next;
    if (KEEP && r0 < r1) next.fetch(a, io, r0);
    for (int64_t row = r0; row < r1; ++row) {
        GradRow<E, SH> in;
        if constexpr (KEEP) {
            in = next;
            if (row + 1 < r1) next.fetch(a, io, row + 1);
        } else {
            in.fetch(a, io, row);
        }
        if (a.gate != nullptr && row / a.gate_rows != gate_at) {
            if (MANY && gate_at >= 0) flush();
            gate_at = row / a.gate_rows;
            if constexpr (KEEP) {
#pragma unroll
                for (int i = 0; i < CH; ++i) kg[i] = gate_row(i);
            }
        }
        in.settle(a, io);
        const float rho1 = in.r1, rho2 = in.r2;
        float t[3] = {0.f, 0.f, 0.f};  // sums of a n2, c base, c n2, with base = dh' + r2 a
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Raw8<E> w1 = w1_of(i), w2 = w2_of(i), gt = gt_of(i);
            float vo[8], vy[8];
            values8<E>(in.o[i], io.oq, vo);
            values8<E>(in.y[i], io.yq, vy);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = in.dx[i].get(e), aw = g * w2.get(e);
                const float n1 = vy[e] * rho1, n2 = vo[e] * rho2;
                sw2[8 * i + e] = __builtin_fmaf(g, n2, sw2[8 * i + e]);
                const float c = gt.get(e) * w1.get(e) * n1;
                t[0] = __builtin_fmaf(aw, n2, t[0]);
                t[1] = __builtin_fmaf(c, __builtin_fmaf(rho2, aw, in.dO[i].get(e)), t[1]);
                t[2] = __builtin_fmaf(c, n2, t[2]);
            }
        }
        sum(t, turn++);
        const float m = t[0] * a.inv_d, rm = rho2 * m;
        const float mb = a.post ? a.beta * a.inv_d * (t[1] - rm * t[2]) : 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            forget(in.y[i]), forget(in.o[i]), forget(in.dx[i]), forget(in.dO[i]);
            const Raw8<E> w1 = w1_of(i), w2 = w2_of(i), gt = gt_of(i);
            float vo[8], vy[8], dh[8], dy[8];
            values8<E>(in.o[i], io.oq, vo);
            values8<E>(in.y[i], io.yq, vy);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n1 = vy[e] * rho1, n2 = vo[e] * rho2;
                const float base = __builtin_fmaf(rho2, in.dx[i].get(e) * w2.get(e), in.dO[i].get(e));
                const float G = __builtin_fmaf(-rm, n2, base);
                dh[e] = a.alpha * G;
                const float bG = a.beta * G;
                ss[8 * i + e] = __builtin_fmaf(bG, n1, ss[8 * i + e]);
                dy[e] = rho1 * __builtin_fmaf(-mb, n1, bG * gt.get(e) * w1.get(e));
            }
            const int c = at(i);
            if (c < d) {
                Raw8<E> r;
                if (io.dH != nullptr) {
                    r.set(dh);
                    store8<E>((st *)io.dH + row * io.lddh, c, a.d, r);
                }
                if (io.dY != nullptr) {
                    r.set(dy);
                    store8<E>((st *)io.dY + row * io.lddy, c, a.d, r);
                }
            }
        }
    }
    if (io.keepX) put_sums<CH>(part.dw2 + worker * part.ld, sw2, TPR, thread, part.ld);
    if (io.keepY) {
        if (MANY) flush();
        put_sums<CH>(part.rest + worker * part.ld, MANY ? sw1 : ss, TPR, thread, part.ld);
    }
}

// The workers' rows added: blocks of 32 columns by 32 shares of the workers for dw2,
// for dw1 and, where many workers share a gate row, for each row of dgate; else
// blocks of 1024 columns of a row of dgate.
constexpr int JOIN_SERIAL = 16;  // workers of a gate row that one thread adds

template <typename E>
__global__ __launch_bounds__(1024) void k_block_join(BlockArgs a, GradPart part, float *__restrict__ dw1,
                                                     float *__restrict__ dw2, float *__restrict__ dgate)
{
    using st = typename E::st;
    __shared__ float red[32][33];
    const GradDeal &deal = part.deal;
    const unsigned nc = (unsigned)((a.d + 31) / 32);
    const auto weight = [&](const void *p, int64_t row, int64_t c) {
        return p != nullptr ? E::wide(((const st *)p)[row + c]) : 1.f;
    };
    if (blockIdx.x >= 2 * nc && deal.share <= JOIN_SERIAL) {
        const unsigned nb = (unsigned)((a.d + 1023) / 1024), u = blockIdx.x - 2 * nc;
        const int64_t c = (int64_t)(u % nb) * 1024 + threadIdx.x, k = u / nb;
        if (c >= a.d) return;
        float s = 0.f;
        for (int64_t i = 0; i < deal.share; ++i) s += part.rest[(k * deal.share + i) * part.ld + c];
        dgate[k * a.d + c] = s * weight(a.w1, 0, c);
        return;
    }
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int what = (int)(blockIdx.x / nc);  // 0: dw2, 1: dw1, 2 + k: row k of dgate
    const int64_t c = (int64_t)(blockIdx.x % nc) * 32 + tx;
    const float *src = what == 0 ? part.dw2 : part.rest;
    float *dst = what == 0 ? dw2 : what == 1 ? dw1 : dgate + (what - 2) * a.d;
    if ((what == 0 ? dw2 : what == 1 ? dw1 : dgate) == nullptr) return;
    const int64_t w0 = what < 2 ? 0 : (what - 2) * deal.share, w1 = what < 2 ? deal.workers : w0 + deal.share;
    const bool gated = what == 1 && deal.share > 0 && a.gate != nullptr;  // sums s, not yet times their gate row
    float s = 0.f;
    if (c < a.d) {
#pragma unroll 16
        for (int64_t w = w0 + ty; w < w1; w += 32) {
            const float v = src[w * part.ld + c];
            s += gated ? v * weight(a.gate, w / deal.share * a.ldg, c) : v;
        }
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty != 0 || c >= a.d) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][tx];
    dst[c] = what < 2 ? s : s * weight(a.w1, 0, c);
}

__global__ __launch_bounds__(256) void k_block_zero(float *__restrict__ a, float *__restrict__ b, int64_t d)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= d) return;
    if (a != nullptr) a[c] = 0.f;
    if (b != nullptr) b[c] = 0.f;
}

BlockArgs block_args(const spec_block *b)
{
    BlockArgs a{};
    a.n = b->n, a.d = b->d;
    a.alpha = (float)b->alpha, a.beta = (float)b->beta, a.eps = (float)b->eps;
    a.inv_d = (float)(1.0 / (double)b->d);
    a.post = b->post;
    a.w1 = b->w_post, a.w2 = b->w_pre, a.gate = b->gate;
    a.ldg = b->ldg, a.gate_rows = b->gate != nullptr ? b->gate_rows : std::max<int64_t>(b->n, 1);
    return a;
}

Stored stored(const spec_mx *m)
{
    return m == nullptr || m->q == nullptr ? Stored{} : Stored{(uint8_t *)m->q, (uint8_t *)m->s, m->ldq, m->lds};
}

// 512 workgroups of a run each where the rows suffice, two to a CU: every one leaves two
// rows of f32 sums (1024 took 194 us where 512 took 186).
GradDeal grad_deal(int64_t n, int64_t d, int64_t gate_rows, bool gate)
{
    const int64_t per = d <= 512 ? 4 : 1;  // workers to a workgroup (RowShape::ROWS)
    const int64_t run = std::max<int64_t>(1, cdiv_h(n, 512 * per));
    const int64_t rows = gate ? std::min(gate_rows, n) : n;
    GradDeal p{};
    p.gates = cdiv_h(n, rows);
    if (p.gates >= 256 || (p.gates > 1 && rows <= run)) {
        p.run = rows * std::max<int64_t>(1, run / rows);
        p.workers = cdiv_h(n, p.run);
    } else {
        p.share = cdiv_h(rows, run);
        p.run = cdiv_h(rows, p.share);
        p.workers = p.gates * p.share;
    }
    return p;
}

int64_t sums_bytes(const GradDeal &p, int64_t d) { return up_h(p.workers * up_h(d, 8) * 4, 256); }

template <typename E>
hipError_t block_norm(hipStream_t stream, const spec_block *b, const void *Y, int64_t ldy, const void *H, int64_t ldh,
                      void *O, int64_t ldo, void *X, int64_t ldx, float *r1, float *r2, const spec_mx *yq,
                      const spec_mx *oq, const spec_mx *xq)
{
    using st = typename E::st;
    const BlockArgs a = block_args(b);
    return pick_norm(b->d, [&](auto shape) {
        using SH = decltype(shape);
        // 16384 x 4096 bf16 with 3, 4, 6 and 8 workgroups of 256 threads per CU: 114, 125, 112
        // and 115 us; 8192 x 4097 f32 137, 114, 117 and 120
        const int64_t grid = std::min<int64_t>(cdiv_h(b->n, SH::ROWS), 256 * 6 * 256 / SH::NT);
        const auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(SH::NT), 0, stream, a, (const st *)Y, ldy, (const st *)H,
                               ldh, (st *)O, ldo, (st *)X, ldx, r1, r2, stored(yq), stored(oq), stored(xq),
                               grid * SH::ROWS);
        };
        if (Y == nullptr)
            go(k_block_norm<E, SH, true>);
        else
            go(k_block_norm<E, SH, false>);
        return hipGetLastError();
    });
}

template <typename E>
hipError_t block_grad(hipStream_t stream, const spec_block *b, GradIo io, float *dw1, float *dw2, char *ws)
{
    BlockArgs a = block_args(b);
    const bool hasY = io.Y != nullptr || io.yq.q != nullptr, hasX = io.dX != nullptr;
    io.keepY = hasY ? ~0u : 0;
    io.keepX = hasX ? ~0u : 0;
    io.keepO = io.dO != nullptr ? ~0u : 0;
    const void *any = hasX ? io.dX : io.dO;  // one of the two is there
    const int64_t ldany = hasX ? io.lddx : io.lddo;
    // (w2 out of the way too: zero times one of its infinities would be NaN)
    if (!hasX) io.dX = io.O = any, io.lddx = io.ldo = ldany, io.oq = Stored{}, io.r2 = nullptr, a.w2 = nullptr;
    if (!io.keepO) io.dO = any, io.lddo = ldany;
    if (!hasY) io.Y = any, io.ldy = ldany, a.post = 0, a.alpha = 1.f;  // (the norm of H itself)
    if (!a.post) io.r1 = nullptr;
    const GradDeal p = grad_deal(a.n, a.d, a.gate_rows, a.gate != nullptr);
    const GradPart part{(float *)ws, (float *)(ws + sums_bytes(p, a.d)), up_h(a.d, 8), p};
    const hipError_t e = pick_grad(b->d, [&](auto shape) {
        using SH = decltype(shape);
        const dim3 grid((unsigned)cdiv_h(p.workers, SH::ROWS)), block(SH::NT);
        if (p.share == 0)
            hipLaunchKernelGGL((k_block_grad<E, SH, true>), grid, block, 0, stream, a, io, part);
        else
            hipLaunchKernelGGL((k_block_grad<E, SH, false>), grid, block, 0, stream, a, io, part);
        return hipGetLastError();
    });
    if (e != hipSuccess || !(hasX || hasY)) return e;
    const int64_t nc = cdiv_h(a.d, 32);
    const int64_t rows = !hasY || io.dgate == nullptr || p.share == 0 ? 0 : p.gates;
    hipLaunchKernelGGL(k_block_join<E>, dim3((unsigned)(2 * nc + rows * (p.share <= JOIN_SERIAL ? cdiv_h(a.d, 1024) : nc))),
                       dim3(1024), 0, stream, a, part, hasY ? dw1 : nullptr, hasX ? dw2 : nullptr,
                       rows > 0 ? io.dgate : nullptr);
    return hipGetLastError();
}

}  // namespace

size_t block_norm_grad_workspace_bytes(const spec_block *b)
{
    if (b->n == 0) return 256;
    return (size_t)(2 * sums_bytes(grad_deal(b->n, b->d, b->gate_rows, b->gate != nullptr), b->d));
}

hipError_t launch_block_norm(hipStream_t stream, const spec_block *b, const void *Y, int64_t ldy, const void *H,
                             int64_t ldh, void *O, int64_t ldo, void *X, int64_t ldx, float *r1, float *r2,
                             const spec_mx *yq, const spec_mx *oq, const spec_mx *xq)
{
    if (b->n == 0) return hipSuccess;
    return b->t == SPEC_BF16 ? block_norm<ElBF16>(stream, b, Y, ldy, H, ldh, O, ldo, X, ldx, r1, r2, yq, oq, xq)
                             : block_norm<ElF32>(stream, b, Y, ldy, H, ldh, O, ldo, X, ldx, r1, r2, yq, oq, xq);
}

hipError_t launch_block_norm_grad(hipStream_t stream, const spec_block *b, const void *Y, int64_t ldy, const spec_mx *yq,
                                  const void *O, int64_t ldo, const spec_mx *oq, const float *r1, const float *r2,
                                  const void *dO, int64_t lddo, const void *dX, int64_t lddx, void *dH, int64_t lddh,
                                  void *dY, int64_t lddy, float *dw1, float *dw2, float *dgate, void *ws)
{
    if (b->n == 0) {
        hipLaunchKernelGGL(k_block_zero, dim3((unsigned)cdiv_h(b->d, 256)), dim3(256), 0, stream, dw1, dw2, b->d);
        return hipGetLastError();
    }
    GradIo io{};
    io.Y = Y, io.O = O, io.dO = dO, io.dX = dX;
    io.ldy = ldy, io.ldo = ldo, io.lddo = lddo, io.lddx = lddx;
    io.yq = stored(yq), io.oq = stored(oq);
    io.r1 = r1, io.r2 = r2;
    io.dH = dH, io.dY = dY, io.lddh = lddh, io.lddy = lddy;
    io.dgate = dgate;
    return b->t == SPEC_BF16 ? block_grad<ElBF16>(stream, b, io, dw1, dw2, (char *)ws)
                             : block_grad<ElF32>(stream, b, io, dw1, dw2, (char *)ws);
}
