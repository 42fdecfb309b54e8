// Tiled matrix products on MFMA shared by the vocabulary cross entropy and the
// Newton-Schulz kernels (gfx950): bf16, f16 and f32 operands, f32 accumulation.
//
//   acc[p][q] = sum_k P(p, k) Q(q, k)
//
// P runs along the contiguous dimension of the result and is the MFMA's row
// (register) operand; Q runs along the result's rows and is its column (lane)
// operand, so a lane holds four consecutive elements of one result row and
// stores them together.  Either operand may lie in memory with k contiguous
// ("Kc": row p, then k) or with k slow ("Ks": row k, then p).
//
// Staging.  A K-step is 128 bytes of every operand row (64 values of 16 bits,
// 32 of f32).  Both layouts are copied to LDS in 16-byte chunks by LDS DMA
// (no registers, no address arithmetic in the loop beyond the base); the
// hardware writes a wave's 64 chunks to consecutive LDS addresses, so bank
// conflicts are avoided by choosing which chunk a lane fetches:
//   Kc  LDS row p = 8 chunks, chunk c in slot c ^ ((p >> 1) & 7): a fragment read
//       takes one chunk of 16 rows per cycle, which are the 16 slots of two rows
//       (the 64 banks) once each; with p & 7 every second LDS cycle was a conflict.
//   Ks  LDS row k = BP / (16 bytes) chunks, chunk c in slot c ^ f(k).  16-bit
//       fragments are read with the transposing LDS load (per 16 lanes: four
//       k-rows of 16 elements, each lane receives its column's four k), whose
//       rows k & 3 go to different 64-byte groups by f = 4 (k & 3); f32
//       fragments read 32 consecutive columns of rows k and k + 4, separated by
//       f = 8 ((k >> 2) & 1).
// The LDS conflict counter reads zero for all forms.  Rows past the end read as
// zero: a lane whose chunk lies outside gets an offset beyond the buffer resource.
#pragma once

#include <type_traits>

#include "common.h"

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef __attribute__((address_space(3))) void lds_void_t;

// Element types: storage, exact widening, rounding to nearest even.
struct ElBF16 {
    using st = uint16_t;
    static SPEC_DEVICE float wide(st x) { return bf16_to_f32(x); }
    static SPEC_DEVICE st round(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
};
struct ElF16 {
    using st = uint16_t;
    static SPEC_DEVICE float wide(st x) { return (float)__builtin_bit_cast(_Float16, x); }
    static SPEC_DEVICE st round(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};
struct ElF32 {
    using st = float;
    static SPEC_DEVICE float wide(st x) { return x; }
    static SPEC_DEVICE st round(float x) { return x; }
};

SPEC_DEVICE int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// four consecutive elements
template <typename E>
struct Vec4 {
    typename E::st v[4];
} __attribute__((aligned(4 * sizeof(typename E::st))));

// One operand of one tile.
struct MmSrc {
    const char *base;  // Kc: row p0, k = 0; Ks: row k = 0, column p0
    int64_t ldb;       // bytes between rows (a multiple of 16; 256 rows stay below 2^31 bytes)
    int lim;           // rows (Kc) or columns (Ks) of the tile inside the matrix, >= 0
    int64_t K;         // end of k: past it the operand is zero (Kc: a multiple of 16 bytes)
};

// f(0), ..., f(N - 1) with the index as a constant
template <int I, int N, typename F>
SPEC_DEVICE void mm_for(F &&f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        mm_for<I + 1, N>(f);
    }
}

template <typename E, int BP, int BQ, int WP, int WQ, bool PS, bool QS>
struct Mm {
    static constexpr int SZ = (int)sizeof(typename E::st);
    static constexpr int EPC = 16 / SZ;    // elements per chunk
    static constexpr int ROW = 128;        // bytes of an operand row per step
    static constexpr int BK = ROW / SZ;    // k per step
    static constexpr int RC = ROW / 16;    // chunks of a row
    static constexpr int KQ = ROW / 32;    // fragments (32 bytes of k) per step
    static constexpr int STAGES = 2;
    static constexpr int NT = 64 * WP * WQ;
    static constexpr int MI = BP / WP / 32, NI = BQ / WQ / 32;
    static constexpr int P_BYTES = BP * ROW, Q_BYTES = BQ * ROW;
    static constexpr int PL = BP * RC / NT, QL = BQ * RC / NT;  // chunks per thread and step
    static_assert(PL >= 1 && QL >= 1 && BP % (32 * WP) == 0 && BQ % (32 * WQ) == 0, "tile");

    static constexpr uint32_t OUT = 0xFFFFFFF0u;

    f32x16_t acc[MI][NI];

    // slot permutation of row p of a Kc tile
    static SPEC_DEVICE int kc_f(int p) { return ROW == 128 ? (p >> 1) & 7 : (p >> 2) & 3; }

    // slot permutation of row k of a Ks tile with R columns
    template <int R>
    static SPEC_DEVICE int ks_f(int k)
    {
        constexpr int CH = R / EPC;
        return (SZ == 2 ? 4 * (k & 3) : 8 * ((k >> 2) & 1)) & (CH - 1);
    }

    // byte offsets of this thread's chunks of a K-step from the step's base; kc:
    // the first k of its chunks (Kc: the same for all of them, the slots repeat every 16 rows)
    template <int R, bool S, int N>
    static SPEC_DEVICE void offsets(const MmSrc &s, uint32_t (&v)[N], int &kc)
    {
        const int tid = threadIdx.x;
        kc = S ? 0 : (((tid % RC) ^ kc_f(tid / RC)) * EPC);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = i * NT + tid;
            if (S) {
                constexpr int CH = R / EPC;
                const int k = q / CH, c = (q % CH) ^ ks_f<R>(k);
                v[i] = c * EPC < s.lim ? (uint32_t)(k * (int)s.ldb + c * 16) : OUT;
            } else {
                const int row = q / RC;
                v[i] = row < s.lim ? (uint32_t)(row * (int)s.ldb + kc * SZ) : OUT;
            }
        }
    }

    // starts the copy of K-step [k0, k0 + BK) of one operand; what lies past its K arrives as zero
    template <bool S, int N>
    static SPEC_DEVICE void stage(const MmSrc &s, const uint32_t (&v)[N], int kc, int64_t k0, char *lds)
    {
        char *dst = lds + ((int)threadIdx.x & ~63) * 16;  // the wave's first chunk
        const int64_t left = s.K - k0;
        int num;
        uint32_t past = 0;
        if (S) {
            const int64_t rem = (left - 1) * s.ldb + (s.lim + EPC - 1) / EPC * 16;
            num = left > 0 && s.lim > 0 ? (int)(rem < 0x7FFFFFF0 ? rem : 0x7FFFFFF0) : 0;
        } else {
            num = 0x7FFFFFF0;
            past = kc < left ? 0u : 0x80000000u;
        }
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void *)(s.base + (left > 0 ? k0 : 0) * (S ? s.ldb : (int64_t)SZ)), 0, num, 0x00020000);
#pragma unroll
        for (int i = 0; i < N; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)(dst + i * NT * 16), 16, (int)(v[i] | past), 0, 0,
                                                     0);
    }

    // the 32-row fragment at rows r0 .. r0 + 31 of the kk-th half of the K-step
    struct Frag {
        f32x4_t x;
    };
    template <int R, bool S>
    static SPEC_DEVICE Frag frag(const char *lds, int r0, int kk, int lane)
    {
        Frag f;
        const int h = lane >> 5;
        if (!S) {
            f.x = *reinterpret_cast<const f32x4_t *>(lds + (r0 + (lane & 31)) * ROW + (((2 * kk + h) ^ kc_f(lane & 31)) << 4));
        } else if (SZ == 2) {
            const int kq = (lane >> 2) & 3;
            const int chunk = (r0 >> 3) + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
            const char *a = lds + (16 * kk + 8 * h + kq) * (R * 2) + ((chunk ^ ks_f<R>(kq)) << 4) + (lane & 1) * 8;
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)a);
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)(a + 4 * R * 2));
            const s16x8_t b = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            f.x = __builtin_bit_cast(f32x4_t, b);
        } else {
            const int k = 8 * kk + 4 * h;
            const int chunk = (r0 >> 2) + ((lane & 31) >> 2);
            const char *a = lds + k * (R * 4) + ((chunk ^ ks_f<R>(k)) << 4) + (lane & 3) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) f.x[j] = *reinterpret_cast<const float *>(a + j * R * 4);
        }
        return f;
    }

    static SPEC_DEVICE f32x16_t mfma(const Frag &a, const Frag &b, f32x16_t c)
    {
        if constexpr (std::is_same<E, ElBF16>::value) {
            return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a.x),
                                                           __builtin_bit_cast(bf16x8_t, b.x), c, 0, 0, 0);
        } else if constexpr (std::is_same<E, ElF16>::value) {
            return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a.x),
                                                          __builtin_bit_cast(f16x8_t, b.x), c, 0, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.x[j], b.x[j], c, 0, 0, 0);
            return c;
        }
    }

    struct Frags {
        Frag a[MI], b[NI];
    };
    static SPEC_DEVICE void fetch(Frags &f, const char *sp, const char *sq, int p0, int q0, int kk, int lane)
    {
#pragma unroll
        for (int m = 0; m < MI; ++m) f.a[m] = frag<BP, PS>(sp, p0 + 32 * m, kk, lane);
#pragma unroll
        for (int n = 0; n < NI; ++n) f.b[n] = frag<BQ, QS>(sq, q0 + 32 * n, kk, lane);
    }
    // the reads before this point stay before the products after it
    SPEC_DEVICE void multiply(const Frags &f)
    {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int n = 0; n < NI; ++n) acc[m][n] = mfma(f.a[m], f.b[n], acc[m][n]);
        __builtin_amdgcn_sched_barrier(0);
    }

    // all but the latest `left` LDS copies of this wave have landed, and so have every wave's
    template <int LEFT>
    static SPEC_DEVICE void landed()
    {
        static_assert(LEFT < 16, "vmcnt");
        __builtin_amdgcn_s_waitcnt(0x0F70 | LEFT);
        __syncthreads();
    }

    // The stages of both operands: separate LDS objects, so that a read of one
    // stage need not wait for the copy into another.
    struct Lds {
        char *p[STAGES], *q[STAGES];
    };

    // acc = sum over k in [kb, K)
    SPEC_DEVICE void run(const MmSrc &P, const MmSrc &Q, int64_t kb, int64_t K, const Lds &s)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int p0 = (wave % WP) * (BP / WP), q0 = (wave / WP) * (BQ / WQ);
        uint32_t vp[PL], vq[QL];
        int kp, kq;
        offsets<BP, PS>(P, vp, kp);
        offsets<BQ, QS>(Q, vq, kq);
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[m][n][e] = 0.f;
        if (kb >= K) return;
        // The fragments of the next half step are read while a half is multiplied.
        // Before the second half's products its fragments are in registers, so
        // the stage is free: there the barrier stands, the stage's next step is
        // requested, and the next stage's first fragments are read behind the
        // products.  Steps past K are requested too (they arrive as zeros), so
        // that the number of copies in flight is always the same.
        constexpr int S = STAGES;
        Frags f0, f1;
        auto request = [&](int64_t k, int i) {
            stage<PS>(P, vp, kp, k, s.p[i]);
            stage<QS>(Q, vq, kq, k, s.q[i]);
        };
        mm_for<0, S>([&](auto I) { request(kb + decltype(I)::value * BK, decltype(I)::value); });
        landed<(S - 1) * (PL + QL)>();
        fetch(f0, s.p[0], s.q[0], p0, q0, 0, lane);
        // S steps per turn, with no way out between them (a copy of every
        // accumulator would be kept for it)
        for (int64_t k0 = kb; k0 < K; k0 += S * BK) {
            mm_for<0, S>([&](auto I) {
                constexpr int i = decltype(I)::value, j = (i + 1) % S;
                mm_for<1, KQ>([&](auto Q_) {
                    constexpr int kk = decltype(Q_)::value;
                    fetch(kk & 1 ? f1 : f0, s.p[i], s.q[i], p0, q0, kk, lane);
                    multiply(kk & 1 ? f0 : f1);
                });
                landed<(S - 2) * (PL + QL)>();
                request(k0 + (i + S) * BK, i);
                fetch(f0, s.p[j], s.q[j], p0, q0, 0, lane);
                multiply(f1);
            });
        }
        landed<0>();  // nothing is left to arrive in LDS that others may use
    }

    // f(p, q, v): four results p .. p + 3 of row q (offsets within the tile)
    template <typename F>
    SPEC_DEVICE void each4(F &&f)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int p0 = (wave % WP) * (BP / WP) + 4 * (lane >> 5), q0 = (wave / WP) * (BQ / WQ) + (lane & 31);
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int m = 0; m < MI; ++m)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[m][n][4 * g + e];
                    f(p0 + 32 * m + 8 * g, q0 + 32 * n, v);
                }
    }
};

// The tile a workgroup takes of an np x nq grid: the hardware deals workgroups
// round-robin over the 8 XCDs, so the ids of one XCD are made consecutive, and
// consecutive ids walk bands of eight q-tiles, p inside the band: the tiles an
// XCD runs together share 8 Q strips and a few P strips in its L2.
SPEC_DEVICE void mm_tile(int64_t id, int np, int nq, int &tp, int &tq)
{
    id = xcd_remap(id, (int64_t)np * nq);
    constexpr int G = 8;
    const int band = (int)(id / ((int64_t)G * np));
    const int w = min(G, nq - band * G);
    const int rest = (int)(id - (int64_t)band * G * np);
    tq = band * G + rest % w;
    tp = rest / w;
}

// Tile shapes: 256 x 256 by eight waves (128 x 64 each, one workgroup per CU:
// 128 KB of LDS) and 128 x 128 by four (64 x 64 each, two workgroups per CU).
struct Tile256 {
    static constexpr int BP = 256, BQ = 256, WP = 2, WQ = 4;
};
struct Tile128 {
    static constexpr int BP = 128, BQ = 128, WP = 2, WQ = 2;
};

template <typename E, typename C, bool PS, bool QS>
using MmOf = Mm<E, C::BP, C::BQ, C::WP, C::WQ, PS, QS>;

// declares the LDS stages of both operands as `lds`
#define MM_STAGES(M)                                                                                           \
    __shared__ __attribute__((aligned(16))) char sp0[M::P_BYTES], sp1[M::P_BYTES], sq0[M::Q_BYTES], sq1[M::Q_BYTES]; \
    const typename M::Lds lds{{sp0, sp1}, {sq0, sq1}}

// two waves per SIMD: one workgroup of Tile256, two of Tile128 per CU
#define MM_BOUNDS(C) __launch_bounds__(64 * C::WP * C::WQ, 2)
