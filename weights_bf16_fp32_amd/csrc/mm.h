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
//       rows k & 3 go to different 64-byte groups by f = 4 (k & 3) (narrower
//       tiles' rows lie in different groups by themselves); f32 fragments read 32
//       consecutive columns of rows k and k + 4, separated by f = 8 ((k >> 2) & 1).
// The LDS conflict counter reads zero for the 16-bit forms.  Rows past the end read as
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

template <typename E, typename C, bool PS, bool QS>
struct Mm {
    static constexpr int BP = C::BP, BQ = C::BQ, WP = C::WP, WQ = C::WQ, WK = C::WK;
    static constexpr int SZ = (int)sizeof(typename E::st);
    static constexpr int EPC = 16 / SZ;    // elements per chunk
    static constexpr int ROW = 128;        // bytes of an operand row per step
    static constexpr int BK = ROW / SZ;    // k per step
    static constexpr int RC = ROW / 16;    // chunks of a row
    static constexpr int KW = ROW / 32 / WK;  // fragments (32 bytes of k) per step and wave
    static constexpr int STAGES = C::STAGES;
    static constexpr int NT = C::NT;
    static constexpr int MI = BP / WP / 32, NI = BQ / WQ / 32;
    static constexpr int P_BYTES = BP * ROW, Q_BYTES = BQ * ROW;
    static constexpr int PL = BP * RC / NT, QL = BQ * RC / NT;  // chunks per thread and step
    static_assert(PL >= 1 && QL >= 1 && BP % (32 * WP) == 0 && BQ % (32 * WQ) == 0, "tile");
    static_assert(NT == 64 * WP * WQ * WK, "threads");

    static constexpr uint32_t OUT = 0xFFFFFFF0u;

    f32x16_t acc[MI][NI];

    // a wave's first row of P and of Q in the tile
    static SPEC_DEVICE int wave_p0(int wave) { return wave % WP * (BP / WP); }
    static SPEC_DEVICE int wave_q0(int wave) { return wave / WP % WQ * (BQ / WQ); }

    // slot permutation of row p of a Kc tile
    static SPEC_DEVICE int kc_f(int p) { return (p >> 1) & 7; }

    // slot permutation of row k of a Ks tile with R columns
    template <int R>
    static SPEC_DEVICE int ks_f(int k)
    {
        constexpr int CH = R / EPC;
        if (SZ == 2) return CH == 16 || CH == 32 ? 4 * (k & 3) : CH >= 8 ? 4 * ((k >> 1) & 1) : 0;
        return CH >= 16 ? 8 * ((k >> 2) & 1) : 0;
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
            return c;  // multiply() orders the four products of a fragment itself
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
        if constexpr (SZ == 4) {
            // a lane's four k in turn, all accumulators in between
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int m = 0; m < MI; ++m)
#pragma unroll
                    for (int n = 0; n < NI; ++n)
                        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x2f32(f.a[m].x[j], f.b[n].x[j], acc[m][n], 0, 0, 0);
        } else {
#pragma unroll
            for (int m = 0; m < MI; ++m)
#pragma unroll
                for (int n = 0; n < NI; ++n) acc[m][n] = mfma(f.a[m], f.b[n], acc[m][n]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    // all but the latest `left` LDS copies of this wave have landed, and so have every wave's
    template <int LEFT>
    static SPEC_DEVICE void landed()
    {
        static_assert(LEFT < 64, "vmcnt");
        __builtin_amdgcn_s_waitcnt(0x0F70 | (LEFT & 15) | (LEFT >> 4) << 14);
        __syncthreads();
    }

    // The stages of both operands: separate LDS objects, so that a read of one
    // stage need not wait for the copy into another (the first STAGES are used).
    struct Lds {
        char *p[8], *q[8];
        float4 *red;  // WK > 1: the waves' sums of one accumulator, 16 KB
    };

    // WK > 1: every wave holds the sums over its share of k of the whole tile.
    // One accumulator at a time they are added, in order of the waves; wave w
    // keeps rows 8 w .. 8 w + 7 of it (each lane four of them, in elements 0..3).
    SPEC_DEVICE void join(const Lds &s)
    {
        static_assert(WK == 1 || (WK == 4 && WP == 1 && WQ == 1), "shares of k");
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int n = 0; n < NI; ++n) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    s.red[(wave * 4 + g) * 64 + lane] = make_float4(acc[m][n][4 * g], acc[m][n][4 * g + 1],
                                                                    acc[m][n][4 * g + 2], acc[m][n][4 * g + 3]);
                __syncthreads();
                float4 r = s.red[wave * 64 + lane];
#pragma unroll
                for (int w = 1; w < WK; ++w) {
                    const float4 o = s.red[(w * 4 + wave) * 64 + lane];
                    r.x += o.x, r.y += o.y, r.z += o.z, r.w += o.w;
                }
                acc[m][n][0] = r.x, acc[m][n][1] = r.y, acc[m][n][2] = r.z, acc[m][n][3] = r.w;
                __syncthreads();
            }
    }

    // acc = sum over k in [kb, K)
    SPEC_DEVICE void run(const MmSrc &P, const MmSrc &Q, int64_t kb, int64_t K, const Lds &s)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int p0 = wave_p0(wave), q0 = wave_q0(wave), kw = wave / (WP * WQ) * KW;
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
        if (kb < K) {
            // The next fragments are read while the present ones are multiplied.
            // Before the last products of a step its fragments are in registers, so
            // the stage is free: there the barrier stands, the stage's next step is
            // requested, and the next stage's first fragments are read behind the
            // products.  Steps past K are requested too (they arrive as zeros), so
            // that the number of copies in flight is always the same.
            constexpr int S = STAGES;
            static_assert(S * KW % 2 == 0 && S <= 8, "stages");
            Frags f[2];
            auto request = [&](int64_t k, int i) {
                stage<PS>(P, vp, kp, k, s.p[i]);
                stage<QS>(Q, vq, kq, k, s.q[i]);
            };
            mm_for<0, S>([&](auto I) { request(kb + decltype(I)::value * BK, decltype(I)::value); });
            landed<(S - 1) * (PL + QL)>();
            fetch(f[0], s.p[0], s.q[0], p0, q0, kw, lane);
            for (int64_t k0 = kb; k0 < K; k0 += S * BK) {
                mm_for<0, S>([&](auto I) {
                    constexpr int i = decltype(I)::value, j = (i + 1) % S;
                    // large tiles run the steps past K of a turn (on zeros): a way out
                    // between steps would keep a copy of every accumulator
                    if (MI * NI <= 4 && i > 0 && k0 + i * BK >= K) return;
                    mm_for<0, KW>([&](auto Q_) {
                        constexpr int kk = decltype(Q_)::value, cur = (i * KW + kk) & 1;
                        if constexpr (kk < KW - 1) {
                            fetch(f[cur ^ 1], s.p[i], s.q[i], p0, q0, kw + kk + 1, lane);
                        } else {
                            landed<(S - 2) * (PL + QL)>();
                            request(k0 + (i + S) * BK, i);
                            fetch(f[cur ^ 1], s.p[j], s.q[j], p0, q0, kw, lane);
                        }
                        multiply(f[cur]);
                    });
                });
            }
            landed<0>();  // nothing is left to arrive in LDS
        }
        if constexpr (WK > 1) join(s);
    }

    // A wave's part of the stages: room for 32 of its rows in f32.
    static SPEC_DEVICE float4 *own_part(const Lds &s)
    {
        constexpr int PC = BP / WP / 4;  // groups of four in a wave's row
        static_assert(32 * PC * 16 * 2 <= P_BYTES && NT / 128 <= 2 * STAGES, "two waves share a stage's operand");
        const int wave = threadIdx.x >> 6, part = wave >> 1;
        char *mine = s.p[0];  // (selected, not indexed: LDS objects have no table of addresses)
        mm_for<1, NT / 128>([&](auto I) {
            constexpr int i = decltype(I)::value;
            if (part == i) mine = i < STAGES ? s.p[i] : s.q[i < STAGES ? 0 : i - STAGES];
        });
        return reinterpret_cast<float4 *>(mine) + (wave & 1) * 32 * PC;
    }

    // put(p, q, v, get(p, q)): four results p .. p + 3 of row q (offsets within the
    // tile), with what get() read for them.  A lane's results lie in one row and
    // the lanes' rows differ, so memory would be met 16 bytes at a time; large
    // tiles pass them through LDS (each wave its own part of the stages) and meet
    // it in runs of a wave's whole width.  The reads of eight groups are issued
    // together, before the first of their stores.
    template <typename G, typename F>
    SPEC_DEVICE void each4(const Lds &s, G &&get, F &&put)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        if constexpr (WK > 1) {
            const int p0 = 8 * wave + 4 * (lane >> 5), q0 = lane & 31;
            decltype(get(0, 0)) old[MI][NI];
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int m = 0; m < MI; ++m) old[m][n] = get(p0 + 32 * m, q0 + 32 * n);
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int m = 0; m < MI; ++m) {
                    float v[4] = {acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]};
                    put(p0 + 32 * m, q0 + 32 * n, v, old[m][n]);
                }
        } else {
            constexpr int PC = BP / WP / 4;  // groups of four in a wave's row
            constexpr int AT = PC / 2 % 8 == 0 ? 8 : PC / 2 % 6 == 0 ? 6 : 4;
            static_assert(PC / 2 % AT == 0, "groups at a time");
            float4 *buf = own_part(s);
            const auto slot = [](int q, int c) { return q * PC + (c ^ (PC == 24 ? (q >> 1) & 7 : PC == 8 ? q & 7 : q & 15)); };
            const int p0 = wave_p0(wave), q0 = wave_q0(wave);
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                wave_sync();
#pragma unroll
                for (int m = 0; m < MI; ++m)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        buf[slot(lane & 31, 8 * m + 2 * g + (lane >> 5))] =
                            make_float4(acc[m][n][4 * g], acc[m][n][4 * g + 1], acc[m][n][4 * g + 2], acc[m][n][4 * g + 3]);
                wave_sync();
#pragma unroll
                for (int i0 = 0; i0 < PC / 2; i0 += AT) {
                    decltype(get(0, 0)) old[AT];
#pragma unroll
                    for (int i = 0; i < AT; ++i) {
                        const int u = 64 * (i0 + i) + lane;
                        old[i] = get(p0 + 4 * (u % PC), q0 + 32 * n + u / PC);
                    }
#pragma unroll
                    for (int i = 0; i < AT; ++i) {
                        const int u = 64 * (i0 + i) + lane, q = u / PC, c = u % PC;
                        const float4 r = buf[slot(q, c)];
                        float v[4] = {r.x, r.y, r.z, r.w};
                        put(p0 + 4 * c, q0 + 32 * n + q, v, old[i]);
                    }
                }
            }
        }
    }
    struct Nothing {
    };
    template <typename F>
    SPEC_DEVICE void each4(const Lds &s, F &&put)
    {
        each4(s, [](int, int) { return Nothing{}; }, [&](int p, int q, float (&v)[4], const Nothing &) { put(p, q, v); });
    }

    // put(p, q, v, get(p, q)): the results of rows q .. q + 3 at p: the tile of the
    // transposed product, in runs of 32 rows
    template <typename G, typename F>
    SPEC_DEVICE void each4_across(const Lds &s, G &&get, F &&put)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int p0 = wave_p0(wave), q0 = wave_q0(wave);
        if constexpr (WK > 1) {
            // rows 8 wave + 4 h .. + 3 of each 32 x 32 block are in this lane's column
            float *buf = reinterpret_cast<float *>(s.red) + wave * 8 * 32;
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int m = 0; m < MI; ++m) {
                    const int p = 32 * m + 8 * wave + (lane >> 3), q = 32 * n + 4 * (lane & 7);
                    const auto old = get(p, q);
                    wave_sync();
#pragma unroll
                    for (int e = 0; e < 4; ++e) buf[(4 * (lane >> 5) + e) * 32 + (lane & 31)] = acc[m][n][e];
                    wave_sync();
                    const float4 r = reinterpret_cast<const float4 *>(buf)[lane];
                    float v[4] = {r.x, r.y, r.z, r.w};
                    put(p, q, v, old);
                }
        } else {
            // rows p of 32 floats; p and p + 4 are written together, so bit 0 of the
            // row is flipped by bit 2 to put them on different banks
            float *buf = reinterpret_cast<float *>(own_part(s));
            const auto row = [](int p) { return (p ^ ((p >> 2) & 1)) * 32; };
            constexpr int PR = BP / WP;
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                wave_sync();
#pragma unroll
                for (int m = 0; m < MI; ++m)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        buf[row(32 * m + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) + (lane & 31)] = acc[m][n][e];
                wave_sync();
                constexpr int AT = PR / 8 % 8 == 0 ? 8 : 6;
                static_assert(PR / 8 % AT == 0, "groups at a time");
#pragma unroll
                for (int i0 = 0; i0 < PR / 8; i0 += AT) {
                    decltype(get(0, 0)) old[AT];
#pragma unroll
                    for (int i = 0; i < AT; ++i) old[i] = get(p0 + 8 * (i0 + i) + (lane >> 3), q0 + 32 * n + 4 * (lane & 7));
#pragma unroll
                    for (int i = 0; i < AT; ++i) {
                        const int p = 8 * (i0 + i) + (lane >> 3);
                        const float4 r = *reinterpret_cast<const float4 *>(buf + row(p) + 4 * (lane & 7));
                        float v[4] = {r.x, r.y, r.z, r.w};
                        put(p0 + p, q0 + 32 * n + 4 * (lane & 7), v, old[i]);
                    }
                }
            }
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

// What bounds it.  bf16 8192^3 takes 870 to 920 us (1200 to 1260 TFLOP/s; the
// library's product 795), 4096^3 112 us.  On zeros it takes 800 us: with random
// operands the clock falls to 2.0 GHz under the MFMAs' power.  With the copies
// left out the products alone take 540 us, the copies alone 680 (64 KB per CU and
// step through the L2, 80 to 90 % of its requests hit).  Not faster, and not kept: four
// stages of half a step (1000 us), a third stage of P in the remaining 32 KB of
// LDS (920 to 950), copies staged through registers.
//
// Tile shapes.  256 x 256 by eight waves (128 x 64 each, one workgroup per CU:
// 128 KB of LDS), 192 x 192 by four (96 x 96 each, three stages in 144 KB) and
// 128 x 128 by four (64 x 64 each, two workgroups per CU).
// Products with few tiles take 64 x 64 or 32 x 32: each of four waves sums a
// quarter of every K-step over the whole tile, and the stages are deeper,
// because a step then lasts less than a copy takes to arrive.
struct Tile256 {
    static constexpr int BP = 256, BQ = 256, WP = 2, WQ = 4, WK = 1, STAGES = 2, NT = 512;
};
struct Tile192 {
    static constexpr int BP = 192, BQ = 192, WP = 2, WQ = 2, WK = 1, STAGES = 3, NT = 256;
};
struct Tile128 {
    static constexpr int BP = 128, BQ = 128, WP = 2, WQ = 2, WK = 1, STAGES = 2, NT = 256;
};
// few rows of Q (one decode step's tokens) against many of P: bound by reading P,
// so narrow, with four stages (two workgroups keep 120 KB per CU in flight)
struct TileRow {
    static constexpr int BP = 128, BQ = 32, WP = 4, WQ = 1, WK = 1, STAGES = 4, NT = 256;
};
struct Tile64 {
    static constexpr int BP = 64, BQ = 64, WP = 1, WQ = 1, WK = 4, STAGES = 4, NT = 256;
};
struct Tile32 {
    static constexpr int BP = 32, BQ = 32, WP = 1, WQ = 1, WK = 4, STAGES = 8, NT = 256;
};

// declares the LDS of a tile as `lds` (what a shape does not use is not allocated)
#define MM_STAGES(M)                                                                                              \
    __shared__ __attribute__((aligned(16))) char P0[M::P_BYTES], P1[M::P_BYTES], Q0[M::Q_BYTES], Q1[M::Q_BYTES];  \
    __shared__ __attribute__((aligned(16))) char P2[M::P_BYTES], P3[M::P_BYTES], Q2[M::Q_BYTES], Q3[M::Q_BYTES];  \
    __shared__ __attribute__((aligned(16))) char P4[M::P_BYTES], P5[M::P_BYTES], Q4[M::Q_BYTES], Q5[M::Q_BYTES];  \
    __shared__ __attribute__((aligned(16))) char P6[M::P_BYTES], P7[M::P_BYTES], Q6[M::Q_BYTES], Q7[M::Q_BYTES];  \
    __shared__ float4 red_[1024];                                                                                 \
    const typename M::Lds lds{{P0, P1, P2, P3, P4, P5, P6, P7}, {Q0, Q1, Q2, Q3, Q4, Q5, Q6, Q7}, red_}

// waves per SIMD that LDS leaves: one workgroup of Tile256 (eight waves) or of
// Tile192 (four), two of the others (four each) per CU
#define MM_BOUNDS(C) __launch_bounds__(C::NT, C::BP == 192 ? 1 : 2)

// Calls f with the tile shape that takes the least time for the busiest CU:
// count(edge) tiles dealt to 256 CUs, a tile's time being its area times what
// that shape takes per result against the largest (16 bits, measured at
// 4096^3 and, for the small ones, 512^3 and 1024^3; f32 is bound by the MFMA
// rate in every shape and loses only what small tiles wait for their copies).
template <typename E, typename N, typename F>
inline hipError_t mm_pick(N &&count, F &&f)
{
    constexpr bool H = sizeof(typename E::st) == 2;
    const int edge[5] = {256, 192, 128, 64, 32};
    const double per[5] = {1.0, 1.1, H ? 1.28 : 1.03, H ? 2.1 : 1.14, H ? 6.0 : 1.53};
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < 5; ++i) {
        const double t = (double)((count((int64_t)edge[i]) + 255) / 256) * edge[i] * edge[i] * per[i];
        if (i == 0 || t < least) {
            least = t;
            best = i;
        }
    }
    switch (best) {
    case 0: return f(Tile256{});
    case 1: return f(Tile192{});
    case 2: return f(Tile128{});
    case 3: return f(Tile64{});
    default: return f(Tile32{});
    }
}
