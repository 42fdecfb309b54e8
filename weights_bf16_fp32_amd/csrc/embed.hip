// Embedding lookup with scaling, and its gradient by sorted tokens, gfx950.
//
//   Y[i] = scale E[ids[i]];   dE[v] = scale sum_{ids[i] = v} dY[i]  (+ dE[v])
//
// A position whose id is no row of E gives a zero row and takes no gradient.
// Both are bound by memory: one read and one write per element.
//
// Gradient: the positions are sorted by id (stable, least significant digit
// first), so that the rows to be added lie next to each other, in the order of
// their positions; sums are formed in f32 in that order and are the same in
// every run.  Text repeats its frequent tokens thousands of times, so the
// sorted positions, not the vocabulary rows, are dealt out: a workgroup adds a
// fixed number of consecutive positions, writes the rows that end inside its
// share, and leaves the sums of the first and last row, where those continue
// in a neighbour's share, to be joined by a second pass.
//
// Lookup of 8192 rows of 4096 bf16: 18.9 us, 7.0 TB/s (repeated ids come from the
// caches); of 8 rows 4 us, a launch.  Gradient of 16384 rows into 131072 x 4096
// bf16: 60 us for the sort and 0.33 GB of zeros, 161 us for the sums and the other
// 0.75 GB (5.5 TB/s), 10 us for the joins.  The joins of one row follow each other in
// one workgroup per 256 threads of columns: with one id in all of 8192 positions of
// 4096 bf16, beta = 1 takes 194 us instead of 60, in all of 65536 428 instead of 327.
//
//   k_embed      lookup
//   k_eg_start   up to 16384 positions sorted by one workgroup; beside it, zeros
//                over the first rows of dE
//   k_sort_hist  more positions: digits per share of the positions,
//   k_sort_scan  first place of every (digit, share),
//   k_sort_move  positions to their places
//   k_eg_sum     sums over sorted positions; beside them, zeros in the other rows
//   k_eg_join    sums of rows that cross shares
#include <algorithm>
#include <limits.h>

#include "internal.h"
#include "mm.h"

namespace {

inline int64_t cdiv_h(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up_h(int64_t a, int64_t b) { return cdiv_h(a, b) * b; }

SPEC_DEVICE int64_t load_id(const void *p, int is64, int64_t i)
{
    return is64 ? reinterpret_cast<const int64_t *>(p)[i] : (int64_t) reinterpret_cast<const int32_t *>(p)[i];
}

// VEC elements of type S as one memory access
template <typename S, int VEC>
struct __attribute__((aligned(VEC * sizeof(S)))) Pack {
    S v[VEC];
};

// zeros that nothing reads back soon: past the caches (LINES), whose room the
// partial sums keep, where rows are whole cache lines; parts of lines meet in the L2
template <typename S, int VEC, bool LINES>
SPEC_DEVICE void put_zero(S *p)
{
    if constexpr (LINES) {
        static_assert(VEC * sizeof(S) == 16, "16 bytes");
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4 *>(p));
    } else {
        *reinterpret_cast<Pack<S, VEC> *>(p) = Pack<S, VEC>{};
    }
}

// a wave per row, and on by the grid's rows where one launch does not hold them all
template <typename E, int VEC>
__global__ __launch_bounds__(256) void k_embed(const typename E::st *__restrict__ tab, int64_t V, int64_t d, int64_t lde,
                                               const void *__restrict__ ids, int is64, int64_t n, float scale,
                                               typename E::st *__restrict__ Y, int64_t ldy)
{
    for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < n; i += 4 * (int64_t)gridDim.x) {
        const int64_t v = load_id(ids, is64, i);
        const bool ok = v >= 0 && v < V;
        const typename E::st *src = tab + (ok ? v : 0) * lde;
        typename E::st *dst = Y + i * ldy;
        for (int64_t c = VEC * (threadIdx.x & 63); c < d; c += VEC * 64) {
            Pack<typename E::st, VEC> x{};
            if (ok) x = *reinterpret_cast<const Pack<typename E::st, VEC> *>(src + c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x.v[e] = ok ? E::round(scale * E::wide(x.v[e])) : (typename E::st)0;
            *reinterpret_cast<Pack<typename E::st, VEC> *>(dst + c) = x;
        }
    }
}

// ------------------------------------------------------------------ sort

constexpr int SORT_SHARE = 2048;  // positions per workgroup (4 waves of 8 x 64)
constexpr int SORT_ROUNDS = SORT_SHARE / 256;
constexpr int DIGIT_MAX = 10;

// the sort key of position i: its id, or V (after every row) where it has none
SPEC_DEVICE int first_key(const void *ids, int is64, int64_t i, int64_t V)
{
    const int64_t v = load_id(ids, is64, i);
    return (int)(v >= 0 && v < V ? v : V);
}

__global__ __launch_bounds__(256) void k_sort_hist(const int *__restrict__ keys, const void *__restrict__ ids, int is64,
                                                   int64_t V, int64_t n, int shift, int bits, int nshare,
                                                   int *__restrict__ hist)
{
    __shared__ int cnt[1 << DIGIT_MAX];
    const int nd = 1 << bits;
    for (int i = threadIdx.x; i < nd; i += 256) cnt[i] = 0;
    __syncthreads();
    const int64_t b = (int64_t)blockIdx.x * SORT_SHARE;
    for (int k = threadIdx.x; k < SORT_SHARE; k += 256)
        if (b + k < n) {
            const int key = keys != nullptr ? keys[b + k] : first_key(ids, is64, b + k, V);
            atomicAdd(&cnt[(key >> shift) & (nd - 1)], 1);  // counts: the order does not matter
        }
    __syncthreads();
    for (int i = threadIdx.x; i < nd; i += 256) hist[i * nshare + blockIdx.x] = cnt[i];
}

// exclusive sums of hist[0 .. m) by one workgroup
__global__ __launch_bounds__(1024) void k_sort_scan(int *__restrict__ hist, int m)
{
    __shared__ int wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (m + 1023) / 1024;
    const int b = tid * per, e = min(m, b + per);
    int s = 0;
    for (int i = b; i < e; ++i) s += hist[i];
    int inc = s;
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 63) wsum[wave] = inc;
    __syncthreads();
    int base = inc - s;
    for (int w = 0; w < wave; ++w) base += wsum[w];
    for (int i = b; i < e; ++i) {
        const int x = hist[i];
        hist[i] = base;
        base += x;
    }
}

__global__ __launch_bounds__(256) void k_sort_move(const int *__restrict__ keys, const int *__restrict__ idx,
                                                   const void *__restrict__ ids, int is64, int64_t V, int64_t n,
                                                   int shift, int bits, int nshare, const int *__restrict__ base,
                                                   int *__restrict__ okeys, int *__restrict__ oidx)
{
    __shared__ int cnt[4][1 << DIGIT_MAX];
    const int nd = 1 << bits;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < 4 * nd; i += 256) cnt[i >> bits][i & (nd - 1)] = 0;
    __syncthreads();
    const int64_t b = (int64_t)blockIdx.x * SORT_SHARE + wave * (SORT_SHARE / 4);
    int key[SORT_ROUNDS], rank[SORT_ROUNDS];
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        const int64_t i = b + r * 64 + lane;
        const bool in = i < n;
        key[r] = !in ? 0 : (keys != nullptr ? keys[i] : first_key(ids, is64, i, V));
        const int dg = (key[r] >> shift) & (nd - 1);
        uint64_t same = __ballot(in);  // lanes with this lane's digit
        for (int k = 0; k < bits; ++k) {
            const uint64_t m = __ballot((dg >> k) & 1);
            same &= (dg >> k) & 1 ? m : ~m;
        }
        const int before = __popcll(same & ((1ull << lane) - 1));
        rank[r] = in ? cnt[wave][dg] + before : 0;
        wave_sync();
        if (in && before == 0) cnt[wave][dg] += __popcll(same);
        wave_sync();
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        const int64_t i = b + r * 64 + lane;
        if (i >= n) continue;
        const int dg = (key[r] >> shift) & (nd - 1);
        int at = base[dg * nshare + blockIdx.x] + rank[r];
        for (int w = 0; w < wave; ++w) at += cnt[w][dg];
        okeys[at] = key[r];
        oidx[at] = idx != nullptr ? idx[i] : (int)i;
    }
}

// ------------------------------------------------------------------ one workgroup's sort

// Positions at most: what its LDS holds.  Against the sort by many workgroups (three
// launches a pass) the gradient takes, with beta = 1 and nothing to hide the sort behind,
// 20 us for 41 at 1024 x 4096 bf16, 60 for 79 at 8192, 88 for 96 at 16384; into the 512
// columns of a table of 4096 rows 18 for 36, 36 for 51, 58 for 57.
constexpr int ONE_MAX = 16384;
constexpr int ONE_BITS = 9;     // of the key per pass

struct __attribute__((aligned(16))) OneLds {
    int cnt[16][1 << ONE_BITS];
    int buf[ONE_MAX];
    int wsum[8];
};

// The positions in order of their keys, by 1024 threads: keys and positions stay
// in registers (wave w holds the places w 64 R .. in rounds of 64) and change
// places through LDS once per pass.
template <int ROUNDS>
SPEC_DEVICE void sort_rounds(OneLds &s, const void *ids, int is64, int64_t V, int n, int passes, int *okeys, int *oidx)
{
    constexpr int ND = 1 << ONE_BITS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int R = (n + 1023) / 1024;
    int key[ROUNDS], idx[ROUNDS], at[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = (wave * R + r) * 64 + lane;
        idx[r] = i;
        key[r] = r < R && i < n ? first_key(ids, is64, i, V) : 0;
    }
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * ONE_BITS;
        for (int i = tid; i < 16 * ND; i += 1024) s.cnt[i / ND][i % ND] = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const bool in = r < R && (wave * R + r) * 64 + lane < n;
            const int dg = (key[r] >> shift) & (ND - 1);
            uint64_t same = __ballot(in);  // lanes with this lane's digit
#pragma unroll
            for (int k = 0; k < ONE_BITS; ++k) {
                const uint64_t m = __ballot((dg >> k) & 1);
                same &= (dg >> k) & 1 ? m : ~m;
            }
            const int before = __popcll(same & ((1ull << lane) - 1));
            at[r] = in ? s.cnt[wave][dg] + before : 0;
            wave_sync();
            if (in && before == 0) s.cnt[wave][dg] += __popcll(same);
            wave_sync();
        }
        __syncthreads();
        // places: digits in order, and of one digit the waves in order
        int total = 0;
        if (tid < ND)
            for (int w = 0; w < 16; ++w) {
                const int x = s.cnt[w][tid];
                s.cnt[w][tid] = total;
                total += x;
            }
        int inc = total;
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 63 && wave < 8) s.wsum[wave] = inc;
        __syncthreads();
        if (tid < ND) {
            int base = inc - total;
            for (int w = 0; w < wave; ++w) base += s.wsum[w];
            for (int w = 0; w < 16; ++w) s.cnt[w][tid] += base;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if (r >= R || (wave * R + r) * 64 + lane >= n) continue;
            at[r] += s.cnt[wave][(key[r] >> shift) & (ND - 1)];
            s.buf[at[r]] = key[r];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int i = (wave * R + r) * 64 + lane;
            if (r < R && i < n) key[r] = s.buf[i];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            if (r < R && (wave * R + r) * 64 + lane < n) s.buf[at[r]] = idx[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int i = (wave * R + r) * 64 + lane;
            if (r < R && i < n) idx[r] = s.buf[i];
        }
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = (wave * R + r) * 64 + lane;
        if (r < R && i < n) {
            okeys[i] = key[r];
            oidx[i] = idx[r];
        }
    }
}

// Up to 256 positions: a thread's place is the number of keys before its own.
SPEC_DEVICE void sort_few(OneLds &s, const void *ids, int is64, int64_t V, int n, int *okeys, int *oidx)
{
    const int tid = threadIdx.x;
    const int key = tid < n ? first_key(ids, is64, tid, V) : INT_MAX;
    if (tid < 256) s.buf[tid] = key;
    __syncthreads();
    if (tid >= n) return;
    int at = 0;
    for (int j = 0; j < n; j += 4) {
        const int4 o = *reinterpret_cast<const int4 *>(&s.buf[j]);
        at += (o.x < key || (o.x == key && j < tid)) + (o.y < key || (o.y == key && j + 1 < tid)) +
              (o.z < key || (o.z == key && j + 2 < tid)) + (o.w < key || (o.w == key && j + 3 < tid));
    }
    okeys[at] = key;
    oidx[at] = tid;
}

// (the rounds are a constant, so that the arrays are registers)
SPEC_DEVICE void sort_one(OneLds &s, const void *ids, int is64, int64_t V, int n, int passes, int *okeys, int *oidx)
{
    if (n <= 256) sort_few(s, ids, is64, V, n, okeys, oidx);
    else if (n <= 2048) sort_rounds<2>(s, ids, is64, V, n, passes, okeys, oidx);
    else if (n <= 4096) sort_rounds<4>(s, ids, is64, V, n, passes, okeys, oidx);
    else if (n <= 8192) sort_rounds<8>(s, ids, is64, V, n, passes, okeys, oidx);
    else sort_rounds<ONE_MAX / 1024>(s, ids, is64, V, n, passes, okeys, oidx);
}

// ------------------------------------------------------------------ sums

// Sorted positions per workgroup: few where there are few, so that they fill the
// chip; more leave fewer rows to be joined.  With 8 and with 32, beta = 1, 4096 bf16 per
// row: 2048 positions 26 and 37 us, 8192 62 and 61, 16384 102 and 88; 1000 per row: 21
// and 33, 42 and 50, 68 and 73.  (Beside the zeros of 131072 rows 32 are better from 4096
// positions on already: 217 and 205 us, at 8192 227 and 202.)
inline int eg_share(int64_t n) { return n <= 8192 ? 8 : 32; }
constexpr int EG_AHEAD = 8;   // rows in flight per thread

// Workgroup 0 sorts (sort != 0); the others write zeros over dE's rows below
// `rows`, about as many as are written while it does.
template <typename O, int VEC, bool LINES>
__global__ __launch_bounds__(1024) void k_eg_start(const void *__restrict__ ids, int is64, int64_t V, int n, int passes,
                                                   int sort, int *__restrict__ okeys, int *__restrict__ oidx,
                                                   typename O::st *__restrict__ dE, int64_t rows, int64_t d, int64_t ldd)
{
    __shared__ OneLds lds;
    if (sort && blockIdx.x == 0) {
        sort_one(lds, ids, is64, V, n, passes, okeys, oidx);
        return;
    }
    const int64_t first = (int64_t)(blockIdx.x - sort) * 16 + (threadIdx.x >> 6), step = 16 * (int64_t)(gridDim.x - sort);
    for (int64_t v = first; v < rows; v += step)
        for (int64_t c = VEC * (threadIdx.x & 63); c < d; c += VEC * 64)
            put_zero<typename O::st, VEC, LINES>(dE + v * ldd + c);
}

template <typename O, int VEC>
SPEC_DEVICE void eg_put(typename O::st *row, int64_t c, const float (&s)[VEC], float scale, int add)
{
    Pack<typename O::st, VEC> x;
    if (add) x = *reinterpret_cast<const Pack<typename O::st, VEC> *>(row + c);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x.v[e] = O::round(add ? O::wide(x.v[e]) + scale * s[e] : scale * s[e]);
    *reinterpret_cast<Pack<typename O::st, VEC> *>(row + c) = x;
}

// Zeros in the rows v0 .. v0 + 63 that no position names: each lane looks one of
// them up in the sorted keys.
template <typename O, int VEC, bool LINES>
SPEC_DEVICE void eg_gaps(const int *__restrict__ keys, int64_t n, int64_t V, int64_t v0, typename O::st *__restrict__ dE,
                         int64_t d, int64_t ldd)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t v = v0 + lane;
    int64_t lo = 0, hi = n;  // first position with a key of v or more
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (keys[mid] < v)
            lo = mid + 1;
        else
            hi = mid;
    }
    const uint64_t absent = __ballot(v < V && (lo == n || keys[lo] != v));
    for (int r = wave * 16; r < wave * 16 + 16; ++r)
        if ((absent >> r) & 1)
            for (int64_t c = VEC * lane; c < d; c += VEC * 64)
                put_zero<typename O::st, VEC, LINES>(dE + (v0 + r) * ldd + c);
}

// The first `sums` workgroups add, cols (column blocks of 256 VEC) of them per
// share from share0 on; the others write the zero rows from row0 on.  head[share] / tail[share]: the sum
// of the share's first / last row where it began before / goes on after.
// Positions are taken EG_AHEAD at a time, their rows requested together.
template <typename E, typename O, int VEC, bool LINES>
__global__ __launch_bounds__(256) void k_eg_sum(const typename E::st *__restrict__ dY, int64_t d, int64_t ldy,
                                                const int *__restrict__ keys, const int *__restrict__ idx, int64_t n,
                                                int64_t V, float scale, int add, typename O::st *__restrict__ dE,
                                                int64_t ldd, float *__restrict__ head, float *__restrict__ tail,
                                                int64_t share0, int64_t sums, int cols, int64_t row0, int len)
{
    if (blockIdx.x >= sums) {
        eg_gaps<O, VEC, LINES>(keys, n, V, row0 + ((int64_t)blockIdx.x - sums) * 64, dE, d, ldd);
        return;
    }
    const int64_t share = share0 + blockIdx.x / cols;
    using P = Pack<typename E::st, VEC>;
    const int64_t b = share * len, e = min<int64_t>(n, b + len);
    const int64_t c = VEC * ((int64_t)(blockIdx.x % cols) * 256 + threadIdx.x);
    if (c >= d || keys[b] >= V) return;
    float s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[k] = 0.f;
    bool open = b > 0 && keys[b - 1] == keys[b];  // the row began before this share
    const auto leave = [&](float *p) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) p[share * d + c + k] = s[k];
    };
    int cur = keys[b];
    for (int64_t i0 = b; i0 < e; i0 += EG_AHEAD) {
        P x[EG_AHEAD];
        int key[EG_AHEAD];
#pragma unroll
        for (int j = 0; j < EG_AHEAD; ++j) {
            const int64_t i = min<int64_t>(i0 + j, e - 1);
            key[j] = i0 + j < e ? keys[i] : (int)V;
            // (positions without a token have the last keys; their rows are not read)
            x[j] = key[j] < V ? *reinterpret_cast<const P *>(dY + (int64_t)idx[i] * ldy + c) : P{};
        }
#pragma unroll
        for (int j = 0; j < EG_AHEAD; ++j) {
            if (key[j] != cur) {
                if (cur < V) {
                    if (open)
                        leave(head);
                    else if (i0 + j < e || e == n || keys[e] != cur)
                        eg_put<O, VEC>(dE + cur * ldd, c, s, scale, add);
                    else
                        leave(tail);
                }
                open = false;
                cur = key[j];
#pragma unroll
                for (int k = 0; k < VEC; ++k) s[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) s[k] += E::wide(x[j].v[k]);
        }
    }
    if (cur < V) {
        if (open)
            leave(head);
        else if (e == n || keys[e] != cur)
            eg_put<O, VEC>(dE + cur * ldd, c, s, scale, add);
        else
            leave(tail);
    }
}

// a row that begins in this share and goes on: its tail here and the heads after it
template <typename O, int VEC>
__global__ __launch_bounds__(256) void k_eg_join(int64_t d, const int *__restrict__ keys, int64_t n, int64_t V,
                                                 float scale, int add, typename O::st *__restrict__ dE, int64_t ldd,
                                                 const float *__restrict__ head, const float *__restrict__ tail,
                                                 int64_t share0, int len)
{
    const int64_t share = share0 + blockIdx.x, b = share * len, e = b + len;
    const int64_t c = VEC * ((int64_t)blockIdx.y * 256 + threadIdx.x);
    if (c >= d || e >= n) return;
    const int key = keys[e - 1];
    if (key >= V || keys[e] != key) return;
    if (keys[b] == key && b > 0 && keys[b - 1] == key) return;  // began earlier
    // the shares it goes through: those whose first position still has its key
    int64_t lo = share + 1, hi = (n - 1) / len;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (keys[mid * len] == key)
            lo = mid;
        else
            hi = mid - 1;
    }
    float s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[k] = tail[share * d + c + k];
#pragma unroll 8
    for (int64_t f = share + 1; f <= lo; ++f)
#pragma unroll
        for (int k = 0; k < VEC; ++k) s[k] += head[f * d + c + k];
    eg_put<O, VEC>(dE + key * ldd, c, s, scale, add);
}

struct EgPlan {
    bool one;  // one workgroup sorts
    int nshare, passes, bits;
    int64_t key[2], idx[2], hist, head, tail, total;
};

EgPlan eg_plan(int64_t n, int64_t V, int64_t d)
{
    EgPlan p{};
    int kb = 1;  // bits of the largest key, V
    while ((V >> kb) != 0) ++kb;
    p.one = n <= ONE_MAX;
    p.passes = (int)cdiv_h(kb, p.one ? ONE_BITS : DIGIT_MAX);
    p.bits = (int)cdiv_h(kb, p.passes);
    const int64_t nn = std::max<int64_t>(n, 1);
    p.nshare = (int)cdiv_h(nn, SORT_SHARE);
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o += up_h(bytes, 256);
        return at;
    };
    for (int i = 0; i < 2; ++i) {
        p.key[i] = take(4 * nn);
        p.idx[i] = take(4 * nn);
    }
    p.hist = take((int64_t)4 * p.nshare << p.bits);
    p.head = take(4 * cdiv_h(nn, eg_share(n)) * d);
    p.tail = take(4 * cdiv_h(nn, eg_share(n)) * d);
    p.total = o;
    return p;
}

template <typename E, typename O, int VEC, bool LINES>
hipError_t eg_launch(hipStream_t stream, const void *dY, int64_t n, int64_t V, int64_t d, int64_t ldy, const void *ids,
                     int is64, float scale, int add, void *dE, int64_t ldd, char *ws)
{
    const EgPlan p = eg_plan(n, V, d);
    typename O::st *out = (typename O::st *)dE;
    const int sort = p.one && n > 0;
    // rows written beside the sort: what 6 TB/s write while it takes its 10 us (2048
    // positions) to 55 us (16384); all of them where there is nothing to sort, none
    // where more positions are sorted by kernels of their own
    const int64_t es = sizeof(typename O::st);
    const int64_t early = add ? 0 : (n == 0 ? V : !p.one ? 0 : std::min<int64_t>(V, (n * 18000 + (32 << 20)) / (d * es) / 64 * 64));
    const int fill = (int)std::min<int64_t>(cdiv_h(early, 16), 2048);
    const int last = p.one ? 0 : (p.passes + 1) & 1;
    int *okeys = (int *)(ws + p.key[last]), *oidx = (int *)(ws + p.idx[last]);
    if (sort + fill > 0) {
        hipLaunchKernelGGL((k_eg_start<O, VEC, LINES>), dim3((unsigned)(sort + fill)), dim3(1024), 0, stream, ids, is64, V, (int)n,
                           p.passes, sort, okeys, oidx, out, early, d, ldd);
        SPEC_LAUNCH_CHECK();
    }
    if (n == 0) return hipSuccess;
    int *hist = (int *)(ws + p.hist);
    for (int k = 0; k < p.passes && !p.one; ++k) {
        const int *keys = k == 0 ? nullptr : (const int *)(ws + p.key[(k + 1) & 1]);
        const int *idx = k == 0 ? nullptr : (const int *)(ws + p.idx[(k + 1) & 1]);
        hipLaunchKernelGGL(k_sort_hist, dim3((unsigned)p.nshare), dim3(256), 0, stream, keys, ids, is64, V, n, k * p.bits,
                           p.bits, p.nshare, hist);
        SPEC_LAUNCH_CHECK();
        hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(1024), 0, stream, hist, p.nshare << p.bits);
        SPEC_LAUNCH_CHECK();
        hipLaunchKernelGGL(k_sort_move, dim3((unsigned)p.nshare), dim3(256), 0, stream, keys, idx, ids, is64, V, n,
                           k * p.bits, p.bits, p.nshare, hist, (int *)(ws + p.key[k & 1]), (int *)(ws + p.idx[k & 1]));
        SPEC_LAUNCH_CHECK();
    }
    const int *keys = okeys, *idx = oidx;
    const int len = eg_share(n);
    const int64_t shares = cdiv_h(n, len), cols = cdiv_h(d, 256 * VEC);
    const int64_t gaps = add ? 0 : cdiv_h(V - early, 64);
    float *head = (float *)(ws + p.head), *tail = (float *)(ws + p.tail);
    // (one launch each unless there are more shares or zero rows than it holds)
    constexpr int64_t most = LAUNCH_THREADS / 256;
    for (int64_t share = 0, gap = 0; share < shares || gap < gaps;) {
        const int64_t ns = std::min(shares - share, most / cols), ng = std::min(gaps - gap, most - ns * cols);
        hipLaunchKernelGGL((k_eg_sum<E, O, VEC, LINES>), dim3((unsigned)(ns * cols + ng)), dim3(256), 0, stream,
                           (const typename E::st *)dY, d, ldy, keys, idx, n, V, scale, add, out, ldd, head, tail, share,
                           ns * cols, (int)cols, early + 64 * gap, len);
        SPEC_LAUNCH_CHECK();
        share += ns;
        gap += ng;
    }
    for (int64_t share = 0; share < shares; share += most) {
        const int64_t ns = std::min(shares - share, most);
        hipLaunchKernelGGL((k_eg_join<O, VEC>), dim3((unsigned)ns, (unsigned)cols), dim3(256), 0, stream, d, keys, n, V,
                           scale, add, out, ldd, head, tail, share, len);
        SPEC_LAUNCH_CHECK();
    }
    return hipSuccess;
}

template <typename E, typename O, int VEC>
hipError_t eg_run(hipStream_t stream, const void *dY, int64_t n, int64_t V, int64_t d, int64_t ldy, const void *ids,
                  int is64, float scale, int add, void *dE, int64_t ldd, char *ws)
{
    constexpr int64_t es = sizeof(typename O::st);
    if constexpr (VEC * es == 16)
        if ((uintptr_t)dE % 128 == 0 && ldd * es % 128 == 0 && d * es % 128 == 0)
            return eg_launch<E, O, VEC, true>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, ws);
    return eg_launch<E, O, VEC, false>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, ws);
}

template <typename E>
hipError_t embed_run(hipStream_t stream, const void *tab, int64_t V, int64_t d, int64_t lde, const void *ids, int is64,
                     int64_t n, float scale, void *Y, int64_t ldy)
{
    using st = typename E::st;
    constexpr int VEC = 16 / sizeof(st);
    const dim3 grid((unsigned)std::min(cdiv_h(n, 4), LAUNCH_THREADS / 256));
    const bool vec = (uintptr_t)tab % 16 == 0 && (uintptr_t)Y % 16 == 0 && d % VEC == 0 && lde % VEC == 0 && ldy % VEC == 0;
    if (vec)
        hipLaunchKernelGGL((k_embed<E, VEC>), grid, dim3(256), 0, stream, (const st *)tab, V, d, lde, ids, is64, n, scale,
                           (st *)Y, ldy);
    else
        hipLaunchKernelGGL((k_embed<E, 1>), grid, dim3(256), 0, stream, (const st *)tab, V, d, lde, ids, is64, n, scale,
                           (st *)Y, ldy);
    return hipGetLastError();
}

}  // namespace

size_t embed_grad_workspace_bytes(int64_t n, int64_t V, int64_t d) { return (size_t)eg_plan(n, V, d).total; }

hipError_t launch_embed(hipStream_t stream, const void *E, int t, int64_t V, int64_t d, int64_t lde, const void *ids,
                        int is64, int64_t n, float scale, void *Y, int64_t ldy)
{
    if (n == 0) return hipSuccess;
    return t == SPEC_BF16 ? embed_run<ElBF16>(stream, E, V, d, lde, ids, is64, n, scale, Y, ldy)
                          : embed_run<ElF32>(stream, E, V, d, lde, ids, is64, n, scale, Y, ldy);
}

hipError_t launch_embed_grad(hipStream_t stream, const void *dY, int yt, int64_t n, int64_t V, int64_t d, int64_t ldy,
                             const void *ids, int is64, float scale, int add, void *dE, int et, int64_t ldd, void *ws)
{
    const int64_t ys = yt == SPEC_BF16 ? 2 : 4, es = et == SPEC_BF16 ? 2 : 4;
    char *w = (char *)ws;
    // eight or four elements per thread where both sides are aligned to them
    const auto can = [&](int64_t k) {
        return d % k == 0 && ldy % k == 0 && ldd % k == 0 && (uintptr_t)dY % (k * ys) == 0 && (uintptr_t)dE % (k * es) == 0;
    };
    if (yt == SPEC_BF16 && et == SPEC_BF16)
        return can(8)   ? eg_run<ElBF16, ElBF16, 8>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, w)
               : can(4) ? eg_run<ElBF16, ElBF16, 4>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, w)
                        : eg_run<ElBF16, ElBF16, 1>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, w);
    if (yt == SPEC_BF16)
        return can(4) ? eg_run<ElBF16, ElF32, 4>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, w)
                      : eg_run<ElBF16, ElF32, 1>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, w);
    return can(4) ? eg_run<ElF32, ElF32, 4>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, w)
                  : eg_run<ElF32, ElF32, 1>(stream, dY, n, V, d, ldy, ids, is64, scale, add, dE, ldd, w);
}
