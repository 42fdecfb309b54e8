// Microscaled storage of matrices and back, gfx950 (the format: mx.h).
//
// Both directions are bound by memory: one read and one write per element, 3.03 bytes
// (bf16 and int8) to 5.03 (f32).  Medians: 16384 x 4096 bf16 to int8 and back 39 and 39 us over
// four matrices in turn (5.2 TB/s), 40 and 33 over one (the codes partly from the caches); 14336 x
// 4096 bf16 to FP4 and back 30 and 30 us (5.0 and 4.9 TB/s), 1000 x 333 f32 4.4 and 3.5 us.
// Four lanes hold a block of 32, eight values each (one 16-byte load of bf16), so the
// block's largest value takes two lane exchanges and nothing goes through LDS.  A row is
// given to as many lanes as it has eights (a power of two, at most 256), several rows of a
// short kind to a workgroup.
#include <algorithm>

#include "mx.h"

namespace {

inline int64_t cdiv_h(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int UNITS = 4;  // eights of a row per lane in flight

// Lane l of the 2^lg lanes of a row takes the eights (tile UNITS + u) 2^lg + l.
struct MxMap {
    int lg;        // log2 of the lanes of a row
    int tiles;     // workgroups along a row
    int64_t groups;  // workgroups along the rows
};

inline MxMap mx_map(int64_t rows, int64_t cols)
{
    MxMap m;
    const int64_t eights = cdiv_h(cols, 32) * 4;
    m.lg = 2;
    while (m.lg < 8 && ((int64_t)UNITS << m.lg) < eights) ++m.lg;
    m.tiles = (int)cdiv_h(eights, (int64_t)UNITS << m.lg);
    m.groups = cdiv_h(rows, 256 >> m.lg);
    return m;
}

template <typename E, int FMT>
__global__ __launch_bounds__(256) void k_mx_quantize(const typename E::st *__restrict__ X, int64_t rows, int64_t cols,
                                                     int64_t ldx, int lg, int tiles, int64_t units,
                                                     uint8_t *__restrict__ Q, int64_t ldq, uint8_t *__restrict__ S,
                                                     int64_t lds)
{
    const int lane = threadIdx.x & ((1 << lg) - 1);
    const int64_t blocks = (cols + 31) / 32, scales = (blocks + 15) / 16 * 16;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t r = (unit / tiles << (8 - lg)) + (threadIdx.x >> lg);
        const int64_t c0 = unit % tiles * ((int64_t)UNITS << lg) + lane;
        if (r >= rows) continue;  // whole groups of four lanes
        const typename E::st *x = X + r * ldx;
        Raw8<E> v[UNITS];
        const int e0 = (int)c0 * 8, d = (int)cols;
        if (d >= 8) {
#pragma unroll
            for (int u = 0; u < UNITS; ++u) v[u] = load8_start<E>(x, e0 + (8 * u << lg), d);
#pragma unroll
            for (int u = 0; u < UNITS; ++u) load8_end<E>(v[u], e0 + (8 * u << lg), d);
        } else {
#pragma unroll
            for (int u = 0; u < UNITS; ++u) v[u] = load8_tiny<E>(x, e0 + (8 * u << lg), d);
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int64_t c = c0 + ((int64_t)u << lg);
            const int b = mx_scale<FMT>(mx_top<E>(v[u]));
            if (c < blocks * 4) {
                if constexpr (FMT == SPEC_MX_INT8)
                    *reinterpret_cast<uint2 *>(Q + r * ldq + c * 8) = mx_encode_int8<E>(v[u], b);
                else
                    *reinterpret_cast<uint32_t *>(Q + r * ldq + c * 4) = mx_encode_fp4<E>(v[u], b);
            }
            if ((c & 3) == 0 && c < blocks * 4) S[r * lds + (c >> 2)] = (uint8_t)b;
        }
        if (unit % tiles == tiles - 1 && lane < scales - blocks) S[r * lds + blocks + lane] = 0;
        if (unit % tiles == tiles - 1 && lg < 4)  // four or eight lanes for up to fifteen bytes
            for (int64_t i = lane + (1 << lg); i < scales - blocks; i += 1 << lg) S[r * lds + blocks + i] = 0;
    }
}

template <typename E, int FMT>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t *__restrict__ Q, int64_t ldq,
                                                       const uint8_t *__restrict__ S, int64_t lds, int64_t rows,
                                                       int64_t cols, int64_t width, int lg, int tiles, int64_t units,
                                                       typename E::st *__restrict__ X, int64_t ldx)
{
    const int lane = threadIdx.x & ((1 << lg) - 1);
    const int64_t blocks = (cols + 31) / 32;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t r = (unit / tiles << (8 - lg)) + (threadIdx.x >> lg);
        const int64_t c0 = unit % tiles * ((int64_t)UNITS << lg) + lane;
        if (r >= rows) continue;
        uint2 q[UNITS];
        int b[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int64_t c = c0 + ((int64_t)u << lg);
            q[u] = make_uint2(0, 0);
            b[u] = 0;
            if (c < blocks * 4) {
                b[u] = S[r * lds + (c >> 2)];
                if constexpr (FMT == SPEC_MX_INT8)
                    q[u] = *reinterpret_cast<const uint2 *>(Q + r * ldq + c * 8);
                else
                    q[u].x = *reinterpret_cast<const uint32_t *>(Q + r * ldq + c * 4);
            }
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int64_t c = c0 + ((int64_t)u << lg);
            float v[8];
            if constexpr (FMT == SPEC_MX_INT8)
                mx_decode_int8(q[u].x, q[u].y, mx_unit_int8(b[u]), v);
            else
                mx_decode_fp4(q[u].x, mx_factor(b[u]), v);
            if (c * 8 < width) store8<E>(X + r * ldx, c * 8, width, mx_raw<E>(v));
        }
    }
}

template <typename E, int FMT>
hipError_t quantize(hipStream_t stream, const void *X, int64_t rows, int64_t cols, int64_t ldx, const spec_mx *out)
{
    const MxMap m = mx_map(rows, cols);
    const int64_t units = m.groups * m.tiles;
    hipLaunchKernelGGL((k_mx_quantize<E, FMT>), dim3((unsigned)std::min(units, LAUNCH_THREADS / 256)), dim3(256), 0,
                       stream, (const typename E::st *)X, rows, cols, ldx, m.lg, m.tiles, units, (uint8_t *)out->q,
                       out->ldq, (uint8_t *)out->s, out->lds);
    return hipGetLastError();
}

template <typename E, int FMT>
hipError_t dequantize(hipStream_t stream, const spec_mx *in, int64_t rows, int64_t cols, int64_t width, void *X,
                      int64_t ldx)
{
    const MxMap m = mx_map(rows, cols);
    const int64_t units = m.groups * m.tiles;
    hipLaunchKernelGGL((k_mx_dequantize<E, FMT>), dim3((unsigned)std::min(units, LAUNCH_THREADS / 256)), dim3(256), 0,
                       stream, (const uint8_t *)in->q, in->ldq, (const uint8_t *)in->s, in->lds, rows, cols, width, m.lg,
                       m.tiles, units, (typename E::st *)X, ldx);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(hipStream_t stream, const void *X, int t, int64_t rows, int64_t cols, int64_t ldx,
                              const spec_mx *out)
{
    if (rows == 0) return hipSuccess;
    if (out->fmt == SPEC_MX_INT8)
        return t == SPEC_BF16 ? quantize<ElBF16, SPEC_MX_INT8>(stream, X, rows, cols, ldx, out)
                              : quantize<ElF32, SPEC_MX_INT8>(stream, X, rows, cols, ldx, out);
    return t == SPEC_BF16 ? quantize<ElBF16, SPEC_MX_FP4>(stream, X, rows, cols, ldx, out)
                          : quantize<ElF32, SPEC_MX_FP4>(stream, X, rows, cols, ldx, out);
}

hipError_t launch_mx_dequantize(hipStream_t stream, const spec_mx *in, int64_t rows, int64_t cols, int64_t width, void *X,
                                int t, int64_t ldx)
{
    if (rows == 0) return hipSuccess;
    if (in->fmt == SPEC_MX_INT8)
        return t == SPEC_BF16 ? dequantize<ElBF16, SPEC_MX_INT8>(stream, in, rows, cols, width, X, ldx)
                              : dequantize<ElF32, SPEC_MX_INT8>(stream, in, rows, cols, width, X, ldx);
    return t == SPEC_BF16 ? dequantize<ElBF16, SPEC_MX_FP4>(stream, in, rows, cols, width, X, ldx)
                          : dequantize<ElF32, SPEC_MX_FP4>(stream, in, rows, cols, width, X, ldx);
}
