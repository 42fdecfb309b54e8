// C ABI of the spectral library: argument validation and dispatch to the
// gfx950 kernels.  Every check runs on the host before anything is enqueued;
// nothing here allocates device memory or synchronises.
#include <hip/hip_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "internal.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

inline int from_hip(hipError_t e) { return e == hipSuccess ? SPEC_OK : SPEC_EHIP; }

inline size_t elt_size(int t) { return t == SPEC_BF16 ? 2 : (t == SPEC_F32 ? 4 : 8); }

// the descriptor parameters for spectra of r values
int check_desc_params(int64_t r, const spec_desc_params *p)
{
    if (p == nullptr || r < 2) return SPEC_EINVAL;
    if (p->k < 1 || p->k >= r || p->n_samples < 1 || p->p_dim < 1) return SPEC_EINVAL;
    if (!(p->top_frac >= 0.0 && p->top_frac <= 1.0) || !(p->tail_frac >= 0.0 && p->tail_frac <= 1.0) ||
        !(p->small_rel >= 0.0))
        return SPEC_EINVAL;
    if (p->sigma2_mode < SPEC_SIGMA2_GIVEN || p->sigma2_mode > SPEC_SIGMA2_MEAN) return SPEC_EINVAL;
    if (p->sigma2_mode == SPEC_SIGMA2_GIVEN && !(p->sigma2 > 0.0 && isfinite(p->sigma2))) return SPEC_EINVAL;
    return SPEC_OK;
}

// the checks spec_descriptors and spec_descriptors_static share
int check_descriptors(const void *w, int wt, int64_t batch, int64_t r, int64_t ldw, const spec_desc_params *p,
                      spec_desc *out)
{
    if (w == nullptr || p == nullptr || out == nullptr) return SPEC_EINVAL;
    if (wt != SPEC_F32 && wt != SPEC_F64) return SPEC_EUNSUPPORTED;
    if (batch < 0 || batch > ((int64_t)1 << 31) - 1 || r < 2 || ldw < r) return SPEC_EINVAL;
    if (p->k < 1 || p->k >= r || p->n_samples < 1 || p->p_dim < 1) return SPEC_EINVAL;
    if (!(p->top_frac >= 0.0 && p->top_frac <= 1.0) || !(p->tail_frac >= 0.0 && p->tail_frac <= 1.0) ||
        !(p->small_rel >= 0.0))
        return SPEC_EINVAL;
    if (p->sigma2_mode < SPEC_SIGMA2_GIVEN || p->sigma2_mode > SPEC_SIGMA2_MEAN) return SPEC_EINVAL;
    if (p->sigma2_mode == SPEC_SIGMA2_GIVEN && !(p->sigma2 > 0.0 && isfinite(p->sigma2))) return SPEC_EINVAL;
    if (!aligned(w, elt_size(wt)) || !aligned(out, 8)) return SPEC_EINVAL;
    return SPEC_OK;
}

// whether a factor that the kernels apply in f32 is finite there
inline bool finite32(double x) { return fabs(x) <= FLT_MAX; }

// sizes shared by the vocabulary operators, and the type of a token id array
int check_rows(int64_t n, int64_t V, int64_t d)
{
    const int64_t lim = (int64_t)1 << 31;
    if (n < 0 || n >= lim || V < 1 || V >= lim - 1 || d < 1 || d > ((int64_t)1 << 20)) return SPEC_EINVAL;
    return SPEC_OK;
}

int check_ids(const void *ids, int idt, int64_t n)
{
    if (idt != SPEC_I32 && idt != SPEC_I64) return SPEC_EUNSUPPORTED;
    if (n > 0 && (ids == nullptr || !aligned(ids, idt == SPEC_I32 ? 4 : 8))) return SPEC_EINVAL;
    return SPEC_OK;
}

int check_xent_sizes(int64_t T, int64_t V, int64_t d, int t)
{
    if (t != SPEC_BF16 && t != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (T > ((int64_t)1 << 22)) return SPEC_EINVAL;
    const int st = check_rows(T, V, d);
    if (st != SPEC_OK) return st;
    // tiles of 128 x 128 logits are counted in 31 bits
    if ((T + 127) / 128 * ((V + 127) / 128) >= ((int64_t)1 << 30)) return SPEC_EUNSUPPORTED;
    return SPEC_OK;
}

int check_ortho_sizes(int64_t batch, int64_t m, int64_t n, int t)
{
    if (t != SPEC_BF16 && t != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (batch < 1 || batch > 65535 || m < 1 || n < 1 || m > 65536 || n > 65536 || (m > 32768 && n > 32768))
        return SPEC_EINVAL;
    return SPEC_OK;
}

// a microscaled matrix of `rows` x `cols` (the sizes are checked)
int check_mx(const spec_mx *m, int64_t rows, int64_t cols)
{
    if (m == nullptr) return SPEC_EINVAL;
    if (m->fmt != SPEC_MX_INT8 && m->fmt != SPEC_MX_FP4) return SPEC_EUNSUPPORTED;
    const int64_t blocks = (cols + 31) / 32;
    if (m->ldq < blocks * (m->fmt == SPEC_MX_INT8 ? 32 : 16) || m->lds < (blocks + 15) / 16 * 16) return SPEC_EINVAL;
    if (m->ldq > ((int64_t)1 << 22) || m->lds > ((int64_t)1 << 22)) return SPEC_EINVAL;
    if (m->ldq % 16 != 0 || m->lds % 16 != 0 || !aligned(m->q, 16) || !aligned(m->s, 16)) return SPEC_EINVAL;
    return rows > 0 && (m->q == nullptr || m->s == nullptr) ? SPEC_EINVAL : SPEC_OK;
}

int check_mx_matrix(const spec_mx *m, const void *X, int t, int64_t rows, int64_t cols, int64_t ldx)
{
    if (t != SPEC_BF16 && t != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (rows < 0 || rows >= (int64_t)1 << 31 || cols < 1 || cols > ((int64_t)1 << 20)) return SPEC_EINVAL;
    if ((X == nullptr && rows > 0) || ldx < cols || !aligned(X, elt_size(t))) return SPEC_EINVAL;
    return check_mx(m, rows, cols);
}

int check_mx_sizes(int64_t T, int64_t N, int64_t K, int t)
{
    if (t != SPEC_BF16 && t != SPEC_F32) return SPEC_EUNSUPPORTED;
    const int64_t lim = (int64_t)1 << 20;
    return T < 0 || T > 4 * lim || N < 1 || N > lim || K < 1 || K > lim ? SPEC_EINVAL : SPEC_OK;
}

// a checkpoint of the norms: absent, or INT8
int check_stored(const spec_mx *m, int64_t n, int64_t d)
{
    if (m == nullptr) return SPEC_OK;
    const int st = check_mx(m, n, d);
    return st == SPEC_OK && m->fmt != SPEC_MX_INT8 ? SPEC_EUNSUPPORTED : st;
}

int check_block(const spec_block *b)
{
    if (b == nullptr) return SPEC_EINVAL;
    if (b->t != SPEC_BF16 && b->t != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (b->n < 0 || b->n >= (int64_t)1 << 31 || b->d < 1 || b->d > BLOCK_MAX_D) return SPEC_EINVAL;
    if (!finite32(b->alpha) || !finite32(b->beta) || !(b->eps >= FLT_MIN) || !finite32(b->eps)) return SPEC_EINVAL;
    const size_t es = elt_size(b->t);
    if (!aligned(b->w_post, es) || !aligned(b->w_pre, es) || !aligned(b->gate, es)) return SPEC_EINVAL;
    if (b->post == 0 && b->w_post != nullptr) return SPEC_EINVAL;
    if (b->gate != nullptr && (b->gate_rows < 1 || (b->gate_rows < b->n && b->ldg < b->d))) return SPEC_EINVAL;
    return SPEC_OK;
}

// a matrix of the norms that is given (or has to be)
bool block_matrix(const spec_block *b, const void *p, int64_t ld, bool needed = false)
{
    if (p == nullptr) return !needed;
    return ld >= b->d && aligned(p, elt_size(b->t));
}

}  // namespace

extern "C" {

const char *spec_strerror(int status)
{
    switch (status) {
    case SPEC_OK: return "success";
    case SPEC_EINVAL: return "invalid argument (pointer, size, stride or parameter)";
    case SPEC_EUNSUPPORTED: return "unsupported dtype combination or size";
    case SPEC_EWORKSPACE: return "workspace missing or too small";
    case SPEC_EHIP: return "HIP runtime error while enqueueing a kernel";
    default: return "unknown status";
    }
}

const char *spec_version(void) { return "0.1.0"; }

int spec_cov_accumulate(void *stream, const void *X, int xt, int64_t n, int64_t d, int64_t ldx, void *C, int ct,
                        int64_t ldc, double alpha, double beta)
{
    if (C == nullptr || (X == nullptr && n > 0)) return SPEC_EINVAL;
    if (n < 0 || d < 1 || ldc < d || (n > 0 && ldx < d)) return SPEC_EINVAL;
    if (!isfinite(alpha) || !isfinite(beta)) return SPEC_EINVAL;
    const bool pair_ok = (xt == SPEC_BF16 && ct == SPEC_F32) || (xt == SPEC_F32 && ct == SPEC_F32) ||
                         (xt == SPEC_F32 && ct == SPEC_F64);
    if (!pair_ok) return SPEC_EUNSUPPORTED;
    if (!aligned(C, elt_size(ct)) || (X != nullptr && !aligned(X, elt_size(xt)))) return SPEC_EINVAL;
    if (d > (int64_t)1 << 20 || n > ((int64_t)1 << 40)) return SPEC_EUNSUPPORTED;
    KTimer kt((hipStream_t)stream, SPEC_KT_SYRK);
    return from_hip(launch_syrk((hipStream_t)stream, X, xt, n, d, ldx, C, ct, ldc, alpha, beta));
}

int spec_gram_window(void *stream, const void *H, int ht, int64_t streams, int64_t T, int64_t d, int64_t ld_t,
                     int64_t ld_s, int N, int stride, double scale, int layout, float *out)
{
    if (H == nullptr || out == nullptr) return SPEC_EINVAL;
    if (ht != SPEC_BF16 && ht != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (streams < 1 || T < 1 || d < 1 || N < 1 || N > 64 || N > T || stride < 1) return SPEC_EINVAL;
    if (ld_t < d || ld_s < T * ld_t) return SPEC_EINVAL;
    if (!aligned(H, elt_size(ht)) || !aligned(out, 4)) return SPEC_EINVAL;
    if (!isfinite(scale)) return SPEC_EINVAL;
    KTimer kt((hipStream_t)stream, SPEC_KT_GRAM);
    if (layout == SPEC_GRAM_BAND)
        return from_hip(launch_gram_band((hipStream_t)stream, H, ht, streams, T, d, ld_t, ld_s, N, out));
    if (layout == SPEC_GRAM_DENSE) {
        if (streams * ((T - N) / stride + 1) > ((int64_t)1 << 31) - 1) return SPEC_EUNSUPPORTED;
        return from_hip(
            launch_gram_dense((hipStream_t)stream, H, ht, streams, T, d, ld_t, ld_s, N, stride, (float)scale, out));
    }
    return SPEC_EINVAL;
}

// the batch source of the small solvers: its kind, strides and batch count
static int check_batch_src(const spec_batch_src *src, int64_t batch, int n)
{
    if (src == nullptr || src->a == nullptr) return SPEC_EINVAL;
    if (batch < 0 || batch > ((int64_t)1 << 31) - 1) return SPEC_EINVAL;
    if (!aligned(src->a, 4)) return SPEC_EINVAL;
    if (src->kind == SPEC_SRC_DENSE) {
        if (src->lda < n || src->stride_a < (int64_t)n * src->lda) return SPEC_EINVAL;
    } else if (src->kind == SPEC_SRC_BAND) {
        if (src->streams < 1 || src->T < n || src->stride < 1 || !isfinite(src->scale)) return SPEC_EINVAL;
        const int64_t W = (src->T - n) / src->stride + 1;
        if (batch != src->streams * W) return SPEC_EINVAL;
    } else {
        return SPEC_EINVAL;
    }
    return SPEC_OK;
}

int spec_eigvalsh_batched(void *stream, const spec_batch_src *src, int64_t batch, int n, float *w, int32_t *info)
{
    if (src == nullptr || w == nullptr || src->a == nullptr) return SPEC_EINVAL;
    if (n < 1 || n > 64) return n > 64 ? SPEC_EUNSUPPORTED : SPEC_EINVAL;
    if (!aligned(w, 4) || (info != nullptr && !aligned(info, 4))) return SPEC_EINVAL;
    const int st = check_batch_src(src, batch, n);
    if (st != SPEC_OK) return st;
    KTimer kt((hipStream_t)stream, SPEC_KT_SMALL_EIG);
    return from_hip(launch_eigvalsh_batched((hipStream_t)stream, src, batch, n, w, info));
}

int spec_eigh_batched(void *stream, const spec_batch_src *src, int64_t batch, int n, float *w, float *V,
                      int32_t *info)
{
    if (src == nullptr || w == nullptr || V == nullptr || src->a == nullptr) return SPEC_EINVAL;
    if (n < 1 || n > 32) return n > 32 ? SPEC_EUNSUPPORTED : SPEC_EINVAL;
    if (!aligned(w, 4) || !aligned(V, 4) || (info != nullptr && !aligned(info, 4))) return SPEC_EINVAL;
    const int st = check_batch_src(src, batch, n);
    if (st != SPEC_OK) return st;
    return from_hip(launch_eigh_batched((hipStream_t)stream, src, batch, n, w, V, info));
}

int spec_eigvalsh_sliding(void *stream, const spec_batch_src *src, int64_t batch, int n, int restart, float *w,
                          int32_t *info)
{
    if (src == nullptr || w == nullptr || src->a == nullptr || src->kind != SPEC_SRC_BAND) return SPEC_EINVAL;
    if (n < 1 || n > 64) return n > 64 ? SPEC_EUNSUPPORTED : SPEC_EINVAL;
    if (batch < 0 || batch > ((int64_t)1 << 31) - 1 || restart < 1) return SPEC_EINVAL;
    if (!aligned(w, 4) || !aligned(src->a, 4) || (info != nullptr && !aligned(info, 4))) return SPEC_EINVAL;
    if (src->streams < 1 || src->T < n || src->stride < 1 || !isfinite(src->scale)) return SPEC_EINVAL;
    const int64_t W = (src->T - n) / src->stride + 1;
    if (batch != src->streams * W) return SPEC_EINVAL;
    return from_hip(launch_eigvalsh_sliding((hipStream_t)stream, src, n, restart, w, info));
}

int spec_eigvalsh_batched_desc(void *stream, const spec_batch_src *src, int64_t batch, int n, float *w, int32_t *info,
                               const spec_desc_params *p, spec_desc *out, void *ws, size_t ws_bytes)
{
    if (src == nullptr || src->a == nullptr || out == nullptr) return SPEC_EINVAL;
    if (n < 2 || n > 32) return n > 32 ? SPEC_EUNSUPPORTED : SPEC_EINVAL;
    if (batch < 0 || batch > ((int64_t)1 << 31) - 1) return SPEC_EINVAL;
    const int st = check_desc_params(n, p);
    if (st != SPEC_OK) return st;
    if ((w != nullptr && !aligned(w, 4)) || !aligned(src->a, 4) || (info != nullptr && !aligned(info, 4)) ||
        !aligned(out, 8))
        return SPEC_EINVAL;
    if (src->kind == SPEC_SRC_DENSE) {
        if (src->lda < n || src->stride_a < (int64_t)n * src->lda) return SPEC_EINVAL;
    } else if (src->kind == SPEC_SRC_BAND) {
        if (src->streams < 1 || src->T < n || src->stride < 1 || !isfinite(src->scale)) return SPEC_EINVAL;
        const int64_t W = (src->T - n) / src->stride + 1;
        if (batch != src->streams * W) return SPEC_EINVAL;
    } else {
        return SPEC_EINVAL;
    }
    if (ws == nullptr || ws_bytes < descriptors_workspace_bytes(n)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    KTimer kt((hipStream_t)stream, SPEC_KT_SMALL_EIG);
    return from_hip(launch_eigvalsh_batched_desc((hipStream_t)stream, src, batch, n, w, info, p, out, ws));
}

int spec_eigvalsh_large_workspace(int64_t n, int t, size_t *bytes)
{
    if (bytes == nullptr || n < 1) return SPEC_EINVAL;
    if (t != SPEC_F32 && t != SPEC_F64) return SPEC_EUNSUPPORTED;
    if ((t == SPEC_F32 && n > 32768) || (t == SPEC_F64 && n > 8192)) return SPEC_EUNSUPPORTED;
    *bytes = eig_large_workspace_bytes(n, t);
    return SPEC_OK;
}

int spec_eigvalsh_large(void *stream, void *A, int t, int64_t n, int64_t lda, void *w, void *ws, size_t ws_bytes,
                        int32_t *info)
{
    size_t need = 0;
    int st = spec_eigvalsh_large_workspace(n, t, &need);
    if (st != SPEC_OK) return st;
    if (A == nullptr || w == nullptr || lda < n || lda >= ((int64_t)1 << 22)) return SPEC_EINVAL;
    if (!aligned(A, 16) || !aligned(w, elt_size(t)) || (info != nullptr && !aligned(info, 4))) return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < need) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_eig_large((hipStream_t)stream, A, t, n, lda, w, ws, info));
}

int spec_eigh_large_workspace(int64_t n, int t, int64_t k, size_t *bytes)
{
    if (bytes == nullptr || n < 1 || k < 1 || k > n) return SPEC_EINVAL;
    if (t != SPEC_F32 && t != SPEC_F64) return SPEC_EUNSUPPORTED;
    if (n > EIGVEC_MAX_N) return SPEC_EUNSUPPORTED;
    *bytes = eigh_large_workspace_bytes(n, t, k);
    return SPEC_OK;
}

int spec_eigh_large(void *stream, void *A, int t, int64_t n, int64_t lda, void *w, void *Z, int64_t ldz, int64_t k,
                    void *ws, size_t ws_bytes, int32_t *info)
{
    size_t need = 0;
    int st = spec_eigh_large_workspace(n, t, k, &need);
    if (st != SPEC_OK) return st;
    if (A == nullptr || w == nullptr || Z == nullptr || lda < n || lda >= ((int64_t)1 << 22) || ldz < k)
        return SPEC_EINVAL;
    if (!aligned(A, 16) || !aligned(w, elt_size(t)) || !aligned(Z, elt_size(t)) ||
        (info != nullptr && !aligned(info, 4)))
        return SPEC_EINVAL;
    // Z is addressed with 32-bit byte offsets (rows up to n + 128 reached)
    if ((n + 128) * ldz * (int64_t)elt_size(t) >= ((int64_t)1 << 31)) return SPEC_EUNSUPPORTED;
    if (ws == nullptr || ws_bytes < need) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_eigh_large((hipStream_t)stream, A, t, n, lda, w, Z, ldz, k, ws, info));
}

int spec_descriptors_workspace(int64_t r, size_t *bytes)
{
    if (bytes == nullptr || r < 1) return SPEC_EINVAL;
    *bytes = descriptors_workspace_bytes(r);
    return SPEC_OK;
}

int spec_descriptors_static(void *stream, const void *w, int wt, int64_t batch, int64_t r, int64_t ldw,
                            const spec_desc_params *p, spec_desc *out)
{
    const int st = check_descriptors(w, wt, batch, r, ldw, p, out);
    if (st != SPEC_OK) return st;
    if (r > DESC_SCRATCH_MAX_R) return SPEC_EUNSUPPORTED;
    return from_hip(launch_descriptors_static((hipStream_t)stream, w, wt, batch, r, ldw, p, out));
}

int spec_descriptors(void *stream, const void *w, int wt, int64_t batch, int64_t r, int64_t ldw,
                     const spec_desc_params *p, spec_desc *out, void *ws, size_t ws_bytes)
{
    const int st = check_descriptors(w, wt, batch, r, ldw, p, out);
    if (st != SPEC_OK) return st;
    if (ws == nullptr || ws_bytes < descriptors_workspace_bytes(r)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_descriptors((hipStream_t)stream, w, wt, batch, r, ldw, p, out, ws));
}

int spec_eigvalsh_topk(void *stream, const void *A, int t, int64_t n, int64_t lda, const void *Omega, int q, void *w,
                       void *ws, size_t ws_bytes)
{
    if (t != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (A == nullptr || Omega == nullptr || w == nullptr) return SPEC_EINVAL;
    if (n < 64 || n > 32768 || lda < n || lda >= ((int64_t)1 << 22) || q < 0 || q > 16) return SPEC_EINVAL;
    if (!aligned(A, 16) || !aligned(Omega, 16) || !aligned(w, 4)) return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < eig_large_workspace_bytes(n, SPEC_F32)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_topk_ritz((hipStream_t)stream, (const float *)A, n, lda, (const float *)Omega, q,
                                     (float *)w, nullptr, 0, ws, nullptr));
}

int spec_eigvecs_topk(void *stream, const void *A, int t, int64_t n, int64_t lda, const void *Omega, int q, void *w,
                      void *P, int64_t ldp, void *ws, size_t ws_bytes, int32_t *info)
{
    if (t != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (A == nullptr || Omega == nullptr || w == nullptr || P == nullptr) return SPEC_EINVAL;
    if (n < 64 || n > 32768 || lda < n || lda >= ((int64_t)1 << 22) || q < 0 || q > 16) return SPEC_EINVAL;
    if (ldp < 32 || ldp >= ((int64_t)1 << 22)) return SPEC_EINVAL;
    if (!aligned(A, 16) || !aligned(Omega, 16) || !aligned(w, 4) || !aligned(P, 4)) return SPEC_EINVAL;
    if (info != nullptr && !aligned(info, 4)) return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < eig_large_workspace_bytes(n, SPEC_F32)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_topk_ritz((hipStream_t)stream, (const float *)A, n, lda, (const float *)Omega, q,
                                     (float *)w, (float *)P, ldp, ws, info));
}

int spec_desc_smooth(void *stream, const spec_desc *in, int64_t streams, int64_t W, double alpha, spec_desc *out)
{
    if (in == nullptr || out == nullptr || streams < 0 || streams > ((int64_t)1 << 31) - 1 || W < 1) return SPEC_EINVAL;
    if (!(alpha > 0.0 && alpha <= 1.0)) return SPEC_EINVAL;
    if (!aligned(in, 8) || !aligned(out, 8)) return SPEC_EINVAL;
    const char *a = (const char *)in, *b = (const char *)out;
    const size_t bytes = (size_t)streams * (size_t)W * sizeof(spec_desc);
    if (a < b + bytes && b < a + bytes) return SPEC_EINVAL;  // overlapping
    return from_hip(launch_desc_smooth((hipStream_t)stream, in, streams, W, alpha, out));
}

int spec_spectrum_robust(void *stream, const void *w, int wt, int64_t batch, int64_t r, int64_t ldw,
                         const spec_robust_params *p, spec_robust *out)
{
    if (w == nullptr || p == nullptr || out == nullptr) return SPEC_EINVAL;
    if (wt != SPEC_F32 && wt != SPEC_F64) return SPEC_EUNSUPPORTED;
    if (batch < 0 || batch > ((int64_t)1 << 31) - 1 || r < 2 || ldw < r) return SPEC_EINVAL;
    if (p->bins < 1 || p->bins > 64 || p->n_samples < 1 || p->p_dim < 1) return SPEC_EINVAL;
    if (!(p->winsor_frac >= 0.0 && p->winsor_frac <= 0.5) || !(p->mad_k > 0.0 && isfinite(p->mad_k)))
        return SPEC_EINVAL;
    if (p->sigma2_mode < SPEC_SIGMA2_GIVEN || p->sigma2_mode > SPEC_SIGMA2_WINSOR) return SPEC_EINVAL;
    if (p->sigma2_mode == SPEC_SIGMA2_GIVEN && !(p->sigma2 > 0.0 && isfinite(p->sigma2))) return SPEC_EINVAL;
    if (!aligned(w, elt_size(wt)) || !aligned(out, 8)) return SPEC_EINVAL;
    return from_hip(launch_spectrum_robust((hipStream_t)stream, w, wt, batch, r, ldw, p, out));
}

int spec_project_weight_workspace(int64_t d, size_t *bytes)
{
    if (bytes == nullptr || d < 1 || d > 65536) return SPEC_EINVAL;
    *bytes = project_weight_workspace_bytes(d);
    return SPEC_OK;
}

int spec_project_weight(void *stream, const void *W, int wt, int64_t d, int64_t ldw, const void *P, int64_t ldp, int k,
                        void *Wp, int64_t ldo, void *X, int64_t ldx, void *ws, size_t ws_bytes)
{
    if (wt != SPEC_BF16 && wt != SPEC_F32) return SPEC_EUNSUPPORTED;
    if (W == nullptr || P == nullptr || Wp == nullptr) return SPEC_EINVAL;
    if (d < 1 || d > 65536 || k < 1 || k > 32 || k > d) return SPEC_EINVAL;
    if (ldw < d || ldp < k || ldo < k || (X != nullptr && ldx < k)) return SPEC_EINVAL;
    const int64_t vec = wt == SPEC_BF16 ? 8 : 4;  // 16-byte rows
    if (!aligned(W, 16) || ldw % vec != 0) return SPEC_EINVAL;
    if (!aligned(P, 4) || !aligned(Wp, 4) || (X != nullptr && !aligned(X, 4))) return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < project_weight_workspace_bytes(d)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_project_weight((hipStream_t)stream, W, wt, d, ldw, (const float *)P, ldp, k, (float *)Wp,
                                          ldo, (float *)X, ldx, ws));
}

int spec_tail_pair_screen(void *stream, const void *U, const void *V, int dt, int64_t n, int64_t ldu, int64_t ldv,
                          int64_t i0, int64_t t, int64_t head_dim, double eps, double *absdot, int64_t ldo,
                          uint8_t *keep, int64_t ldk, int64_t *count)
{
    if (dt != SPEC_F32 && dt != SPEC_F64) return SPEC_EUNSUPPORTED;
    if (U == nullptr || V == nullptr || keep == nullptr) return SPEC_EINVAL;
    if (n < 1 || i0 < 0 || t < 1 || t > 65535 || head_dim < 1 || !(eps > 0.0 && isfinite(eps))) return SPEC_EINVAL;
    if (i0 + t > ldu || i0 + t > ldv || ldk < t || (absdot != nullptr && ldo < t)) return SPEC_EINVAL;
    if (!aligned(U, elt_size(dt)) || !aligned(V, elt_size(dt))) return SPEC_EINVAL;
    if ((absdot != nullptr && !aligned(absdot, 8)) || (count != nullptr && !aligned(count, 8))) return SPEC_EINVAL;
    return from_hip(launch_tail_pair_screen((hipStream_t)stream, U, V, dt, n, ldu, ldv, i0, t, head_dim, eps, absdot,
                                            ldo, keep, ldk, count));
}

int spec_embed(void *stream, const void *E, int t, int64_t V, int64_t d, int64_t lde, const void *ids, int idt,
               int64_t n, double scale, void *Y, int64_t ldy)
{
    if (t != SPEC_BF16 && t != SPEC_F32) return SPEC_EUNSUPPORTED;
    int st = check_rows(n, V, d);
    if (st != SPEC_OK) return st;
    st = check_ids(ids, idt, n);
    if (st != SPEC_OK) return st;
    if (E == nullptr || (Y == nullptr && n > 0) || lde < d || ldy < d || !finite32(scale)) return SPEC_EINVAL;
    if (!aligned(E, elt_size(t)) || !aligned(Y, elt_size(t))) return SPEC_EINVAL;
    return from_hip(launch_embed((hipStream_t)stream, E, t, V, d, lde, ids, idt == SPEC_I64, n, (float)scale, Y, ldy));
}

int spec_embed_grad_workspace(int64_t n, int64_t V, int64_t d, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_rows(n, V, d);
    if (st != SPEC_OK) return st;
    *bytes = embed_grad_workspace_bytes(n, V, d);
    return SPEC_OK;
}

int spec_embed_grad(void *stream, const void *dY, int yt, int64_t n, int64_t V, int64_t d, int64_t ldy, const void *ids,
                    int idt, double scale, double beta, void *dE, int et, int64_t ldd, void *ws, size_t ws_bytes)
{
    const bool pair_ok = (yt == SPEC_BF16 && (et == SPEC_BF16 || et == SPEC_F32)) || (yt == SPEC_F32 && et == SPEC_F32);
    if (!pair_ok) return SPEC_EUNSUPPORTED;
    int st = check_rows(n, V, d);
    if (st != SPEC_OK) return st;
    st = check_ids(ids, idt, n);
    if (st != SPEC_OK) return st;
    if (dE == nullptr || (dY == nullptr && n > 0) || ldy < d || ldd < d || !finite32(scale)) return SPEC_EINVAL;
    if (!aligned(dY, elt_size(yt)) || !aligned(dE, elt_size(et))) return SPEC_EINVAL;
    if (beta != 0.0 && beta != 1.0) return isfinite(beta) ? SPEC_EUNSUPPORTED : SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < embed_grad_workspace_bytes(n, V, d)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_embed_grad((hipStream_t)stream, dY, yt, n, V, d, ldy, ids, idt == SPEC_I64, (float)scale,
                                      beta == 1.0, dE, et, ldd, ws));
}

int spec_linear_xent_workspace(int64_t T, int64_t V, int64_t d, int t, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_xent_sizes(T, V, d, t);
    if (st != SPEC_OK) return st;
    *bytes = linear_xent_workspace_bytes(T, V, d, t);
    return SPEC_OK;
}

// what both directions of the cross entropy ask of H, W and the targets
static int check_xent(const void *H, const void *W, int t, int64_t T, int64_t V, int64_t d, int64_t ldh, int64_t ldw,
                      const void *target, int tt, double scale)
{
    int st = check_xent_sizes(T, V, d, t);
    if (st != SPEC_OK) return st;
    st = check_ids(target, tt, T);
    if (st != SPEC_OK) return st;
    const int64_t most = ((int64_t)1 << 20) + 64;
    if (W == nullptr || (H == nullptr && T > 0) || ldh < d || ldw < d || ldh > most || ldw > most || !finite32(scale))
        return SPEC_EINVAL;
    if (!aligned(H, elt_size(t)) || !aligned(W, elt_size(t))) return SPEC_EINVAL;
    return SPEC_OK;
}

int spec_linear_xent(void *stream, const void *H, const void *W, int t, int64_t T, int64_t V, int64_t d, int64_t ldh,
                     int64_t ldw, const void *target, int tt, double scale, float *loss, float *lse, void *ws,
                     size_t ws_bytes)
{
    const int st = check_xent(H, W, t, T, V, d, ldh, ldw, target, tt, scale);
    if (st != SPEC_OK) return st;
    if (T > 0 && (loss == nullptr || lse == nullptr)) return SPEC_EINVAL;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < linear_xent_workspace_bytes(T, V, d, t)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_linear_xent((hipStream_t)stream, H, W, t, T, V, d, ldh, ldw, target, tt == SPEC_I64,
                                       (float)scale, loss, lse, ws));
}

int spec_linear_xent_grad_workspace(int64_t T, int64_t V, int64_t d, int t, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_xent_sizes(T, V, d, t);
    if (st != SPEC_OK) return st;
    *bytes = linear_xent_grad_workspace_bytes(T, V, d, t);
    return SPEC_OK;
}

int spec_linear_xent_grad(void *stream, const void *H, const void *W, int t, int64_t T, int64_t V, int64_t d,
                          int64_t ldh, int64_t ldw, const void *target, int tt, double scale, const float *lse,
                          const float *dloss, double beta, void *dH, int64_t lddh, void *dW, int64_t lddw, void *ws,
                          size_t ws_bytes)
{
    const int st = check_xent(H, W, t, T, V, d, ldh, ldw, target, tt, scale);
    if (st != SPEC_OK) return st;
    if (T > 0 && (lse == nullptr || dloss == nullptr || dH == nullptr)) return SPEC_EINVAL;
    if (dW == nullptr || lddh < d || lddw < d || !finite32(beta)) return SPEC_EINVAL;
    if (!aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dH, elt_size(t)) || !aligned(dW, elt_size(t)))
        return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < linear_xent_grad_workspace_bytes(T, V, d, t)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_linear_xent_grad((hipStream_t)stream, H, W, t, T, V, d, ldh, ldw, target, tt == SPEC_I64,
                                            (float)scale, lse, dloss, dH, lddh, dW, lddw, (float)beta, ws));
}

int spec_orthogonalize_workspace(int64_t batch, int64_t m, int64_t n, int t, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_ortho_sizes(batch, m, n, t);
    if (st != SPEC_OK) return st;
    *bytes = orthogonalize_workspace_bytes(batch, m, n, t);
    return SPEC_OK;
}

int spec_orthogonalize(void *stream, const void *G, int t, int64_t batch, int64_t m, int64_t n, int64_t ldg, int64_t sg,
                       const double *coeffs, int steps, double eps, double scale, void *O, int64_t ldo, int64_t so,
                       void *ws, size_t ws_bytes)
{
    const int st = check_ortho_sizes(batch, m, n, t);
    if (st != SPEC_OK) return st;
    if (G == nullptr || O == nullptr || coeffs == nullptr || ldg < n || ldo < n) return SPEC_EINVAL;
    if (batch > 1 && (sg / m < ldg || so / m < ldo)) return SPEC_EINVAL;  // (m * ldg may not be an int64)
    if (steps < 1 || steps > 32 || !(eps >= 0.0) || !isfinite(eps) || !finite32(scale)) return SPEC_EINVAL;
    for (int i = 0; i < 3 * steps; ++i)
        if (!finite32(coeffs[i])) return SPEC_EINVAL;
    if (t == SPEC_BF16 && !orthogonalize_bounded(coeffs, steps)) return SPEC_EINVAL;
    if (!aligned(G, elt_size(t)) || !aligned(O, elt_size(t))) return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < orthogonalize_workspace_bytes(batch, m, n, t)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_orthogonalize((hipStream_t)stream, G, t, batch, m, n, ldg, sg, coeffs, steps, eps, scale, O,
                                         ldo, so, ws));
}

int spec_mx_row_bytes(int fmt, int64_t cols, int64_t *codes, int64_t *scales)
{
    if (fmt != SPEC_MX_INT8 && fmt != SPEC_MX_FP4) return SPEC_EUNSUPPORTED;
    if (codes == nullptr || scales == nullptr || cols < 1 || cols > ((int64_t)1 << 20)) return SPEC_EINVAL;
    const int64_t blocks = (cols + 31) / 32;
    *codes = blocks * (fmt == SPEC_MX_INT8 ? 32 : 16);
    *scales = (blocks + 15) / 16 * 16;
    return SPEC_OK;
}

int spec_mx_quantize(void *stream, const void *X, int t, int64_t rows, int64_t cols, int64_t ldx, const spec_mx *out)
{
    const int st = check_mx_matrix(out, X, t, rows, cols, ldx);
    if (st != SPEC_OK) return st;
    return from_hip(launch_mx_quantize((hipStream_t)stream, X, t, rows, cols, ldx, out));
}

int spec_mx_dequantize(void *stream, const spec_mx *in, int64_t rows, int64_t cols, void *X, int t, int64_t ldx)
{
    const int st = check_mx_matrix(in, X, t, rows, cols, ldx);
    if (st != SPEC_OK) return st;
    return from_hip(launch_mx_dequantize((hipStream_t)stream, in, rows, cols, cols, X, t, ldx));
}

int spec_mx_plan(int op, int64_t T, int64_t N, int64_t K, int t, int *edge, int *shares)
{
    if (op != SPEC_MX_OP_LINEAR && op != SPEC_MX_OP_PRODUCT && op != SPEC_MX_OP_WEIGHT_GRAD) return SPEC_EUNSUPPORTED;
    if (edge == nullptr || shares == nullptr) return SPEC_EINVAL;
    const int st = check_mx_sizes(T, N, K, t);
    if (st != SPEC_OK) return st;
    mx_plan(op, T, N, K, t, edge, shares);
    return SPEC_OK;
}

int spec_mx_linear_workspace(int64_t T, int64_t N, int64_t K, int t, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_mx_sizes(T, N, K, t);
    if (st != SPEC_OK) return st;
    *bytes = mx_linear_workspace_bytes(T, N, K, t);
    return SPEC_OK;
}

int spec_mx_linear(void *stream, const void *X, int t, int64_t T, int64_t N, int64_t K, int64_t ldx, const spec_mx *W,
                   void *Y, int64_t ldy, void *ws, size_t ws_bytes)
{
    int st = check_mx_sizes(T, N, K, t);
    if (st != SPEC_OK) return st;
    if (T > 0 && (X == nullptr || Y == nullptr)) return SPEC_EINVAL;
    if (ldx < K || ldx > ((int64_t)1 << 20) + 64 || ldy < N) return SPEC_EINVAL;
    if (!aligned(X, elt_size(t)) || !aligned(Y, elt_size(t))) return SPEC_EINVAL;
    st = check_mx(W, N, K);
    if (st != SPEC_OK) return st;
    if (W->fmt != SPEC_MX_FP4) return SPEC_EUNSUPPORTED;
    if (ws == nullptr || ws_bytes < mx_linear_workspace_bytes(T, N, K, t)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_mx_linear((hipStream_t)stream, X, t, T, N, K, ldx, W, Y, ldy, ws));
}

int spec_mx_product_workspace(int64_t T, int64_t N, int64_t K, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_mx_sizes(T, N, K, SPEC_BF16);
    if (st != SPEC_OK) return st;
    *bytes = mx_product_workspace_bytes(T, N, K);
    return SPEC_OK;
}

int spec_mx_product(void *stream, const spec_mx *X, const spec_mx *W, int64_t T, int64_t N, int64_t K, void *Y, int yt,
                    int64_t ldy, void *ws, size_t ws_bytes)
{
    int st = check_mx_sizes(T, N, K, yt);
    if (st != SPEC_OK) return st;
    if ((Y == nullptr && T > 0) || ldy < N || !aligned(Y, elt_size(yt))) return SPEC_EINVAL;
    st = check_mx(X, T, K);
    if (st != SPEC_OK) return st;
    st = check_mx(W, N, K);
    if (st != SPEC_OK) return st;
    if (X->fmt != SPEC_MX_FP4 || W->fmt != SPEC_MX_FP4) return SPEC_EUNSUPPORTED;
    if (ws == nullptr || ws_bytes < mx_product_workspace_bytes(T, N, K)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_mx_product((hipStream_t)stream, X, W, T, N, K, Y, yt, ldy, ws));
}

int spec_mx_weight_grad_workspace(int64_t T, int64_t N, int64_t K, int t, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_mx_sizes(T, N, K, t);
    if (st != SPEC_OK) return st;
    *bytes = mx_weight_grad_workspace_bytes(T, N, K, t);
    return SPEC_OK;
}

int spec_mx_weight_grad(void *stream, const void *dY, int t, int64_t T, int64_t N, int64_t K, int64_t ldy,
                        const spec_mx *X, double beta, void *dW, int64_t lddw, void *ws, size_t ws_bytes)
{
    int st = check_mx_sizes(T, N, K, t);
    if (st != SPEC_OK) return st;
    if (dW == nullptr || (dY == nullptr && T > 0) || ldy < N || ldy > ((int64_t)1 << 20) + 64 || lddw < K)
        return SPEC_EINVAL;
    if (!aligned(dY, elt_size(t)) || !aligned(dW, elt_size(t)) || !finite32(beta)) return SPEC_EINVAL;
    st = check_mx(X, T, K);
    if (st != SPEC_OK) return st;
    if (X->fmt != SPEC_MX_INT8) return SPEC_EUNSUPPORTED;
    if (ws == nullptr || ws_bytes < mx_weight_grad_workspace_bytes(T, N, K, t)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_mx_weight_grad((hipStream_t)stream, dY, t, T, N, K, ldy, X, (float)beta, dW, lddw, ws));
}

int spec_block_norm(void *stream, const spec_block *b, const void *Y, int64_t ldy, const void *H, int64_t ldh,
                    void *Hout, int64_t ldo, void *X, int64_t ldx, float *r_post, float *r_pre, const spec_mx *y8,
                    const spec_mx *h8, const spec_mx *x8)
{
    int st = check_block(b);
    if (st != SPEC_OK) return st;
    const bool some = b->n > 0;
    if (!block_matrix(b, H, ldh, some) || !block_matrix(b, Y, ldy) || !block_matrix(b, Hout, ldo) ||
        !block_matrix(b, X, ldx) || !aligned(r_post, 4) || !aligned(r_pre, 4))
        return SPEC_EINVAL;
    if (some && Y == nullptr && (Hout != nullptr || r_post != nullptr || y8 != nullptr || h8 != nullptr)) return SPEC_EINVAL;
    if (r_post != nullptr && b->post == 0) return SPEC_EINVAL;
    for (const spec_mx *m : {y8, h8, x8}) {
        st = check_stored(m, b->n, b->d);
        if (st != SPEC_OK) return st;
    }
    return from_hip(launch_block_norm((hipStream_t)stream, b, Y, ldy, H, ldh, Hout, ldo, X, ldx, r_post, r_pre, y8, h8, x8));
}

int spec_block_norm_grad_workspace(const spec_block *b, size_t *bytes)
{
    if (bytes == nullptr) return SPEC_EINVAL;
    const int st = check_block(b);
    if (st != SPEC_OK) return st;
    *bytes = block_norm_grad_workspace_bytes(b);
    return SPEC_OK;
}

int spec_block_norm_grad(void *stream, const spec_block *b, const void *Y, int64_t ldy, const spec_mx *y8,
                         const void *Hout, int64_t ldo, const spec_mx *h8, const float *r_post, const float *r_pre,
                         const void *dHout, int64_t lddo, const void *dX, int64_t lddx, void *dH, int64_t lddh, void *dY,
                         int64_t lddy, float *dw_post, float *dw_pre, float *dgate, void *ws, size_t ws_bytes)
{
    int st = check_block(b);
    if (st != SPEC_OK) return st;
    const bool some = b->n > 0;
    if (!block_matrix(b, Y, ldy) || !block_matrix(b, Hout, ldo) || !block_matrix(b, dHout, lddo) ||
        !block_matrix(b, dX, lddx) || !block_matrix(b, dH, lddh) || !block_matrix(b, dY, lddy))
        return SPEC_EINVAL;
    st = check_stored(y8, b->n, b->d);
    if (st != SPEC_OK) return st;
    st = check_stored(h8, b->n, b->d);
    if (st != SPEC_OK) return st;
    const bool hasY = Y != nullptr || y8 != nullptr;
    if (some && !hasY && (dY != nullptr || dw_post != nullptr || dgate != nullptr)) return SPEC_EINVAL;
    if (some && dX != nullptr && ((Hout == nullptr && h8 == nullptr) || r_pre == nullptr)) return SPEC_EINVAL;
    if (some && dX == nullptr && (dw_pre != nullptr || dHout == nullptr)) return SPEC_EINVAL;
    if (some && hasY && b->post != 0 && r_post == nullptr) return SPEC_EINVAL;
    if ((b->post == 0 && dw_post != nullptr) || (b->gate == nullptr && dgate != nullptr)) return SPEC_EINVAL;
    for (const float *p : {r_post, r_pre, (const float *)dw_post, (const float *)dw_pre, (const float *)dgate})
        if (!aligned(p, 4)) return SPEC_EINVAL;
    if (ws == nullptr || ws_bytes < block_norm_grad_workspace_bytes(b)) return SPEC_EWORKSPACE;
    if (!aligned(ws, 256)) return SPEC_EINVAL;
    return from_hip(launch_block_norm_grad((hipStream_t)stream, b, Y, ldy, y8, Hout, ldo, h8, r_post, r_pre, dHout, lddo,
                                           dX, lddx, dH, lddh, dY, lddy, dw_post, dw_pre, dgate, ws));
}

}  // extern "C"
