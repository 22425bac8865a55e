// The C ABI of the paged-cache operators: argument checks, rotation constants
// and kernel dispatch.  Nothing here allocates device memory.
#include <climits>
#include <cmath>
#include <cstring>

#include "paged_internal.cuh"

namespace hga {

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

namespace {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
// held by the fp32 that the kernels take it in: 0, or a normal number there.  (An eps that
// became 0 would make a row of zeros NaN, a magnitude that did so a rotated part of 0.)
inline bool held32(double x) { return x == 0.0 || std::isnormal((float)x); }
inline size_t esize(int dtype) { return dtype == HGA_BF16 ? 2 : 4; }

hga_status check_pages(const hga_paged_dims *d) {
    if (!d || d->B < 1 || d->num_pages < 1 || d->page_size < 1 || d->max_pages < 1)
        return HGA_ERR_INVALID_ARG;
    if (d->page_size & (d->page_size - 1)) return HGA_ERR_UNSUPPORTED;
    if (d->B > 65535 || (long long)d->num_pages * d->page_size > INT_MAX ||
        (long long)d->max_pages * d->page_size > INT_MAX || (long long)d->B * d->max_pages > INT_MAX)
        return HGA_ERR_UNSUPPORTED;
    return HGA_OK;
}

hga_status check_heads(int Hq, int Hkv, int D, int dtype) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv) return HGA_ERR_INVALID_ARG;
    if (dtype != HGA_F32 && dtype != HGA_BF16) return HGA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return HGA_ERR_UNSUPPORTED;
    if (Hq > 65535) return HGA_ERR_UNSUPPORTED;
    return HGA_OK;
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Tokens of a call, whose rows the kernels number with 64 bits.
hga_status check_tokens(const hga_dims *d) {
    if (!d || d->B < 1 || d->T < 0) return HGA_ERR_INVALID_ARG;
    const hga_status s = check_heads(d->Hq, d->Hkv, d->D, d->dtype);
    if (s != HGA_OK) return s;
    return (long long)d->B * d->T > INT_MAX ? HGA_ERR_UNSUPPORTED : HGA_OK;
}

hga_status form_rope(const hga_rope *r, int D, PairRope *out) {
    std::memset(out, 0, sizeof(*out));
    out->magnitude = 1.f;
    if (r->layout != HGA_ROPE_HALF && r->layout != HGA_ROPE_INTERLEAVED) return HGA_ERR_INVALID_ARG;
    if (r->rotary_dim < 0 || r->rotary_dim > D) return HGA_ERR_INVALID_ARG;
    if (r->rotary_dim % 16) return HGA_ERR_UNSUPPORTED;
    out->interleaved = r->layout == HGA_ROPE_INTERLEAVED;
    const int R = out->R = r->rotary_dim;
    if (R == 0) return HGA_OK;
    if (!(r->theta > 1.0) || !std::isfinite(r->theta)) return HGA_ERR_INVALID_ARG;
    if (!held32(r->magnitude) || r->magnitude < 0.0) return HGA_ERR_INVALID_ARG;
    const bool yarn = r->scaling == HGA_ROPE_YARN;
    if (r->scaling != HGA_ROPE_UNSCALED && r->scaling != HGA_ROPE_LINEAR && !yarn)
        return HGA_ERR_INVALID_ARG;
    if (r->scaling != HGA_ROPE_UNSCALED && (!(r->factor >= 1.0) || !std::isfinite(r->factor)))
        return HGA_ERR_INVALID_ARG;
    double lo = 0.0, hi = 1.0, magnitude = 1.0;
    if (yarn) {
        if (r->original_len < 1 || !(r->beta_slow > 0.0) || !(r->beta_fast >= r->beta_slow) ||
            !std::isfinite(r->beta_fast))
            return HGA_ERR_INVALID_ARG;
        auto dim = [&](double turns) {
            return R * std::log(r->original_len / (2.0 * M_PI * turns)) / (2.0 * std::log(r->theta));
        };
        lo = std::fmax(std::floor(dim(r->beta_fast)), 0.0);
        hi = std::fmin(std::ceil(dim(r->beta_slow)), (double)(R - 1));
        // every pair on one side of the ramp (a trained length of a few tokens, or of more
        // turns than any pair has): the ramp would run backwards
        if (hi < lo) return HGA_ERR_INVALID_ARG;
        if (hi == lo) hi = lo + 0.001;
        magnitude = 0.1 * std::log(r->factor) + 1.0;
    }
    for (int i = 0; i < R / 2; ++i) {
        double w = std::pow(r->theta, -2.0 * i / R);
        if (r->scaling == HGA_ROPE_LINEAR) w /= r->factor;
        if (yarn) {
            const double g = std::fmin(1.0, std::fmax(0.0, (i - lo) / (hi - lo)));
            w = w * (1.0 - g) + w / r->factor * g;
        }
        // turns per position as a 64-bit fraction (extended precision on the host)
        const long double two_pi = 6.283185307179586476925286766559L;
        out->turn[i] = (unsigned long long)llroundl((long double)w / two_pi * 18446744073709551616.0L);
    }
    out->magnitude = (float)(r->magnitude > 0.0 ? r->magnitude : magnitude);
    return HGA_OK;
}

// The constants of a rotation, kept per thread for the one used last: R / 2 powers
// and extended-precision products take longer than a small step's kernel.
hga_status make_rope(const hga_rope *r, int D, PairRope *out) {
    thread_local hga_rope last;
    thread_local int last_D = 0;               // 0: nothing kept
    thread_local PairRope kept;
    if (!r) return HGA_ERR_INVALID_ARG;
    if (last_D != D || std::memcmp(&last, r, sizeof(last))) {
        last_D = 0;
        const hga_status s = form_rope(r, D, &kept);
        if (s != HGA_OK) return s;
        last = *r;
        last_D = D;
    }
    *out = kept;
    return HGA_OK;
}

// A strided [tokens, H, D] tensor: base and token stride on 16 bytes, tokens apart.
bool rows_ok(const void *p, int64_t stride, int H, int D, size_t e) {
    return p && aligned(p, 16) && stride >= (int64_t)H * D && stride * (int64_t)e % 16 == 0 &&
           stride <= (int64_t)1 << 40;
}

}  // namespace
}  // namespace hga

using namespace hga;

extern "C" {

size_t hga_paged_plan_workspace(int32_t B, int32_t n_slots) {
    return B < 1 || B > 65535 || n_slots < 0 ? 0 : plan_workspace_bytes(B, n_slots);
}

hga_status hga_paged_plan(const hga_paged_dims *dims, const hga_paged_plan_io *io, int32_t n_slots,
                          void *workspace, size_t workspace_bytes, void *stream) {
    const hga_status s = check_pages(dims);
    if (s != HGA_OK) return s;
    if (!io || n_slots < 0) return HGA_ERR_INVALID_ARG;
    const void *need[] = {io->lens, io->new_tokens, io->free_pages, io->free_count, io->block_table,
                          io->lens_out, io->free_count_out, io->cu_tokens, io->granted};
    for (const void *p : need)
        if (!p || !aligned(p, 4)) return HGA_ERR_INVALID_ARG;
    if (n_slots > 0 && (!io->slot || !io->pos)) return HGA_ERR_INVALID_ARG;
    if (!aligned(io->slot, 4) || !aligned(io->pos, 4) || !aligned(io->release, 4))
        return HGA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < plan_workspace_bytes(dims->B, n_slots) ||
        !aligned(workspace, 256))
        return HGA_ERR_WORKSPACE;
    PlanArgs a;
    a.B = dims->B;
    a.num_pages = dims->num_pages;
    a.log2_page = log2_of(dims->page_size);
    a.max_pages = dims->max_pages;
    a.n_slots = n_slots;
    a.io = *io;
    a.first = static_cast<int32_t *>(workspace);
    return launch_paged_plan(a, (cudaStream_t)stream);
}

hga_status hga_qk_norm_rope(const hga_dims *dims, const hga_rope *rope, const hga_qk_io *io,
                            void *stream) {
    hga_status s = check_tokens(dims);
    if (s != HGA_OK) return s;
    QkArgs a;
    s = make_rope(rope, dims->D, &a.rope);
    if (s != HGA_OK) return s;
    if (!io) return HGA_ERR_INVALID_ARG;
    if (dims->T == 0) return HGA_OK;
    const size_t e = esize(dims->dtype);
    const int D = dims->D;
    if (!(io->eps >= 0.0) || !held32(io->eps)) return HGA_ERR_INVALID_ARG;
    if (a.rope.R && (!io->pos || !aligned(io->pos, 4))) return HGA_ERR_INVALID_ARG;
    const bool wk = io->k_out || io->k_pages, wv = io->v_out || io->v_pages;
    if ((io->q_out && !rows_ok(io->q, io->q_stride, dims->Hq, D, e)) ||
        (wk && !rows_ok(io->k, io->k_stride, dims->Hkv, D, e)) ||
        (wv && !rows_ok(io->v, io->v_stride, dims->Hkv, D, e)))
        return HGA_ERR_INVALID_ARG;
    const void *rows[] = {io->q_out, io->k_out, io->v_out, io->k_pages, io->v_pages, io->q_weight,
                          io->k_weight};
    for (const void *p : rows)
        if (!aligned(p, 16)) return HGA_ERR_INVALID_ARG;
    if (io->k_pages || io->v_pages) {
        if (!io->slot || !aligned(io->slot, 4) || io->num_slots < 1) return HGA_ERR_INVALID_ARG;
        if (io->num_slots > INT_MAX) return HGA_ERR_UNSUPPORTED;
    }
    a.tokens = (int64_t)dims->B * dims->T;
    a.Hq = dims->Hq;
    a.Hkv = dims->Hkv;
    a.io = *io;
    if (!io->k_pages && !io->v_pages) a.io.slot = nullptr;
    return launch_qk_norm_rope(a, dims->dtype, D, (cudaStream_t)stream);
}

size_t hga_qk_norm_rope_backward_workspace(const hga_dims *dims) {
    return check_tokens(dims) == HGA_OK ? qk_grad_workspace_bytes(dims->D) : 0;
}

hga_status hga_qk_norm_rope_backward(const hga_dims *dims, const hga_rope *rope,
                                     const hga_qk_grad_io *io, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    hga_status s = check_tokens(dims);
    if (s != HGA_OK) return s;
    QkGradArgs a;
    s = make_rope(rope, dims->D, &a.rope);
    if (s != HGA_OK) return s;
    if (!io) return HGA_ERR_INVALID_ARG;
    const size_t e = esize(dims->dtype);
    const int D = dims->D;
    if (io->grad_dtype != HGA_F32 && io->grad_dtype != dims->dtype) return HGA_ERR_INVALID_ARG;
    if (!(io->eps >= 0.0) || !held32(io->eps)) return HGA_ERR_INVALID_ARG;
    if (!io->q_weight != !io->d_q_weight || !io->k_weight != !io->d_k_weight ||
        !io->d_v != !io->dv)
        return HGA_ERR_INVALID_ARG;
    if (!aligned(io->d_q_weight, 4) || !aligned(io->d_k_weight, 4)) return HGA_ERR_INVALID_ARG;
    const bool weights = io->q_weight || io->k_weight;
    // read for an empty batch too, whose gradients of zero the kernel writes
    if (!aligned(io->q_weight, 16) || !aligned(io->k_weight, 16)) return HGA_ERR_INVALID_ARG;
    if (dims->T > 0) {
        if (a.rope.R && (!io->pos || !aligned(io->pos, 4))) return HGA_ERR_INVALID_ARG;
        if (!io->d_q || !io->d_k || !rows_ok(io->dq, io->dq_stride, dims->Hq, D, e) ||
            !rows_ok(io->dk, io->dk_stride, dims->Hkv, D, e) ||
            (io->dv && !rows_ok(io->dv, io->dv_stride, dims->Hkv, D, e)) ||
            (io->q_weight && !rows_ok(io->q, io->q_stride, dims->Hq, D, e)) ||
            (io->k_weight && !rows_ok(io->k, io->k_stride, dims->Hkv, D, e)))
            return HGA_ERR_INVALID_ARG;
        const void *rows[] = {io->d_q, io->d_k, io->d_v};
        for (const void *p : rows)
            if (!aligned(p, 16)) return HGA_ERR_INVALID_ARG;
    }
    if (weights && (!workspace || workspace_bytes < qk_grad_workspace_bytes(D) ||
                    !aligned(workspace, 256)))
        return HGA_ERR_WORKSPACE;
    a.tokens = (int64_t)dims->B * dims->T;
    a.Hq = dims->Hq;
    a.Hkv = dims->Hkv;
    a.io = *io;
    a.part = static_cast<float *>(workspace);
    return launch_qk_norm_rope_backward(a, dims->dtype, D, (cudaStream_t)stream);
}

size_t hga_paged_decode_workspace(const hga_paged_dims *dims) {
    if (check_pages(dims) != HGA_OK ||
        check_heads(dims->Hq, dims->Hkv, dims->D, dims->dtype) != HGA_OK)
        return 0;
    return paged_decode_workspace_bytes(dims->B, dims->Hq, dims->Hkv, dims->D, dims->dtype);
}

hga_status hga_paged_decode(const hga_paged_dims *dims, const void *q, const void *k_pages,
                            const void *v_pages, const int32_t *block_table, const int32_t *lens,
                            int32_t window, int32_t sinks, double scale, void *out, float *lse,
                            void *workspace, size_t workspace_bytes, void *stream) {
    hga_status s = check_pages(dims);
    if (s != HGA_OK) return s;
    s = check_heads(dims->Hq, dims->Hkv, dims->D, dims->dtype);
    if (s != HGA_OK) return s;
    if (!q || !k_pages || !v_pages || !block_table || !lens || !out) return HGA_ERR_INVALID_ARG;
    const void *rows[] = {q, k_pages, v_pages, out};
    for (const void *p : rows)
        if (!aligned(p, 16)) return HGA_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(lens, 4) || !aligned(lse, 4)) return HGA_ERR_INVALID_ARG;
    if (window < 0 || sinks < 0 || !(scale >= 0.0) || !held32(scale * M_LOG2E))
        return HGA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < paged_decode_workspace_bytes(dims->B, dims->Hq, dims->Hkv, dims->D,
                                                       dims->dtype))
        return HGA_ERR_WORKSPACE;
    PagedArgs a;
    a.B = dims->B;
    a.Hq = dims->Hq;
    a.Hkv = dims->Hkv;
    a.G = dims->Hq / dims->Hkv;
    a.num_pages = dims->num_pages;
    a.log2_page = log2_of(dims->page_size);
    a.max_pages = dims->max_pages;
    a.window = window;
    a.sinks = window > 0 ? sinks : 0;
    a.scale_log2 = (float)((scale > 0.0 ? scale : 1.0 / std::sqrt((double)dims->D)) * M_LOG2E);
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    a.table = block_table;
    a.lens = lens;
    a.out = out;
    a.lse = lse;
    return launch_paged_decode(a, dims->dtype, dims->D, workspace, (cudaStream_t)stream);
}

}  // extern "C"
