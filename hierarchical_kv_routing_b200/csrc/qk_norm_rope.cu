// Per-head RMS norms of queries and keys with the position rotation in the same
// pass, and its gradient (hga_qk_norm_rope, hga_qk_norm_rope_backward).
//
//   r = (mean x^2 + eps)^(-1/2),  y_d = r (x_d A_d + x_d' B_d)
// where d' is d's partner in its rotation pair, A_d = w_d cos and
// B_d = -+ w_d' sin (d outside the rotated part: A = w, B = 0): weight and
// rotation of a dimension are one multiply-add with constants that depend on the
// token alone, so a row costs a load, a sum of squares and 2 products a value.
//
// Bound by HBM: every row is read once and written once.  A row is spread over
// 16 bytes a lane (16 lanes for bf16 heads of 128), a warp takes the rows of one
// token so that its cos and sin (64-bit fixed-point angles, sincospif) are formed
// once, kUnroll loads are in flight per lane before the first is used, and the
// partner of a half-layout pair comes from the lane that holds it by a shuffle.
#include <algorithm>

#include "paged_internal.cuh"
#include "vec.cuh"

namespace hga {

__device__ int g_qk_error = 0;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <typename T, int D> struct Row {
    static constexpr int V = 16 / (int)sizeof(T);      // values per lane
    static constexpr int L = D / V;                    // lanes per row
    static constexpr int N = 32 / L;                   // rows per warp and step
};

// cos and sin (times the magnitude) of the pairs of position p -> cs[R / 2].
__device__ __forceinline__ void angles(const PairRope &r, int32_t p, float2 *cs) {
    for (int i = threadIdx.x & 31; i < r.R / 2; i += 32) {
        // the angle in turns modulo 1 as a wrapping 64-bit product: exact for any p
        const unsigned long long u = (unsigned long long)(long long)p * r.turn[i];
        float s, c;
        sincospif((float)(int)(u >> 32) * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * r.magnitude, s * r.magnitude);
    }
    __syncwarp();
}

// Where a lane's values stand in the rotation: the lane of their partners, the
// first pair, and whether they are first members of their pairs.
struct Place {
    int partner, pair;
    float sign;       // of sin in the forward: -1 for first members, +1 for second, 0 outside
};
template <typename T, int D, bool kInter> __device__ __forceinline__ Place place(int R) {
    using W = Row<T, D>;
    const int lane = threadIdx.x & 31, d0 = (lane % W::L) * W::V;
    Place p = {lane, 0, 0.f};
    if (d0 >= R) return p;
    if (kInter) {
        p.pair = d0 / 2;
        p.sign = 1.f;
    } else if (d0 < R / 2) {
        p = {lane + R / 2 / W::V, d0, -1.f};
    } else {
        p = {lane - R / 2 / W::V, d0 - R / 2, 1.f};
    }
    return p;
}

// cos and signed sin of a lane's values (interleaved: even values -sin, odd +sin).
template <int V, bool kInter>
__device__ __forceinline__ void trig(const Place &p, const float2 *cs, float (&c)[V], float (&s)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
        if (p.sign != 0.f) {
            const float2 t = cs[p.pair + (kInter ? e / 2 : e)];
            c[e] = t.x;
            s[e] = kInter ? (e % 2 ? t.y : -t.y) : p.sign * t.y;
        }
    }
}

// The partners of a lane's values, given as the 16-byte words that hold them.
template <typename T, int V, bool kInter, int NW>
__device__ __forceinline__ void partners(const uint4 (&w)[NW], const float (&x)[V], int src,
                                         float (&xp)[V]) {
    if (kInter) {
#pragma unroll
        for (int e = 0; e < V; ++e) xp[e] = x[e ^ 1];
    } else {
        uint4 o[NW];
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            o[i].x = __shfl_sync(0xffffffffu, w[i].x, src);
            o[i].y = __shfl_sync(0xffffffffu, w[i].y, src);
            o[i].z = __shfl_sync(0xffffffffu, w[i].z, src);
            o[i].w = __shfl_sync(0xffffffffu, w[i].w, src);
        }
        unpack_words<T, V>(o, xp);
    }
}

template <int L> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, int V> __device__ __forceinline__ void load_weight(const void *w, int d0, float (&x)[V]) {
    if (w) {
        load_slice<T, V>(static_cast<const T *>(w) + d0, x);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = 1.f;
    }
}

struct QkWork {
    int nq, nk, nv;    // rows of a token that are wanted
    int sq, sk, sv;    // steps of W::N rows they take
    int split;         // warps per token
};

constexpr int kUnroll = 4;

template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 3) k_qk_norm_rope(const QkArgs A, const QkWork K) {
    using W = Row<T, D>;
    constexpr int V = W::V;
    __shared__ float2 cs_all[kWarps][kMaxHalf];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / W::L;
    const int d0 = (lane % W::L) * V;
    const int64_t wg = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t tok = wg / K.split;
    if (tok >= A.tokens) return;
    const int steps = K.sq + K.sk + K.sv, part = (int)(wg % K.split);
    const int s0 = (int)((int64_t)steps * part / K.split);
    const int s1 = (int)((int64_t)steps * (part + 1) / K.split);
    int64_t slot = -1;
    if (A.io.slot && s1 > K.sq) {
        slot = A.io.slot[tok];
        if (slot < -1 || slot >= A.io.num_slots) {
            if (lane == 0) atomicExch(&g_qk_error, (int)HGA_ERR_BOUNDS);
            slot = -1;
        }
    }
    float2 *cs = cs_all[warp];
    if (A.rope.R && s0 < K.sq + K.sk) angles(A.rope, A.io.pos[tok], cs);
    const Place pl = place<T, D, kInter>(A.rope.R);

    // rows of one kind: steps [a, b) of its own numbering
    auto rows = [&](int a, int b, int count, const void *src, int64_t stride, const void *weight,
                    void *dense, int H, void *pages, bool turn) {
        if (a >= b) return;
        float ca[V], cb[V];
        if (turn) {
            float w[V], wp[V];
            trig<V, kInter>(pl, cs, ca, cb);
            load_weight<T, V>(weight, d0, w);
            if (kInter) {
#pragma unroll
                for (int e = 0; e < V; ++e) wp[e] = w[e ^ 1];
            } else {
                load_weight<T, V>(weight, (pl.partner % W::L) * V, wp);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                ca[e] *= w[e];
                cb[e] *= wp[e];
            }
        }
        const T *in = static_cast<const T *>(src) + tok * stride + d0;
        T *out = dense ? static_cast<T *>(dense) + tok * H * D + d0 : nullptr;
        T *pg = pages && slot >= 0 ? static_cast<T *>(pages) + slot * H * D + d0 : nullptr;
        for (int i = a; i < b; i += kUnroll) {
            uint4 x4[kUnroll][1];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int h = (i + u) * W::N + sub;
                if (i + u < b && h < count) x4[u][0] = __ldg(reinterpret_cast<const uint4 *>(in + h * D));
                else x4[u][0] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (i + u >= b) break;                 // the same for the whole warp
                const int h = (i + u) * W::N + sub;
                if (turn) {
                    float x[V], xp[V], y[V], r = 1.f;
                    unpack_words<T, V>(x4[u], x);
                    partners<T, V, kInter>(x4[u], x, pl.partner, xp);
                    if (weight) {
                        float ss = 0.f;
#pragma unroll
                        for (int e = 0; e < V; ++e) ss = fmaf(x[e], x[e], ss);
                        r = rsqrtf(row_sum<W::L>(ss) * (1.f / D) + (float)A.io.eps);
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] = r * fmaf(x[e], ca[e], xp[e] * cb[e]);
                    alignas(16) T packed[V];
                    store_slice<T, V>(packed, y);
                    x4[u][0] = *reinterpret_cast<const uint4 *>(packed);
                }
                if (h < count) {
                    if (out) *reinterpret_cast<uint4 *>(out + h * D) = x4[u][0];
                    if (pg) *reinterpret_cast<uint4 *>(pg + h * D) = x4[u][0];
                }
            }
        }
    };
    rows(s0, min(s1, K.sq), K.nq, A.io.q, A.io.q_stride, A.io.q_weight, A.io.q_out, A.Hq, nullptr, true);
    rows(max(s0 - K.sq, 0), min(s1 - K.sq, K.sk), K.nk, A.io.k, A.io.k_stride, A.io.k_weight,
         A.io.k_out, A.Hkv, A.io.k_pages, true);
    rows(max(s0 - K.sq - K.sk, 0), s1 - K.sq - K.sk, K.nv, A.io.v, A.io.v_stride, nullptr, A.io.v_out,
         A.Hkv, A.io.v_pages, false);
}

// ---- gradient.  With g = R^T dy, u = g w:
//   dw_d += g_d x_d r,   dx = r u - x r^3 mean(u x)
// A warp walks tokens in a fixed order and keeps the sums of its lanes' weight
// gradients in registers; a CTA adds its warps', k_qk_weight_grad the CTAs'.
constexpr int kGradUnroll = 2, kGradCtas = 148 * 2;

template <typename T, typename G, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) k_qk_grad(const QkGradArgs A, const QkWork K) {
    using W = Row<T, D>;
    constexpr int V = W::V, GW = V * (int)sizeof(G) / 16;
    __shared__ float2 cs_all[kWarps][kMaxHalf];
    __shared__ float red[kWarps][2][D];
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / W::L;
    const int d0 = (lane % W::L) * V;
    const Place pl = place<T, D, kInter>(A.rope.R);
    const int steps = K.sq + K.sk + K.sv;
    float2 *cs = cs_all[warp];
    float wq[V], wk[V], sumq[V], sumk[V];
    load_weight<T, V>(A.io.q_weight, d0, wq);
    load_weight<T, V>(A.io.k_weight, d0, wk);
#pragma unroll
    for (int e = 0; e < V; ++e) sumq[e] = sumk[e] = 0.f;

    for (int64_t wg = (int64_t)blockIdx.x * kWarps + warp; wg < A.tokens * K.split;
         wg += (int64_t)gridDim.x * kWarps) {
        const int64_t tok = wg / K.split;
        const int part = (int)(wg % K.split);
        const int s0 = (int)((int64_t)steps * part / K.split);
        const int s1 = (int)((int64_t)steps * (part + 1) / K.split);
        __syncwarp();
        if (A.rope.R && s0 < K.sq + K.sk) angles(A.rope, A.io.pos[tok], cs);
        float c[V], s[V];
        trig<V, kInter>(pl, cs, c, s);      // R^T: cos and minus the forward's signed sin

        auto rows = [&](int a, int b, int count, const void *src, int64_t stride, const float (&w)[V],
                        bool norm, const void *dsrc, void *dst, int64_t dstride, int H,
                        float (&sum)[V]) {
            const T *in = static_cast<const T *>(src) + tok * stride + d0;
            const G *gin = static_cast<const G *>(dsrc) + tok * H * D + d0;
            T *out = static_cast<T *>(dst) + tok * dstride + d0;
            for (int i = a; i < b; i += kGradUnroll) {
                uint4 x4[kGradUnroll][1], g4[kGradUnroll][GW];
#pragma unroll
                for (int u = 0; u < kGradUnroll; ++u) {
                    const int h = (i + u) * W::N + sub;
                    const bool live = i + u < b && h < count;
                    x4[u][0] = make_uint4(0u, 0u, 0u, 0u);
                    if (live && norm) x4[u][0] = __ldg(reinterpret_cast<const uint4 *>(in + h * D));
#pragma unroll
                    for (int j = 0; j < GW; ++j)
                        g4[u][j] = live ? __ldg(reinterpret_cast<const uint4 *>(gin + h * D) + j)
                                        : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int u = 0; u < kGradUnroll; ++u) {
                    if (i + u >= b) break;
                    const int h = (i + u) * W::N + sub;
                    float x[V], g[V], gp[V];
                    unpack_words<T, V>(x4[u], x);
                    unpack_words<G, V>(g4[u], g);
                    partners<G, V, kInter>(g4[u], g, pl.partner, gp);
#pragma unroll
                    for (int e = 0; e < V; ++e) g[e] = fmaf(g[e], c[e], -gp[e] * s[e]);
                    if (norm) {
                        float ss = 0.f, ux = 0.f;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            ss = fmaf(x[e], x[e], ss);
                            ux = fmaf(g[e] * w[e], x[e], ux);
                        }
                        ss = row_sum<W::L>(ss);
                        ux = row_sum<W::L>(ux);
                        const float r = rsqrtf(ss * (1.f / D) + (float)A.io.eps);
                        // a row beyond the count is all zeros: with eps 0 its r is infinite
                        const float rr = h < count ? r : 0.f;
                        const float f = rr * rr * rr * ux * (1.f / D);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            sum[e] = fmaf(g[e] * x[e], rr, sum[e]);
                            g[e] = fmaf(rr, g[e] * w[e], -x[e] * f);
                        }
                    }
                    if (h < count) store_slice<T, V>(out + h * D, g);
                }
            }
        };
        rows(s0, min(s1, K.sq), K.nq, A.io.q, A.io.q_stride, wq, A.io.q_weight != nullptr, A.io.d_q,
             A.io.dq, A.io.dq_stride, A.Hq, sumq);
        rows(max(s0 - K.sq, 0), min(s1 - K.sq, K.sk), K.nk, A.io.k, A.io.k_stride, wk,
             A.io.k_weight != nullptr, A.io.d_k, A.io.dk, A.io.dk_stride, A.Hkv, sumk);
        // values: rounded to the inputs' type
        const G *gin = static_cast<const G *>(A.io.d_v) + tok * A.Hkv * D + d0;
        T *out = static_cast<T *>(A.io.dv) + tok * A.io.dv_stride + d0;
        for (int i = max(s0 - K.sq - K.sk, 0); i < s1 - K.sq - K.sk; ++i) {
            const int h = i * W::N + sub;
            if (h >= K.nv) continue;
            float g[V];
            load_slice<G, V>(gin + h * D, g);
            store_slice<T, V>(out + h * D, g);
        }
    }
    if (!A.part) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int o = W::L; o < 32; o <<= 1) {
            sumq[e] += __shfl_xor_sync(0xffffffffu, sumq[e], o);
            sumk[e] += __shfl_xor_sync(0xffffffffu, sumk[e], o);
        }
        if (sub == 0) {
            red[warp][0][d0 + e] = sumq[e];
            red[warp][1][d0 + e] = sumk[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += red[w][i / D][i % D];
        A.part[(int64_t)blockIdx.x * 2 * D + i] = x;
    }
}

// Sums of the CTAs' parts, 32 columns a CTA, in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) k_qk_weight_grad(const float *part, int ctas, float *dqw,
                                                         float *dkw) {
    __shared__ float red[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
    float s = 0.f;
    for (int i = y; i < ctas; i += 32) s += part[(int64_t)i * 2 * D + col];
    red[y][x] = s;
    __syncthreads();
    s = red[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (x) return;
    const int c = blockIdx.x * 32 + y;
    float *dst = c < D ? dqw : dkw;
    if (dst) dst[c % D] = s;
}

template <typename T, int D> QkWork make_work(int64_t tokens, int nq, int nk, int nv) {
    constexpr int N = Row<T, D>::N;
    QkWork K;
    K.nq = nq, K.nk = nk, K.nv = nv;
    K.sq = (nq + N - 1) / N, K.sk = (nk + N - 1) / N, K.sv = (nv + N - 1) / N;
    // a warp per token where that fills the card; fewer tokens are spread over more
    // warps (each forms the angles again), down to one step a warp
    const int64_t want = 148 * 16;
    const int steps = std::max(1, K.sq + K.sk + K.sv);
    K.split = tokens == 0 ? 1 : (int)std::min<int64_t>(steps, std::max<int64_t>(1, (want + tokens - 1) / tokens));
    return K;
}

template <typename T, int D> hga_status forward(const QkArgs &A, cudaStream_t st) {
    const QkWork K = make_work<T, D>(A.tokens, A.io.q_out ? A.Hq : 0,
                                     A.io.k_out || A.io.k_pages ? A.Hkv : 0,
                                     A.io.v_out || A.io.v_pages ? A.Hkv : 0);
    if (K.sq + K.sk + K.sv == 0) return HGA_OK;
    const unsigned grid = (unsigned)((A.tokens * K.split + kWarps - 1) / kWarps);
    if (A.rope.interleaved) k_qk_norm_rope<T, D, true><<<grid, kThreads, 0, st>>>(A, K);
    else k_qk_norm_rope<T, D, false><<<grid, kThreads, 0, st>>>(A, K);
    return cuda_status(cudaGetLastError());
}

template <typename T, typename G, int D> hga_status backward(const QkGradArgs &A0, cudaStream_t st) {
    QkGradArgs A = A0;
    const bool weights = A.io.d_q_weight || A.io.d_k_weight;
    if (!weights) A.part = nullptr;
    if (A.tokens == 0 && !weights) return HGA_OK;
    const QkWork K = make_work<T, D>(A.tokens, A.Hq, A.Hkv, A.io.dv ? A.Hkv : 0);
    // without tokens one CTA writes the weights' zero gradients
    const int grid = (int)std::max<int64_t>(
        1, std::min<int64_t>(kGradCtas, (A.tokens * K.split + kWarps - 1) / kWarps));
    if (A.rope.interleaved) k_qk_grad<T, G, D, true><<<grid, kThreads, 0, st>>>(A, K);
    else k_qk_grad<T, G, D, false><<<grid, kThreads, 0, st>>>(A, K);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !weights) return cuda_status(e);
    return cuda_status(launch_dependent(k_qk_weight_grad<D>, dim3(2 * D / 32), dim3(1024), 0, st,
                                        (const float *)A.part, grid, A.io.d_q_weight,
                                        A.io.d_k_weight));
}

}  // namespace

hga_status launch_qk_norm_rope(const QkArgs &a, int dtype, int D, cudaStream_t st) {
    if (dtype == HGA_BF16)
        return D == 128 ? forward<__nv_bfloat16, 128>(a, st) : forward<__nv_bfloat16, 64>(a, st);
    return D == 128 ? forward<float, 128>(a, st) : forward<float, 64>(a, st);
}

size_t qk_grad_workspace_bytes(int D) { return (size_t)kGradCtas * 2 * D * 4; }

hga_status launch_qk_norm_rope_backward(const QkGradArgs &a, int dtype, int D, cudaStream_t st) {
    if (dtype == HGA_F32)
        return D == 128 ? backward<float, float, 128>(a, st) : backward<float, float, 64>(a, st);
    if (a.io.grad_dtype == HGA_F32)
        return D == 128 ? backward<__nv_bfloat16, float, 128>(a, st)
                        : backward<__nv_bfloat16, float, 64>(a, st);
    return D == 128 ? backward<__nv_bfloat16, __nv_bfloat16, 128>(a, st)
                    : backward<__nv_bfloat16, __nv_bfloat16, 64>(a, st);
}

hga_status qk_error_take(cudaStream_t st, bool clear) { return take_error_word(g_qk_error, st, clear); }

}  // namespace hga
