// Per-head RMS norms of queries and keys with the position rotation in the same
// pass, and its gradient (hga_qk_norm_rope, hga_qk_norm_rope_backward).
//
//   r = (mean x^2 + eps)^(-1/2), and for a pair (a, b) of a row
//   y_a = r (a (w_a cos) - b (w_b sin)),  y_b = r (b (w_b cos) + a (w_a sin))
// (dimensions outside the rotated part: y_a = r a w_a): weight and rotation are one
// multiply-add with constants that depend on the token alone.
//
// Bound by HBM: every row is read once and written once.  A warp walks tokens and
// takes a token's rows N at a time (a step: 512 bytes of rows, 16 lanes to a bf16
// row of 128), so that cos and sin (64-bit fixed-point angles, sincospif) are formed
// once a token.  The steps ahead, the next tokens' among them, are on their way to
// a ring of shared memory (cp.async, 16 bytes a lane), so that what is in flight does
// not depend on registers.  From there a lane reads V / 2 pairs of its row, both
// members, so that no value crosses lanes and only the sum of squares does; the
// arithmetic is two-lane fp32.
// Measured, 32K tokens of 32 + 4 + 4 bf16 heads of 128 (671 MB): 144 us with a
// 16-byte word per lane loaded to registers and partners exchanged by shuffles
// (bound by issue and shuffle latency), 121 us with whole pairs per lane and four
// rows in flight per lane, 111 with the ring; the gradient with fp32 dy (1.31 GB) 259,
// 231 and 193 us (6.8 TB/s).  Heads of 64 in small numbers are bound by issue, by what
// a token costs before its rows (2 + 1 + 1 heads of 64: 36 us for 32K tokens).
#include <algorithm>
#include <type_traits>

#include "paged_internal.cuh"
#include "sm100.cuh"
#include "vec.cuh"

namespace hga {

__device__ int g_qk_error = 0;

namespace {

using sm100::f2_fma;
using sm100::f2_mul;
using sm100::f2_pack;
using sm100::f2_unpack;

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <typename T, int D> struct Row {
    static constexpr int V = 16 / (int)sizeof(T);      // values per lane
    static constexpr int P = V / 2;                    // pairs per lane
    static constexpr int L = D / V;                    // lanes per row
    static constexpr int N = 32 / L;                   // rows per warp and step
};

// cos and sin of a token's pairs.  A lane forms those of pairs lane and lane + 32: it
// keeps their turn rates (an index into the kernel's parameters that differs from
// lane to lane is read one lane after the other), and the position of its next token
// is on its way while this one's rows are worked on.  (Both read at each token's
// start: 44 us instead of 35 for 8K tokens of 32 + 4 + 4 heads of 128.)
template <int D> struct Angles {
    static constexpr int J = D / 64;      // pairs per lane
    unsigned long long turn[J];
    __device__ __forceinline__ void begin(const PairRope &r) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < J; ++j) turn[j] = lane + 32 * j < r.R / 2 ? r.turn[lane + 32 * j] : 0;
    }
    // the angles of position p, times the magnitude -> cs[R / 2]
    __device__ __forceinline__ void form(const PairRope &r, int32_t p, float2 *cs) const {
        const int lane = threadIdx.x & 31;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            // the angle in turns modulo 1 as a wrapping 64-bit product: exact for any p
            const unsigned long long u = (unsigned long long)(long long)p * turn[j];
            float s, c;
            sincospif((float)(int)(u >> 32) * 0x1p-31f, &s, &c);
            // pairs outside the rotated part: 1
            const float m = lane + 32 * j < r.R / 2 ? r.magnitude : 1.f;
            cs[lane + 32 * j] = make_float2(c * m, s * m);
        }
        __syncwarp();
    }
};

// The dimensions a lane owns: P at lo and P at hi.  In the half layout these are the
// first and second members of its pairs (outside the rotated part any two words);
// in the interleaved layout they are adjacent and alternate.
struct Place {
    int lo, hi, pair;     // pair: of its first pair
    bool turns;           // inside the rotated part
};
template <typename T, int D, bool kInter> __device__ __forceinline__ Place place(int R) {
    using W = Row<T, D>;
    const int l = (threadIdx.x & 31) % W::L;
    Place p = {l * W::V, l * W::V + W::P, l * W::P, l * W::V < R};
    if (!kInter && p.turns) {
        p.lo = l * W::P;
        p.hi = R / 2 + l * W::P;
    }
    return p;
}

// What a lane's partners add to its dimensions: outside the rotated part nothing, also
// where a partner is infinite and its product with a sine of 0 is NaN (-0, which
// leaves every x as it is).  Where all of the head turns the kernels leave this out.
struct Turns {
    uint64_t keep, none;
    __device__ __forceinline__ explicit Turns(const Place &p)
        : keep(p.turns ? ~0ull : 0ull), none(p.turns ? 0ull : 0x8000000080000000ull) {}
    __device__ __forceinline__ uint64_t cross(uint64_t x) const { return (x & keep) | none; }
};

// A lane's part of a row as it lies in memory: 16 bytes (fp32 gradients of bf16
// rows: 32).
template <typename T, int P> struct Raw {
    static constexpr int B = P * (int)sizeof(T) / 4;   // 32-bit words per half: 2 or 4
    uint32_t w[2 * B];
};
// (ordinary loads: a read-only one may be moved ahead of the wait for the kernel before)
template <typename T, int P, bool kInter>
__device__ __forceinline__ void load_raw(Raw<T, P> &x, const T *row, const Place &p) {
    static_assert(Raw<T, P>::B == 2, "8 bytes a half");
    if constexpr (kInter) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + p.lo);
        x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint2 v = *reinterpret_cast<const uint2 *>(row + (h ? p.hi : p.lo));
            x.w[2 * h] = v.x, x.w[2 * h + 1] = v.y;
        }
    }
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
// the same from shared memory: lo and hi are the addresses of the lane's words
template <typename T, int P, bool kInter>
__device__ __forceinline__ void read_raw(Raw<T, P> &x, uint32_t lo, uint32_t hi) {
    constexpr int B = Raw<T, P>::B;
    if constexpr (B == 2 && kInter) {
        const uint4 v = lds128(lo);
        x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (B == 4) {
                const uint4 v = lds128(h ? hi : lo);
                x.w[4 * h] = v.x, x.w[4 * h + 1] = v.y, x.w[4 * h + 2] = v.z, x.w[4 * h + 3] = v.w;
            } else {
                const uint2 v = lds64(h ? hi : lo);
                x.w[2 * h] = v.x, x.w[2 * h + 1] = v.y;
            }
        }
    }
}
template <typename T, int P, bool kInter>
__device__ __forceinline__ void store_raw(T *lo, T *hi, const Raw<T, P> &x) {
    if constexpr (kInter) {
        *reinterpret_cast<uint4 *>(lo) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    } else {
        *reinterpret_cast<uint2 *>(lo) = make_uint2(x.w[0], x.w[1]);
        *reinterpret_cast<uint2 *>(hi) = make_uint2(x.w[2], x.w[3]);
    }
}

// First and second members of the pairs, two values to a 64-bit register.
template <int P> struct Pairs {
    uint64_t a[P / 2], b[P / 2];
};
template <typename T> __device__ __forceinline__ float value(const uint32_t *w, int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}
template <typename T, int P, bool kInter>
__device__ __forceinline__ Pairs<P> unpack(const Raw<T, P> &x) {
    Pairs<P> y;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
        if (kInter) {
            y.a[i] = f2_pack(value<T>(x.w, 4 * i), value<T>(x.w, 4 * i + 2));
            y.b[i] = f2_pack(value<T>(x.w, 4 * i + 1), value<T>(x.w, 4 * i + 3));
        } else {
            y.a[i] = f2_pack(value<T>(x.w, 2 * i), value<T>(x.w, 2 * i + 1));
            y.b[i] = f2_pack(value<T>(x.w, P + 2 * i), value<T>(x.w, P + 2 * i + 1));
        }
    }
    return y;
}
template <typename T, int P, bool kInter>
__device__ __forceinline__ Raw<T, P> pack(const Pairs<P> &y) {
    Raw<T, P> x;
    float v[2 * P];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
        const float2 a = f2_unpack(y.a[i]), b = f2_unpack(y.b[i]);
        if (kInter) {
            v[4 * i] = a.x, v[4 * i + 1] = b.x, v[4 * i + 2] = a.y, v[4 * i + 3] = b.y;
        } else {
            v[2 * i] = a.x, v[2 * i + 1] = a.y, v[P + 2 * i] = b.x, v[P + 2 * i + 1] = b.y;
        }
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) x.w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            x.w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return x;
}

// cos and sin of a lane's pairs.
template <int P>
__device__ __forceinline__ void trig(const Place &p, const float2 *cs, float (&c)[P], float (&s)[P]) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const float2 t = cs[p.pair + e];
        c[e] = t.x;
        s[e] = t.y;
    }
}

// A lane's weights as they lie in memory; ones where there are none.
template <typename T, int P, bool kInter>
__device__ __forceinline__ void load_weight(Raw<T, P> &x, const void *w, const Place &p) {
    if (w) {
        load_raw<T, P, kInter>(x, static_cast<const T *>(w), p);
        return;
    }
    Pairs<P> y;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) y.a[i] = y.b[i] = f2_pack(1.f, 1.f);
    x = pack<T, P, kInter>(y);
}

template <int L> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float both(uint64_t x) {
    const float2 f = f2_unpack(x);
    return f.x + f.y;
}

// What a call does, by kind of row: 0 queries, 1 keys, 2 values.  The kernels index
// these with a kind that is the same for the whole warp.
struct QkWork {
    int n[3];                  // rows of a token that are wanted
    int steps[3];              // steps they take
    int full[3], rest[3];      // steps with all their rows, rows of a ragged last one
    int H[3];                  // heads: rows of a token in the dense tensors
    const void *in[3];         // forward: the inputs; gradient: x
    int64_t in_stride[3];
    const void *grad[3];       // gradient: dense dy
    void *out[3];              // forward: dense outputs; gradient: dx
    int64_t out_stride[3];
    void *pages[3];
    const void *weight[3];
    int split;                 // warps per token
    unsigned warps;            // tokens * split: below 2^31, as only few tokens are split
};

// The token of warp wg and, of each kind, its steps [a, b): all of them without
// kSplit; else the warps of a token share the kinds' steps in a row.
template <bool kSplit> struct Part {
    unsigned tok;
    int s0, s1;
    __device__ __forceinline__ void of(const QkWork &K, unsigned wg) {
        tok = wg;
        if (kSplit) {
            const unsigned all = (unsigned)(K.steps[0] + K.steps[1] + K.steps[2]);
            const unsigned part = wg % (unsigned)K.split;
            tok = wg / (unsigned)K.split;
            s0 = (int)(all * part / (unsigned)K.split);
            s1 = (int)(all * (part + 1) / (unsigned)K.split);
        }
    }
    __device__ __forceinline__ int a(const QkWork &K, int kind) const {
        return kSplit ? max(s0 - at(K, kind), 0) : 0;
    }
    __device__ __forceinline__ int b(const QkWork &K, int kind) const {
        return kSplit ? min(s1 - at(K, kind), K.steps[kind]) : K.steps[kind];
    }
    __device__ __forceinline__ int at(const QkWork &K, int kind) const {
        return kind == 0 ? 0 : kind == 1 ? K.steps[0] : K.steps[0] + K.steps[1];
    }
};

// The walk that runs ahead: the rows of a warp's tokens, a step of N rows at a time.
// The first `full` steps left of a kind have all their rows; a last one may be ragged.
template <int N, bool kSplit> struct Walk {
    unsigned wg, stride;
    Part<kSplit> part;
    int kind, left, full;      // kind 3: none left
    int h;                     // first row
    __device__ __forceinline__ void begin(const QkWork &K, unsigned first, unsigned stride_) {
        wg = first, stride = stride_;
        kind = 2;
        next(K);
    }
    // the next kind with steps, of this token or the following ones
    __device__ __forceinline__ void next(const QkWork &K) {
        for (;;) {
            if (kind == 2) {
                if (wg >= K.warps) {
                    kind = 3, left = 0;
                    return;
                }
                part.of(K, wg);
                wg += stride;
                kind = -1;
            }
            ++kind;
            const int a = part.a(K, kind), b = part.b(K, kind);
            h = a * N;
            left = b - a;
            full = (kSplit ? min(b, K.full[kind]) : K.full[kind]) - a;
            if (left > 0) return;
        }
    }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// the same for data that L2 need not keep
__device__ __forceinline__ void cp16_once(uint32_t dst, const void *src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "l"(policy)
                 : "memory");
}
// zeros, and no read, where live is false
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- forward: steps of 2 N rows (1 KB); 128 registers and 24 KB of ring a CTA, two
// CTAs per SM.  Half of the traffic is writes, and what bounds the pass is how HBM
// takes both: more loads in flight make it slower (32K tokens of 32 + 4 + 4 bf16 heads
// of 128: depth 8 126 us, 3 118; 2 is worse for small heads), and telling L2 that
// what is read is not read again gives 111 (a plain copy of these 671 MB takes 103).
// For the gradient, three quarters reads, the hint is worse (217 us for 193).
constexpr int kDepth = 3, kStep = 1024, kCtas = 148 * 2;

// Two rows of a lane (at lo/hi and 512 bytes on in shared memory, N rows on in
// memory): y = r (x A + x' B), to `to` and, where given, `also`.
template <typename T, int D, bool kInter, bool kWhole, bool kCheck>
__device__ __forceinline__ void two_rows(uint32_t lo, uint32_t hi, bool norm, float eps,
                                         const Pairs<Row<T, D>::P> &c, const Pairs<Row<T, D>::P> &s,
                                         const Turns &turns, T *to, T *also, int skip, bool live0, bool live1) {
    using W = Row<T, D>;
    constexpr int P = W::P;
    Pairs<P> x[2];
    float r[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        Raw<T, P> raw;
        read_raw<T, P, kInter>(raw, lo + u * 512, hi + u * 512);
        x[u] = unpack<T, P, kInter>(raw);
    }
    if (norm) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint64_t ss = f2_mul(x[u].a[0], x[u].a[0]);
#pragma unroll
            for (int e = 1; e < P / 2; ++e) ss = f2_fma(x[u].a[e], x[u].a[e], ss);
#pragma unroll
            for (int e = 0; e < P / 2; ++e) ss = f2_fma(x[u].b[e], x[u].b[e], ss);
            r[u] = both(ss);
        }
#pragma unroll
        for (int o = W::L / 2; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < 2; ++u) r[u] += __shfl_xor_sync(0xffffffffu, r[u], o);
#pragma unroll
        for (int u = 0; u < 2; ++u) r[u] = rsqrtf(fmaf(r[u], 1.f / D, eps));
    } else {
        r[0] = r[1] = 1.f;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint64_t rr = f2_pack(r[u], r[u]);
        Pairs<P> y;
#pragma unroll
        for (int e = 0; e < P / 2; ++e) {
            const uint64_t a = f2_mul(x[u].b[e], s.a[e]), b = f2_mul(x[u].a[e], s.b[e]);
            y.a[e] = f2_mul(f2_fma(x[u].a[e], c.a[e], kWhole ? a : turns.cross(a)), rr);
            y.b[e] = f2_mul(f2_fma(x[u].b[e], c.b[e], kWhole ? b : turns.cross(b)), rr);
        }
        const Raw<T, P> z = pack<T, P, kInter>(y);
        if (!kCheck || (u ? live1 : live0)) {
            T *at = to + u * W::N * D;
            store_raw<T, P, kInter>(at, at + skip, z);
            if (also) {
                at = also + u * W::N * D;
                store_raw<T, P, kInter>(at, at + skip, z);
            }
        }
    }
}

template <typename T, int D, bool kInter, bool kSplit>
__global__ void __launch_bounds__(kThreads, 2) k_qk_norm_rope(const QkArgs A, const QkWork K) {
    using W = Row<T, D>;
    constexpr int P = W::P, N2 = 2 * W::N, E = (int)sizeof(T);
    __shared__ float2 cs_all[kWarps][kMaxHalf];
    extern __shared__ __align__(16) char ring_all[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / W::L;
    const int d0 = (lane % W::L) * W::V;
    const unsigned first = blockIdx.x * (unsigned)kWarps + warp, stride = gridDim.x * kWarps;
    const uint32_t ring = sm100::smem_addr(ring_all) + warp * kDepth * kStep, mine = ring + lane * 16;
    float2 *cs = cs_all[warp];
    const Place pl = place<T, D, kInter>(A.rope.R);
    const Turns turns(pl);
    const uint32_t lo = ring + (sub * D + pl.lo) * E, hi = ring + (sub * D + pl.hi) * E;
    const float eps = (float)A.io.eps;

    const uint64_t once = sm100::l2_policy_evict_first();

    // ---- the steps ahead
    Walk<N2, kSplit> p = {};
    const T *src = nullptr;
    auto find = [&]() {
        if (p.kind == 3) return;
        src = static_cast<const T *>(K.in[p.kind]) + p.part.tok * K.in_stride[p.kind] + (p.h + sub) * D + d0;
    };
    p.begin(K, first, stride);
    find();
    auto issue = [&](uint32_t at) {               // at: offset of a ring slot
        if (p.left > 0) {
            if (p.full > 0) {
                cp16_once(mine + at, src, once);
                cp16_once(mine + at + 512, src + W::N * D, once);
                --p.full;
            } else {
                // rows beyond the last are zeros; the address given for them is row 0's
                const int rest = K.rest[p.kind];
                const T *row0 = src - sub * D;
                cp16(mine + at, sub < rest ? src : row0, sub < rest);
                cp16(mine + at + 512, sub + W::N < rest ? src + W::N * D : row0, sub + W::N < rest);
            }
            src += N2 * D;
            if (--p.left == 0) {
                p.next(K);
                find();
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) issue(i * kStep);

    // ---- the rows at hand
    Angles<D> ang;
    ang.begin(A.rope);
    Raw<T, P> wraw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) load_weight<T, P, kInter>(wraw[i], K.weight[i], pl);
    int32_t next_pos = 0, next_row = -1;          // of the token that comes next
    auto ahead = [&](unsigned wg) {
        if (wg >= K.warps) return;
        const unsigned t = kSplit ? wg / (unsigned)K.split : wg;
        if (A.rope.R) next_pos = A.io.pos[t];
        if (A.io.slot) next_row = A.io.slot[t];
    };
    ahead(first);
    uint32_t at = 0, to_fill = (kDepth - 1) * kStep;     // ring offsets
    auto step = [&]() {                           // makes the next step's rows readable
        __syncwarp();                             // the slot filled now has been read
        issue(to_fill);
        to_fill = to_fill == (kDepth - 1) * kStep ? 0 : to_fill + kStep;
        cp_wait<kDepth - 1>();
        __syncwarp();
    };
    auto done = [&]() { at = at == (kDepth - 1) * kStep ? 0 : at + kStep; };
    if (A.rope.R == 0) ang.form(A.rope, 0, cs);   // rates of 0: cos 1, sin 0
    for (unsigned wg = first; wg < K.warps; wg += stride) {
        Part<kSplit> c;
        c.of(K, wg);
        const unsigned tok = c.tok;
        const int32_t pos = next_pos;
        int page_row = next_row;
        ahead(wg + stride);
        if (page_row < -1 || page_row >= A.io.num_slots) {
            if (A.io.slot && lane == 0) atomicExch(&g_qk_error, (int)HGA_ERR_BOUNDS);
            page_row = -1;
        }
        if (A.rope.R && (!kSplit || c.s0 < K.steps[0] + K.steps[1])) ang.form(A.rope, pos, cs);
#pragma unroll
        for (int kind = 0; kind < 3; ++kind) {
            const int first_step = c.a(K, kind), last_step = c.b(K, kind);
            if (first_step >= last_step) continue;
            const int rest = K.rest[kind], off = (first_step * N2 + sub) * D + (kind == 2 ? d0 : pl.lo);
            const bool live0 = sub < rest, live1 = sub + W::N < rest;   // of a ragged last step
            int full = (kSplit ? min(last_step, K.full[kind]) : K.full[kind]) - first_step;
            const int ragged = last_step - first_step - full;
            // where the rows go: `to`, and `also` where both are wanted
            void *pages = page_row < 0 ? nullptr : K.pages[kind];
            T *to = static_cast<T *>(K.out[kind]), *also = static_cast<T *>(pages);
            if (to) to += tok * (int64_t)(K.H[kind] * D) + off;
            if (also) also += page_row * (int64_t)(K.H[kind] * D) + off;
            if (!to) to = also, also = nullptr;
            if (!to) {                            // nowhere: read and dropped
                for (int n = full + ragged; n > 0; --n) {
                    step();
                    done();
                }
                continue;
            }
            if (kind == 2) {                      // values: copied
                for (int n = full + ragged; n > 0; --n, --full) {
                    step();
                    const uint4 x = lds128(mine + at), y = lds128(mine + at + 512);
                    done();
                    if (full > 0 || live0) {
                        *reinterpret_cast<uint4 *>(to) = x;
                        if (also) *reinterpret_cast<uint4 *>(also) = x;
                    }
                    if (full > 0 || live1) {
                        *reinterpret_cast<uint4 *>(to + W::N * D) = y;
                        if (also) *reinterpret_cast<uint4 *>(also + W::N * D) = y;
                    }
                    to += N2 * D;
                    if (also) also += N2 * D;
                }
                continue;
            }
            const bool norm = K.weight[kind] != nullptr;
            Pairs<P> ct, st;                      // w_a cos, w_b cos; -w_b sin, w_a sin
            {
                float cf[P], tf[P];
                trig<P>(pl, cs, cf, tf);
                const Pairs<P> w = unpack<T, P, kInter>(wraw[kind]);
#pragma unroll
                for (int i = 0; i < P / 2; ++i) {
                    const uint64_t cc = f2_pack(cf[2 * i], cf[2 * i + 1]);
                    ct.a[i] = f2_mul(w.a[i], cc);
                    ct.b[i] = f2_mul(w.b[i], cc);
                    st.a[i] = f2_mul(w.b[i], f2_pack(-tf[2 * i], -tf[2 * i + 1]));
                    st.b[i] = f2_mul(w.a[i], f2_pack(tf[2 * i], tf[2 * i + 1]));
                }
            }
            const int skip = pl.hi - pl.lo;
            auto rows = [&](auto whole) {
                constexpr bool W = decltype(whole)::value;
                for (int n = full; n > 0; --n) {
                    step();
                    two_rows<T, D, kInter, W, false>(lo + at, hi + at, norm, eps, ct, st, turns, to, also,
                                                     skip, true, true);
                    done();
                    to += N2 * D;
                    if (also) also += N2 * D;
                }
                if (ragged) {
                    step();
                    two_rows<T, D, kInter, W, true>(lo + at, hi + at, norm, eps, ct, st, turns, to, also,
                                                    skip, live0, live1);
                    done();
                }
            };
            if (A.rope.R == D) rows(std::true_type{});
            else rows(std::false_type{});
        }
    }
    cp_wait<0>();
}

// ---- gradient.  With g = R^T dy, u = g w:
//   dw_d += g_d x_d r,   dx = r u - x r^3 mean(u x)
// A warp walks tokens in a fixed order and keeps the sums of its lanes' weight
// gradients in registers; a CTA adds its warps', k_qk_weight_grad the CTAs'.
// Steps of N rows; 128 registers and at most 48 KB of ring a CTA, two CTAs per SM.
constexpr int kGradDepth = 4, kGradCtas = 148 * 2;

template <typename T, typename G> constexpr int grad_step() {    // bytes of a step: x and dy
    return 512 + 512 * (int)(sizeof(G) / sizeof(T));
}

template <typename T, typename G, int D, bool kInter, bool kSplit>
__global__ void __launch_bounds__(kThreads, 2) k_qk_grad(const QkGradArgs A, const QkWork K) {
    using W = Row<T, D>;
    constexpr int P = W::P, V = W::V, GW = (int)(sizeof(G) / sizeof(T)), S = grad_step<T, G>();
    constexpr int E = (int)sizeof(T), EG = (int)sizeof(G);
    extern __shared__ __align__(16) char ring_all[];
    __shared__ float2 cs_all[kWarps][kMaxHalf];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / W::L;
    const int d0 = (lane % W::L) * V;
    const unsigned first = blockIdx.x * (unsigned)kWarps + warp, stride = gridDim.x * kWarps;
    const uint32_t ring = sm100::smem_addr(ring_all) + warp * kGradDepth * S;
    float2 *cs = cs_all[warp];
    const Place pl = place<T, D, kInter>(A.rope.R);
    const Turns turns(pl);
    const float eps = (float)A.io.eps;
    // a lane's words of a step's slot: x at 0, dy at 512
    const uint32_t xlo = ring + (sub * D + pl.lo) * E, xhi = ring + (sub * D + pl.hi) * E;
    const uint32_t glo = ring + 512 + (sub * D + pl.lo) * EG, ghi = ring + 512 + (sub * D + pl.hi) * EG;

    // ---- the steps ahead
    Walk<W::N, kSplit> p = {};
    const T *src = nullptr;
    const char *gsrc = nullptr;
    bool has_x = false;
    auto find = [&]() {
        if (p.kind == 3) return;
        has_x = K.weight[p.kind] != nullptr;
        if (has_x)
            src = static_cast<const T *>(K.in[p.kind]) + p.part.tok * K.in_stride[p.kind] + (p.h + sub) * D + d0;
        gsrc = static_cast<const char *>(K.grad[p.kind]) +
               (p.part.tok * (int64_t)(K.H[p.kind] * D) + (p.h + sub) * D) * EG + (lane % W::L) * 16;
    };
    const uint32_t xto = ring + lane * 16, gto = ring + 512 + sub * D * EG + (lane % W::L) * 16;
    p.begin(K, first, stride);
    find();
    auto issue = [&](uint32_t at) {
        if (p.left > 0) {
            if (p.full > 0) {
                if (has_x) cp16(xto + at, src);
#pragma unroll
                for (int j = 0; j < GW; ++j)     // a row's 16-byte words, L at a time
                    cp16(gto + at + j * W::L * 16, gsrc + j * W::L * 16);
                --p.full;
            } else {
                const int rest = K.rest[p.kind];
                const bool live = sub < rest;     // for the others: zeros, and row 0's address
                if (has_x) cp16(xto + at, live ? src : src - sub * D, live);
#pragma unroll
                for (int j = 0; j < GW; ++j)
                    cp16(gto + at + j * W::L * 16,
                         (live ? gsrc : gsrc - sub * D * EG) + j * W::L * 16, live);
            }
            src += W::N * D;
            gsrc += W::N * D * EG;
            if (--p.left == 0) {
                p.next(K);
                find();
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kGradDepth - 1; ++i) issue(i * S);

    Raw<T, P> wraw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) load_weight<T, P, kInter>(wraw[i], K.weight[i], pl);
    Pairs<P> sumq, sumk;
#pragma unroll
    for (int e = 0; e < P / 2; ++e) sumq.a[e] = sumq.b[e] = sumk.a[e] = sumk.b[e] = f2_pack(0.f, 0.f);

    // ---- the rows at hand
    Angles<D> ang;
    ang.begin(A.rope);
    int32_t next_pos = 0;                         // of the token that comes next
    auto ahead = [&](unsigned wg) {
        if (wg < K.warps && A.rope.R) next_pos = A.io.pos[kSplit ? wg / (unsigned)K.split : wg];
    };
    ahead(first);
    uint32_t at = 0, to_fill = (kGradDepth - 1) * S;     // ring offsets
    auto step = [&]() {                           // makes the next step's rows readable
        __syncwarp();                             // the slot filled now has been read
        issue(to_fill);
        to_fill = to_fill == (kGradDepth - 1) * S ? 0 : to_fill + S;
        cp_wait<kGradDepth - 1>();
        __syncwarp();
    };
    auto done = [&]() { at = at == (kGradDepth - 1) * S ? 0 : at + S; };
    uint64_t cc[P / 2], tt[P / 2], tn[P / 2];
    // one row of a lane; live: it exists (a ragged last step's others are zeros)
    auto row = [&](auto whole, const Pairs<P> &w, bool norm, T *out, bool live, Pairs<P> &sum) {
        step();
        Raw<G, P> graw;
        read_raw<G, P, kInter>(graw, glo + at, ghi + at);
        const Pairs<P> d = unpack<G, P, kInter>(graw);
        Pairs<P> g;
#pragma unroll
        for (int e = 0; e < P / 2; ++e) {
            const uint64_t a = f2_mul(d.b[e], tt[e]), b = f2_mul(d.a[e], tn[e]);
            g.a[e] = f2_fma(d.a[e], cc[e], decltype(whole)::value ? a : turns.cross(a));
            g.b[e] = f2_fma(d.b[e], cc[e], decltype(whole)::value ? b : turns.cross(b));
        }
        if (norm) {
            Raw<T, P> raw;
            read_raw<T, P, kInter>(raw, xlo + at, xhi + at);
            const Pairs<P> x = unpack<T, P, kInter>(raw);
            Pairs<P> u;
            uint64_t s2 = f2_mul(x.a[0], x.a[0]), s1x;
#pragma unroll
            for (int e = 0; e < P / 2; ++e) {
                u.a[e] = f2_mul(g.a[e], w.a[e]);
                u.b[e] = f2_mul(g.b[e], w.b[e]);
                if (e) s2 = f2_fma(x.a[e], x.a[e], s2);
                s2 = f2_fma(x.b[e], x.b[e], s2);
                s1x = e ? f2_fma(u.a[e], x.a[e], s1x) : f2_mul(u.a[e], x.a[e]);
                s1x = f2_fma(u.b[e], x.b[e], s1x);
            }
            float ss = both(s2), ux = both(s1x);
#pragma unroll
            for (int o = W::L / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                ux += __shfl_xor_sync(0xffffffffu, ux, o);
            }
            // a row that does not exist is all zeros: with eps 0 its r is infinite
            const float r = live ? rsqrtf(fmaf(ss, 1.f / D, eps)) : 0.f;
            // r^3 mean(u x) from the inside: r^3 alone leaves fp32 for rows of 1e13 or 1e-13
            const float f = -(r * ux * (1.f / D)) * r * r;
            const uint64_t rr = f2_pack(r, r), ff = f2_pack(f, f);
#pragma unroll
            for (int e = 0; e < P / 2; ++e) {
                sum.a[e] = f2_fma(f2_mul(g.a[e], x.a[e]), rr, sum.a[e]);
                sum.b[e] = f2_fma(f2_mul(g.b[e], x.b[e]), rr, sum.b[e]);
                g.a[e] = f2_fma(x.a[e], ff, f2_mul(u.a[e], rr));
                g.b[e] = f2_fma(x.b[e], ff, f2_mul(u.b[e], rr));
            }
        }
        done();
        if (live) store_raw<T, P, kInter>(out, out + (pl.hi - pl.lo), pack<T, P, kInter>(g));
    };
    if (A.rope.R == 0) ang.form(A.rope, 0, cs);   // rates of 0: cos 1, sin 0
    for (unsigned wg = first; wg < K.warps; wg += stride) {
        Part<kSplit> c;
        c.of(K, wg);
        const unsigned tok = c.tok;
        const int32_t pos = next_pos;
        ahead(wg + stride);
        if (A.rope.R && (!kSplit || c.s0 < K.steps[0] + K.steps[1])) ang.form(A.rope, pos, cs);
        {
            float cf[P], tf[P];
            trig<P>(pl, cs, cf, tf);
#pragma unroll
            for (int e = 0; e < P / 2; ++e) {
                cc[e] = f2_pack(cf[2 * e], cf[2 * e + 1]);
                tt[e] = f2_pack(tf[2 * e], tf[2 * e + 1]);
                tn[e] = f2_pack(-tf[2 * e], -tf[2 * e + 1]);
            }
        }
#pragma unroll
        for (int kind = 0; kind < 3; ++kind) {
            const int first_step = c.a(K, kind), last_step = c.b(K, kind);
            if (first_step >= last_step) continue;
            int full = (kSplit ? min(last_step, K.full[kind]) : K.full[kind]) - first_step;
            const int ragged = last_step - first_step - full;
            const bool exists = sub < K.rest[kind];       // the row of a ragged last step
            T *out = static_cast<T *>(K.out[kind]) + tok * K.out_stride[kind] +
                     (first_step * W::N + sub) * D + (kind == 2 ? d0 : pl.lo);
            if (kind < 2) {
                const Pairs<P> w = unpack<T, P, kInter>(wraw[kind]);
                const bool norm = K.weight[kind] != nullptr;
                auto rows = [&](auto whole) {
                    for (; full > 0; --full) {
                        row(whole, w, norm, out, true, kind ? sumk : sumq);
                        out += W::N * D;
                    }
                    if (ragged) row(whole, w, norm, out, exists, kind ? sumk : sumq);
                };
                if (A.rope.R == D) rows(std::true_type{});
                else rows(std::false_type{});
                continue;
            }
            for (int n = full + ragged; n > 0; --n, --full) {   // values: rounded to T
                step();
                uint4 raw[GW];
#pragma unroll
                for (int j = 0; j < GW; ++j) raw[j] = lds128(ring + at + 512 + (sub * D + d0) * EG + j * 16);
                done();
                float g[V];
                unpack_words<G, V>(raw, g);
                if (full > 0 || exists) store_slice<T, V>(out, g);
                out += W::N * D;
            }
        }
    }
    cp_wait<0>();
    if (!A.part) return;
    // a lane's sums in the order of its dimensions, in the ring's place
    float *red = reinterpret_cast<float *>(ring_all + warp * kGradDepth * S);
    __syncwarp();
    auto put = [&](const Pairs<P> &sum, float *dst) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
            float a = e % 2 ? f2_unpack(sum.a[e / 2]).y : f2_unpack(sum.a[e / 2]).x;
            float b = e % 2 ? f2_unpack(sum.b[e / 2]).y : f2_unpack(sum.b[e / 2]).x;
#pragma unroll
            for (int o = W::L; o < 32; o <<= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                b += __shfl_xor_sync(0xffffffffu, b, o);
            }
            if (sub == 0) {
                dst[kInter ? pl.lo + 2 * e : pl.lo + e] = a;
                dst[kInter ? pl.lo + 2 * e + 1 : pl.hi + e] = b;
            }
        }
    };
    static_assert(kGradDepth * S >= 2 * D * 4, "a warp's sums fit its ring");
    put(sumq, red);
    put(sumk, red + D);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w)
            x += reinterpret_cast<const float *>(ring_all + w * kGradDepth * S)[i];
        A.part[(int64_t)blockIdx.x * 2 * D + i] = x;
    }
}

// Sums of the CTAs' parts, 32 columns a CTA, in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) k_qk_weight_grad(const float *part, int ctas, float *dqw,
                                                         float *dkw) {
    __shared__ float red[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
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

// N: rows of a step
void set_work(QkWork &K, int N, int64_t tokens) {
    int steps = 0;
    for (int i = 0; i < 3; ++i) {
        K.full[i] = K.n[i] / N;
        K.rest[i] = K.n[i] % N;
        K.steps[i] = K.full[i] + (K.rest[i] > 0);
        steps += K.steps[i];
    }
    // Few tokens are spread over several warps each, up to four warps per SM and down
    // to one step a warp; every warp forms the angles again.  Spread / a warp per token /
    // spread up to sixteen warps per SM, us:
    //                              16 tokens          256                512
    //   32 + 4 + 4 bf16 x 128   3.6 / 6.3 / 3.6   4.9 / 6.4 / 5.9   5.5 / 6.5 / 6.4
    //     gradient (fp32 dy)    5.2 /10.7 / 5.2   8.0 /11.3 / 8.8   9.4 /11.7 /11.4
    //   2 + 1 + 1 bf16 x 64     3.0 / 3.5 / 3.0   3.3 / 3.6 / 3.2   3.6 / 3.7 / 3.9
    //     gradient              4.4 / 4.7 / 4.4   5.3 / 5.3 / 5.3   5.3 / 5.5 / 6.0
    //   8 + 8 + 8 fp32 x 64     3.0 / 4.1 / 3.0   3.4 / 4.2 / 3.8   4.1 / 4.3 / 4.6
    //     gradient              4.4 / 6.5 / 4.4   5.9 / 6.8 / 6.8   6.4 / 7.2 / 7.5
    const int64_t want = 148 * 4;
    K.split = tokens == 0 ? 1 : (int)std::min<int64_t>(std::max(steps, 1), std::max<int64_t>(1, (want + tokens - 1) / tokens));
    K.warps = (unsigned)(tokens * K.split);
}

template <typename T, int D> hga_status forward(const QkArgs &A, cudaStream_t st) {
    const hga_qk_io &io = A.io;
    QkWork K = {{io.q_out ? A.Hq : 0, io.k_out || io.k_pages ? A.Hkv : 0, io.v_out || io.v_pages ? A.Hkv : 0},
                {}, {}, {}, {A.Hq, A.Hkv, A.Hkv}, {io.q, io.k, io.v},
                {io.q_stride, io.k_stride, io.v_stride}, {}, {io.q_out, io.k_out, io.v_out}, {},
                {nullptr, io.k_pages, io.v_pages}, {io.q_weight, io.k_weight, nullptr}, 1, 0u};
    set_work(K, 2 * Row<T, D>::N, A.tokens);
    if (K.steps[0] + K.steps[1] + K.steps[2] == 0) return HGA_OK;
    const unsigned grid = std::min<unsigned>(kCtas, (K.warps + kWarps - 1) / kWarps);
    auto *k = A.rope.interleaved ? K.split > 1 ? k_qk_norm_rope<T, D, true, true> : k_qk_norm_rope<T, D, true, false>
              : K.split > 1      ? k_qk_norm_rope<T, D, false, true>
                                 : k_qk_norm_rope<T, D, false, false>;
    const size_t smem = (size_t)kWarps * kDepth * kStep;
    const cudaError_t e = ensure_smem((const void *)k, smem);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_dependent(k, dim3(grid), dim3(kThreads), smem, st, A, K));
}

template <typename T, typename G, int D> hga_status backward(const QkGradArgs &A0, cudaStream_t st) {
    QkGradArgs A = A0;
    const hga_qk_grad_io &io = A.io;
    const bool weights = io.d_q_weight || io.d_k_weight;
    if (!weights) A.part = nullptr;
    if (A.tokens == 0 && !weights) return HGA_OK;
    QkWork K = {{A.Hq, A.Hkv, io.dv ? A.Hkv : 0}, {}, {}, {}, {A.Hq, A.Hkv, A.Hkv}, {io.q, io.k, nullptr},
                {io.q_stride, io.k_stride, 0}, {io.d_q, io.d_k, io.d_v}, {io.dq, io.dk, io.dv},
                {io.dq_stride, io.dk_stride, io.dv_stride}, {}, {io.q_weight, io.k_weight, nullptr}, 1, 0u};
    set_work(K, Row<T, D>::N, A.tokens);
    // without tokens one CTA writes the weights' zero gradients
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(kGradCtas, ((int64_t)K.warps + kWarps - 1) / kWarps));
    auto *k = A.rope.interleaved ? K.split > 1 ? k_qk_grad<T, G, D, true, true> : k_qk_grad<T, G, D, true, false>
              : K.split > 1      ? k_qk_grad<T, G, D, false, true>
                                 : k_qk_grad<T, G, D, false, false>;
    const size_t smem = (size_t)kWarps * kGradDepth * grad_step<T, G>();
    cudaError_t e = ensure_smem((const void *)k, smem);
    if (e != cudaSuccess) return cuda_status(e);
    e = launch_dependent(k, dim3(grid), dim3(kThreads), smem, st, A, K);
    if (e != cudaSuccess || !weights) return cuda_status(e);
    return cuda_status(launch_dependent(k_qk_weight_grad<D>, dim3(2 * D / 32), dim3(1024), 0, st,
                                        (const float *)A.part, grid, io.d_q_weight, io.d_k_weight));
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

cudaError_t qk_error_word(int **word) { return cudaGetSymbolAddress((void **)word, g_qk_error); }

}  // namespace hga
