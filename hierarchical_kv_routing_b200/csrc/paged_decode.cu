// Attention of one new token per sequence over a paged key/value cache.
//
//   o = sum_j softmax_j(scale q.k_j) v_j   over the visible tokens j of a row:
//   j < len, and with a window w only j >= len - w or j < sinks.
//
// Bound by HBM: a visible key costs 2 D e bytes of K and V per KV head and
// 4 D G FLOP, G FLOP per byte for bf16.  So every K and V row is read once for the
// query heads that a CTA takes: 16 of bf16 heads of 128, 32 of 64, 8 of fp32; of a
// larger group G each chunk of that many reads K and V again, from L2.  bf16 products
// run on warp-level tensor-core tiles with the query heads as rows, whose operands a
// warp takes from its own ring without meeting the others; they fill a fifth of the
// tensor pipe up to 16 heads.  (On tcgen05 the keys would have to be the 64 or 128
// rows, as a group is fewer; for groups above 16, which are bound by issue here, that
// has not been built.)  fp32 products run on CUDA cores.  The design is about keeping
// loads in flight and every SM equally loaded.
//
// The visible tokens of a row are numbered 0 .. n-1 without a gap: the first
// min(sinks, lo) and then lo .. len-1, lo = max(0, len - window).  Tiles, splits
// and masks work on those numbers, so a windowed row costs what it attends, and
// only a row's last tile is ragged.
//
// Split: an item is a sequence and the KV heads (and query heads) one CTA takes
// together; its visible keys are cut into units.  The units of all items form one
// line, of which CTA i of n takes [U i / n, U (i + 1) / n): every CTA has the
// same work to one unit whatever the lengths are, and no length is read on the
// host.  A CTA's range covers whole items, whose rows it writes itself, and at
// most one item it continues and one it leaves open: those rows go to the
// workspace, and k_paged_join adds them up in CTA order.
//
// A CTA is four warps that run on their own: each streams tiles of 4 KB of K and
// 4 KB of V through a ring of kStages in shared memory (cp.async, 16 bytes a
// lane), three deep, so two CTAs per SM keep 128 KB in flight, above the ~50 KB
// that 7 TB/s and a microsecond of latency ask for.  The page of each key comes
// from the block table one tile ahead of its loads.  The warps of a KV head take
// its tiles in turn and are merged in shared memory at an item's end.
#include <algorithm>

#include "paged_internal.cuh"
#include "paged_walk.cuh"
#include "sm100.cuh"

namespace hga {

__device__ int g_paged_error = 0;

namespace {

using sm100::ex2;
using sm100::f2_fma;
using sm100::f2_mul;
using sm100::f2_pack;
using sm100::f2_unpack;

constexpr int kWarps = 4, kThreads = kWarps * 32, kStages = 3;
constexpr int kTileBytes = 4096;             // of K, and of V, per warp and stage
constexpr int kMaxCtas = 2 * 148;            // two per SM
constexpr int kUnitTiles = 4;                // tiles of a unit, over the warps of one head

struct Split {
    int items;         // per sequence: Hkv / hw
    int hw;            // adjacent KV heads of a CTA
    int gsplit, gch;   // chunks of a KV head's query heads, heads per chunk
    int rows;          // hw * gch: rows of a CTA's item
    int n;             // ranges; gsplit CTAs, one per chunk, walk each
    int by_item;       // join entries indexed by item (else by the CTA that starts it)
    float *part;       // [CTAs][2][rows][D]: continued and opened item, unnormalised
    float2 *ml;        // [CTAs][2][rows]: running maximum (base 2) and sum
    int4 *join;        // entry: (sequence, item, first range, last range); first -1: not split
};

// 16 bytes to shared memory; zeros, and no read, where live is false
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Weights (not negative, or NaN) as sums of two bf16: hi is the largest bf16 below the
// weight, at most 2^-7 of it short, lo the rest, rounded by at most half a step, 2^-8:
// together 2^-15 of the weight.  Neither is zero where the weight is not, nor of
// another sign, so that under an infinite value both give infinity.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const uint32_t ha = (uint32_t)max((int)__float_as_uint(a) - 1, 0) & 0xffff0000u;
    const uint32_t hb = (uint32_t)max((int)__float_as_uint(b) - 1, 0) & 0xffff0000u;
    hi = __byte_perm(ha, hb, 0x7632);
    lo = pack2(a - __uint_as_float(ha), b - __uint_as_float(hb));
}

// Where chunk c (16 bytes) of merge row r lies in its row: the four rows that a
// half-warp's 8-byte stores touch fall in different banks.
__device__ __forceinline__ int merge_chunk(int c, int r) { return c ^ (2 * r); }

// The visible tokens of a row: s first ones, then lo .. ; n in all.
struct Visible {
    int s, lo, n;
};
__device__ __forceinline__ Visible visible(const PagedArgs &A, int b) {
    int len = A.lens[b];
    if (len < 0 || (long long)len > ((long long)A.max_pages << A.log2_page)) len = 0;
    Visible v;
    v.lo = A.window > 0 ? max(0, len - A.window) : 0;
    v.s = min(A.sinks, v.lo);
    v.n = v.s + len - v.lo;
    return v;
}

// A CTA's walk over its units: the segment [k0, k1) of item (b, it) that is next.
struct Walk {
    int b, it, u, nu, cnt;
    int left;
    Visible v;
    __device__ __forceinline__ void take() { cnt = min(nu - u, left); }
    __device__ __forceinline__ bool next(const PagedArgs &A, const Split &S, int uk) {
        left -= cnt;
        if (left <= 0) return false;
        u = 0;
        if (++it == S.items) {
            it = 0;
            do {
                if (++b >= A.B) return false;
                v = visible(A, b);
                nu = units_of(v.n, uk);
            } while (nu == 0);
        }
        take();
        return true;
    }
};

// ---- bf16: m16n8k16 tiles.  S = Q K^T with the queries as the 16-row A operand
// (rows beyond the chunk's heads are zero) and K rows as its columns; the S
// accumulator, exponentiated and split into two bf16, is the A operand of O += P V, V
// read transposed.  Rows of shared memory are XOR-swizzled in 16-byte chunks so the
// eight rows of an ldmatrix fall in different banks.  The weights' lower parts are the
// upper half of a tile of 8 rows, at no product more, and a second product of one of
// 16 (64 x 16K tokens, one bf16 for a weight against two: 8/8 heads of 64 310 and 312
// us, 16/1 50 and 51, 32/1 59 and 68).  kRows = 24 and 32 are two tiles that share every
// fragment of K and V; 24 rows need the second product in one of them only (24/1 heads:
// 61 us, 69 on 32 rows).
template <int D, int kRows> struct TileBf16 {
    using T = __nv_bfloat16;
    static constexpr int kKeys = kTileBytes / (D * 2), kSwz = 7, kMerge = 8;
    static constexpr int M = (kRows + 15) / 16, R = kRows > 8 ? 2 : 1;   // tiles; groups of 8 rows
    // groups of tile t that are rows; where it is one, the other holds its lower parts
    static constexpr __host__ __device__ int groups(int t) { return kRows - 16 * t > 8 ? 2 : 1; }
    uint32_t q[M][D / 16][4];
    float o[M][D / 8][4];
    float m[M][R], l[M][R];

    __device__ __forceinline__ void begin(const PagedArgs &A, int b, int head0, int heads) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = (lane & 3) * 2;
        const T *base = static_cast<const T *>(A.q) + ((int64_t)b * A.Hq + head0) * D + c;
#pragma unroll
        for (int t = 0; t < M; ++t) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = t * 16 + g + (j & 1) * 8;
                    q[t][i][j] = 0;
                    if ((j & 1) < groups(t) && row < heads)
                        q[t][i][j] = *reinterpret_cast<const uint32_t *>(base + row * D + i * 16 + (j >> 1) * 8);
                }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
#pragma unroll
            for (int r = 0; r < groups(t); ++r) m[t][r] = -INFINITY, l[t][r] = 0.f;
        }
    }

    // valid: bit k set if key k of the tile counts
    __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, uint32_t valid, float scale,
                                         float *) {
        constexpr int NT = kKeys / 8;
        const int lane = threadIdx.x & 31, c = (lane & 3) * 2;
        float s[M][NT][4];
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[t][n][j] = 0.f;
        // matrices of an x4 load: keys 0-7 and 8-15 of the pair, two chunks of 8 dimensions
        const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t f[4];
                ldsm4(f, ks + (n * 8 + krow) * (D * 2) + (((i * 2 + kch) ^ (lane & 7)) << 4));
#pragma unroll
                for (int t = 0; t < M; ++t) {
                    mma16816(s[t][n], q[t][i], f[0], f[1]);
                    mma16816(s[t][n + 1], q[t][i], f[2], f[3]);
                }
            }
        constexpr uint32_t full = kKeys == 32 ? 0xffffffffu : (1u << (kKeys & 31)) - 1u;
        float top[M][R];
        bool grow = false;
#pragma unroll
        for (int t = 0; t < M; ++t) {
#pragma unroll
            for (int r = 0; r < groups(t); ++r) top[t][r] = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2 * groups(t); ++j) {
                    float &x = s[t][n][j];
                    x *= scale;
                    if (valid != full && !((valid >> (n * 8 + c + (j & 1))) & 1u)) x = -INFINITY;
                    top[t][j >> 1] = fmaxf(top[t][j >> 1], x);
                }
#pragma unroll
            for (int r = 0; r < groups(t); ++r) {
                top[t][r] = fmaxf(top[t][r], __shfl_xor_sync(0xffffffffu, top[t][r], 1));
                top[t][r] = fmaxf(top[t][r], __shfl_xor_sync(0xffffffffu, top[t][r], 2));
                // the reference moves only when the maximum passes it by 2^8: weights and
                // sums stay far from fp32's range, and O is rarely rescaled
                grow |= top[t][r] > m[t][r] + 8.f;
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int t = 0; t < M; ++t)
#pragma unroll
                for (int r = 0; r < groups(t); ++r) {
                    const float nm = top[t][r] > m[t][r] + 8.f ? top[t][r] : m[t][r];
                    const float f = nm == -INFINITY ? 1.f : ex2(m[t][r] - nm);
                    m[t][r] = nm;
                    l[t][r] *= f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
#pragma unroll
                        for (int j = 2 * r; j < (groups(t) == 1 ? 4 : 2 * r + 2); ++j) o[t][i][j] *= f;
                }
        }
#pragma unroll
        for (int t = 0; t < M; ++t) {
            float ref[R];
#pragma unroll
            for (int r = 0; r < groups(t); ++r) ref[r] = m[t][r] == -INFINITY ? 0.f : m[t][r];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2 * groups(t); ++j) {
                    s[t][n][j] = ex2(s[t][n][j] - ref[j >> 1]);
                    l[t][j >> 1] += s[t][n][j];
                }
        }
        const int vrow = lane & 15, vch = lane >> 4;
#pragma unroll
        for (int kb = 0; kb < kKeys / 16; ++kb) {
            // p: the weights' upper parts; the lower ones are in its other half with one
            // group of rows, else in low
            uint32_t p[M][4], low[M][4];
#pragma unroll
            for (int t = 0; t < M; ++t)
#pragma unroll
                for (int j = 0; j < 4; j += 3 - groups(t)) {
                    const float *x = s[t][2 * kb + (j >> 1)] + (j & 1) * 2;
                    split2(x[0], x[1], p[t][j], groups(t) == 1 ? p[t][j + 1] : low[t][j]);
                }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t f[4];
                ldsm4_t(f, vs + (kb * 16 + vrow) * (D * 2) + (((i * 2 + vch) ^ (lane & 7)) << 4));
#pragma unroll
                for (int t = 0; t < M; ++t) {
                    mma16816(o[t][2 * i], p[t], f[0], f[1]);
                    mma16816(o[t][2 * i + 1], p[t], f[2], f[3]);
                    if (groups(t) == 2) {
                        mma16816(o[t][2 * i], low[t], f[0], f[1]);
                        mma16816(o[t][2 * i + 1], low[t], f[2], f[3]);
                    }
                }
            }
        }
    }

    __device__ __forceinline__ void end() {
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int r = 0; r < groups(t); ++r) {
                l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 1);
                l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 2);
            }
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int i = 0; groups(t) == 1 && i < D / 8; ++i) {
                o[t][i][0] += o[t][i][2];
                o[t][i][1] += o[t][i][3];
            }
    }
    // rows round * kMerge .. + kMerge of this warp
    __device__ __forceinline__ void put(int round, float *rows, float2 *ml) const {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int r = 0; r < groups(t); ++r)
                if (t * 2 + r == round) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        *reinterpret_cast<float2 *>(rows + g * D + merge_chunk(i * 2 + (c >> 2), g) * 4 +
                                                    (c & 2)) =
                            make_float2(o[t][i][2 * r], o[t][i][2 * r + 1]);
                    if ((lane & 3) == 0) ml[g] = make_float2(m[t][r], l[t][r]);
                }
    }
};

// ---- fp32: CUDA cores, two-lane arithmetic.  A group of eight lanes takes a key
// (four keys at a time), each lane 16 bytes of every 128, for all rows; the eight
// lanes' partial scores are summed so that lane i of the group ends with row i's
// (each step halves the rows a lane keeps: kRows - 1 shuffles instead of 3 kRows),
// and the softmax of a row is one lane's.  The weights pass through shared memory,
// doubled for the two-lane products, and for P V a lane owns four dimensions (with
// D = 64 the half-warps take alternate halves of the tile's keys).
template <int D, int kRows> struct TileF32 {
    using T = float;
    static constexpr int kKeys = kTileBytes / (D * 4), kSwz = 0, kMerge = 4;
    static constexpr int QC = D / 32, KG = kKeys / 4, LPR = D / 4;   // lanes per V row
    static constexpr int VK = kKeys * LPR / 32;                        // V rows per lane
    uint64_t q[kRows][2 * QC];
    uint64_t o[kRows][2];
    float m, l;                               // of row lane % kRows

    __device__ __forceinline__ void begin(const PagedArgs &A, int b, int head0, int heads) {
        const int lane = threadIdx.x & 31;
        const float *base = static_cast<const float *>(A.q) + ((int64_t)b * A.Hq + head0) * D;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int i = 0; i < QC; ++i) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < heads) x = *reinterpret_cast<const float4 *>(base + r * D + i * 32 + (lane & 7) * 4);
                q[r][2 * i] = f2_pack(x.x, x.y);
                q[r][2 * i + 1] = f2_pack(x.z, x.w);
            }
            o[r][0] = o[r][1] = f2_pack(0.f, 0.f);
        }
        m = -INFINITY;
        l = 0.f;
    }

    __device__ __forceinline__ void tile(uint32_t ks_, uint32_t vs_, uint32_t valid, float scale,
                                         float *ps) {
        const int lane = threadIdx.x & 31, l8 = lane & 7, kg = lane >> 3;
        const ulonglong2 *ks = static_cast<const ulonglong2 *>(__cvta_shared_to_generic(ks_));
        const ulonglong2 *vs = static_cast<const ulonglong2 *>(__cvta_shared_to_generic(vs_));
        float s[KG];                          // of this lane's row
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            ulonglong2 x[QC];
#pragma unroll
            for (int i = 0; i < QC; ++i) x[i] = ks[((k * 4 + kg) * D + i * 32 + l8 * 4) / 4];
            float a[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                uint64_t acc = f2_mul(q[r][0], x[0].x);
                acc = f2_fma(q[r][1], x[0].y, acc);
#pragma unroll
                for (int i = 1; i < QC; ++i) {
                    acc = f2_fma(q[r][2 * i], x[i].x, acc);
                    acc = f2_fma(q[r][2 * i + 1], x[i].y, acc);
                }
                const float2 f = f2_unpack(acc);
                a[r] = f.x + f.y;
            }
            // lane i keeps the rows whose bit agrees with its own, and sends the others
#pragma unroll
            for (int w = kRows / 2; w > 0; w >>= 1) {
                const bool up = (l8 & w) != 0;
#pragma unroll
                for (int r = 0; r < w; ++r) {
                    const float send = up ? a[r] : a[r + w], keep = up ? a[r + w] : a[r];
                    a[r] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
            }
#pragma unroll
            for (int w = kRows; w < 8; w <<= 1) a[0] += __shfl_xor_sync(0xffffffffu, a[0], w);
            s[k] = (valid >> (k * 4 + kg)) & 1u ? a[0] * scale : -INFINITY;
        }
        float top = s[0];
#pragma unroll
        for (int k = 1; k < KG; ++k) top = fmaxf(top, s[k]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const bool grow = top > m + 8.f;
        if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? ex2(m - top) : 1.f;
            if (grow) m = top;
            l *= f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float fr = __shfl_sync(0xffffffffu, f, r);
                o[r][0] = f2_mul(o[r][0], f2_pack(fr, fr));
                o[r][1] = f2_mul(o[r][1], f2_pack(fr, fr));
            }
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            const float p = ex2(s[k] - ref);
            l += p;
            if (l8 < kRows)
                *reinterpret_cast<float2 *>(ps + (l8 * kKeys + k * 4 + kg) * 2) = make_float2(p, p);
        }
        __syncwarp();
        const int k0 = LPR == 32 ? 0 : (lane / LPR) * VK;
#pragma unroll
        for (int k = 0; k < VK; k += 2) {
            const ulonglong2 x = vs[((k0 + k) * D + (lane % LPR) * 4) / 4];
            const ulonglong2 y = vs[((k0 + k + 1) * D + (lane % LPR) * 4) / 4];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(ps + (r * kKeys + k0 + k) * 2);
                o[r][0] = f2_fma(p.x, x.x, o[r][0]);
                o[r][1] = f2_fma(p.x, x.y, o[r][1]);
                o[r][0] = f2_fma(p.y, y.x, o[r][0]);
                o[r][1] = f2_fma(p.y, y.y, o[r][1]);
            }
        }
        __syncwarp();
    }

    __device__ __forceinline__ void end() {
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (LPR == 16) {
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 f = f2_unpack(o[r][j]);
                    o[r][j] = f2_pack(f.x + __shfl_xor_sync(0xffffffffu, f.x, 16),
                                      f.y + __shfl_xor_sync(0xffffffffu, f.y, 16));
                }
        }
    }
    __device__ __forceinline__ void put(int round, float *rows, float2 *ml) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (r / kMerge == round && lane < LPR)
                *reinterpret_cast<ulonglong2 *>(rows + (r % kMerge) * D +
                                                merge_chunk(lane, r % kMerge) * 4) =
                    make_ulonglong2(o[r][0], o[r][1]);
        if (lane < kRows && lane / kMerge == round) ml[lane % kMerge] = make_float2(m, l);
    }
};

template <typename Tile, int D> constexpr size_t smem_bytes() {
    return (size_t)kWarps * kStages * 2 * kTileBytes + (size_t)kWarps * Tile::kMerge * D * 4;
}

template <typename T> __device__ __forceinline__ void put4(T *p, float4 x);
template <> __device__ __forceinline__ void put4<float>(float *p, float4 x) {
    *reinterpret_cast<float4 *>(p) = x;
}
template <> __device__ __forceinline__ void put4<__nv_bfloat16>(__nv_bfloat16 *p, float4 x) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
}

constexpr float kLn2 = 0.693147180559945f;

// The rows of empty sequences, shared out over the CTAs; bad lengths are reported here.
template <typename T, int D>
__device__ __forceinline__ void empty_rows(const PagedArgs &A, const Split &S) {
    for (int b = blockIdx.x; b < A.B; b += gridDim.x) {
        if (visible(A, b).n) continue;
        if (threadIdx.x == 0 && A.lens[b] != 0) atomicExch(&g_paged_error, (int)HGA_ERR_BOUNDS);
        T *o = static_cast<T *>(A.out) + (int64_t)b * A.Hq * D;
        for (int i = threadIdx.x; i < A.Hq * D / 4; i += kThreads)
            put4<T>(o + i * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        for (int h = threadIdx.x; A.lse && h < A.Hq; h += kThreads)
            A.lse[(int64_t)b * A.Hq + h] = -INFINITY;
        if (S.by_item)
            for (int i = threadIdx.x; i < S.items * S.gsplit; i += kThreads)
                S.join[(int64_t)b * S.items * S.gsplit + i] = make_int4(0, 0, -1, -1);
    }
}

// kHw: adjacent KV heads of a CTA; the warps of a head take its tiles in turn.
template <typename Tile, int D, int kRows, int kHw>
__global__ void __launch_bounds__(kThreads, 2) k_paged_decode(const PagedArgs A, const Split S) {
    using T = typename Tile::T;
    constexpr int kKeys = Tile::kKeys, kCpr = D * (int)sizeof(T) / 16, kLoads = kTileBytes / 512;
    extern __shared__ __align__(1024) char ring[];
    __shared__ int start[6];       // of the CTA's first unit: b, item, unit; the row's Visible
    __shared__ int sums[kWarps];
    __shared__ uint32_t valid[kWarps][kStages];
    __shared__ float2 ml[kWarps][Tile::kMerge];
    __shared__ __align__(16) float ps[sizeof(T) == 4 ? kWarps * kRows * kKeys * 2 : 1];
    float *merge = reinterpret_cast<float *>(ring + kWarps * kStages * 2 * kTileBytes);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const int range = cta / S.gsplit, chunk = cta % S.gsplit;
    const int g0 = chunk * S.gch, heads = min(S.gch, A.G - g0);
    constexpr int kKw = kWarps / kHw;
    const int hsub = warp % kHw, ksub = warp / kHw;        // the warp's head, and its tiles
    const int uk = kUnitTiles * kKeys;
    // ---- where this CTA's units begin: sums over runs of sequences, one per thread
    const int per = (A.B + kThreads - 1) / kThreads;
    const int r0 = min(A.B, tid * per), r1 = min(A.B, r0 + per);
    int mine = 0;
    Visible v = {0, 0, 0};
    for (int b = r0; b < r1; ++b) {
        v = visible(A, b);
        mine += units_of(v.n, uk) * S.items;
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int before = upto - mine, U = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        U += sums[w];
    }
    // with fewer units than CTAs the last ones take none, so that a split item's
    // parts lie in CTAs without a gap
    const int n = min(U, S.n);
    // floor(U i / n) = U / n i + (U mod n) i / n, whose products fit 32 bits
    const int each = n ? U / n : 0, rest = n ? U - each * n : 0;
    auto begin_of = [&](int i) { return each * i + rest * i / n; };
    const int u0 = range < n ? begin_of(range) : 0, u1 = range < n ? begin_of(range + 1) : 0;
    if (u0 < u1 && u0 >= before && u0 < before + mine) {
        int at = u0 - before;
        for (int b = r0; b < r1; ++b) {
            if (per > 1) v = visible(A, b);
            const int nu = units_of(v.n, uk);
            if (at < nu * S.items) {
                start[0] = b;
                start[1] = at / nu;
                start[2] = at % nu;
                start[3] = v.s, start[4] = v.lo, start[5] = v.n;
                break;
            }
            at -= nu * S.items;
        }
    }
    __syncthreads();
    if (u0 >= u1) {
        if (tid == 0 && !S.by_item) S.join[cta] = make_int4(0, 0, -1, -1);
        empty_rows<T, D>(A, S);
        return;
    }

    Walk C;
    C.b = start[0], C.it = start[1], C.u = start[2];
    C.left = u1 - u0;
    C.v = {start[3], start[4], start[5]};
    C.nu = units_of(C.v.n, uk);
    C.take();
    Walk P = C;
    char *kring = ring + warp * kStages * 2 * kTileBytes;
    const uint32_t ring_s = sm100::smem_addr(kring);
    const int64_t row_bytes = (int64_t)A.Hkv * D * (int)sizeof(T);
    const int page_mask = (1 << A.log2_page) - 1;

    // ---- producer: the next tile's page entries are read one tile ahead of its rows
    auto keys = [&](const Walk &w) { return key_walk(w.u, w.cnt, w.nu, w.v.n, uk, ksub, kKw, kKeys); };
    KeyWalk pk = keys(P);
    bool plive = true;                              // false: no tile left
    int ptok = 0, ppage = 0, phead = 0;
    bool pin = false;
    auto fetch = [&]() {
        while (!pk.more()) {
            if (!P.next(A, S, uk)) {
                plive = false;
                return;
            }
            pk = keys(P);
        }
        const unsigned key = pk.key(lane & (kKeys - 1), pin);
        ptok = (int)(key < (unsigned)P.v.s ? key : key - (unsigned)P.v.s + (unsigned)P.v.lo);
        ppage = pin ? A.table[(int64_t)P.b * A.max_pages + (ptok >> A.log2_page)] : 0;
        phead = P.it * kHw + hsub;
        pk.next();
    };
    auto issue = [&](int stage) {
        if (plive) {
            const bool ok = pin && (unsigned)ppage < (unsigned)A.num_pages;
            if (pin && !ok) atomicExch(&g_paged_error, (int)HGA_ERR_BOUNDS);
            const int slot = ok ? (ppage << A.log2_page) + (ptok & page_mask) : -1;
            const uint32_t bits = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) valid[warp][stage] = kKeys == 32 ? bits : bits & ((1u << (kKeys & 31)) - 1u);
            const char *kb = static_cast<const char *>(A.k) + (int64_t)phead * D * sizeof(T);
            const char *vb = static_cast<const char *>(A.v) + (int64_t)phead * D * sizeof(T);
            const uint32_t dst = ring_s + stage * 2 * kTileBytes;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int row = (j * 32 + lane) / kCpr, ch = (j * 32 + lane) % kCpr;
                const int sl = __shfl_sync(0xffffffffu, slot, row);
                const int64_t off = (sl < 0 ? 0 : (int64_t)sl * row_bytes) + ch * 16;
                const uint32_t to = dst + row * (kCpr * 16) + ((ch ^ (row & Tile::kSwz)) << 4);
                cp16(to, kb + off, sl >= 0);
                cp16(to + kTileBytes, vb + off, sl >= 0);
            }
            fetch();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // while the first tiles are on their way
    empty_rows<T, D>(A, S);

    // ---- consumer
    Tile t;
    int stage = 0;
    int4 joined = make_int4(0, 0, -1, -1);
    int done = 0;                                   // units before the segment
    t.begin(A, C.b, (C.it * kHw + hsub) * A.G + g0, heads);
    for (bool more = true; more;) {
        const int h0 = C.it * kHw, b = C.b;
        for (KeyWalk k = keys(C); k.more(); k.next()) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();
            issue(stage == 0 ? kStages - 1 : stage - 1);
            const uint32_t ks = ring_s + stage * 2 * kTileBytes;
            t.tile(ks, ks + kTileBytes, valid[warp][stage], A.scale_log2,
                   ps + (sizeof(T) == 4 ? warp * kRows * kKeys * 2 : 0));
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        t.end();
        // ---- the segment's rows: merged over the warps, then out or parked
        const bool cont = C.u > 0, open = C.u + C.cnt < C.nu, whole = !cont && !open;
        const int64_t row_at = ((int64_t)cta * 2 + (cont ? 0 : 1)) * S.rows;
        if (!cont) {
            if (open) {
                // the range that holds the item's last unit: a guess, put right
                const int last = u0 + done + C.nu - 1;
                int r = min(n - 1, (int)((float)last * (float)n / (float)U));
                while (begin_of(r) > last) --r;
                while (r + 1 < n && begin_of(r + 1) <= last) ++r;
                joined = make_int4(b, C.it, range, r);
            }
            if (S.by_item && tid == 0)
                S.join[((int64_t)b * S.items + C.it) * S.gsplit + chunk] = joined;
        }
        done += C.cnt;
        constexpr int kRounds = (kRows + Tile::kMerge - 1) / Tile::kMerge;
#pragma unroll
        for (int round = 0; round < kRounds; ++round) {
            t.put(round, merge + warp * Tile::kMerge * D, ml[warp]);
            if (round == kRounds - 1) {
                // the next segment's queries come while this one's rows are merged
                more = C.next(A, S, uk);
                if (more) t.begin(A, C.b, (C.it * kHw + hsub) * A.G + g0, heads);
            }
            __syncthreads();
            for (int e = tid; e < kHw * Tile::kMerge * (D / 4); e += kThreads) {
                const int ch = e % (D / 4), d = ch * 4, r = e / (D / 4) % Tile::kMerge;
                const int hs = e / (D / 4 * Tile::kMerge), row = round * Tile::kMerge + r;
                if (row >= heads) continue;
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kKw; ++k) top = fmaxf(top, ml[k * kHw + hs][r].x);
                const float ref = top == -INFINITY ? 0.f : top;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < kKw; ++k) {
                    const int w = k * kHw + hs;
                    const float f = ex2(ml[w][r].x - ref);
                    const float4 x = *reinterpret_cast<const float4 *>(
                        merge + (w * Tile::kMerge + r) * D + merge_chunk(ch, r) * 4);
                    sum = fmaf(ml[w][r].y, f, sum);
                    a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y);
                    a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
                }
                if (whole) {
                    const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
                    const int64_t at = (int64_t)b * A.Hq + (h0 + hs) * A.G + g0 + row;
                    put4<T>(static_cast<T *>(A.out) + at * D + d,
                            make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
                    if (A.lse && d == 0) A.lse[at] = (top + log2f(sum)) * kLn2;
                } else {
                    const int64_t at = row_at + hs * S.gch + row;
                    *reinterpret_cast<float4 *>(S.part + at * D + d) = a;
                    if (d == 0) S.ml[at] = make_float2(top, sum);
                }
            }
            __syncthreads();
        }
    }
    if (!S.by_item && tid == 0) S.join[cta] = joined;
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Adds up the parts of the items that were split, in CTA order; a programmatic
// dependent of k_paged_decode.  grid: (possible split items, rows).  Latency
// bound: an item of up to kFew parts is joined by its first CTA, a group of D / 4
// lanes per row and four parts loaded at a time; beyond that every row has its
// CTA, whose groups share the parts.  (Whole calls, caches cold: 96 rows of 640 keys,
// 384 items of 2 or 3 parts, 32 us, 40 with a CTA per row; 1 x 32K, 4 items of 74
// parts, 20.5 us, 32.7 with a CTA per item; fp32 5 x 2K, 20 items of up to 15 parts,
// 11.3 and 10.4.)
constexpr int kJoinThreads = 256, kAhead = 8, kFew = 16;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const PagedArgs A, const Split S) {
    constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
    __shared__ float2 w[kMaxCtas];
    __shared__ float red[kJoinThreads / 32];
    __shared__ float4 acc[kGroups][kLanes];
    __shared__ float sum_s;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int4 j = S.join[blockIdx.x];
    if (j.z < 0) return;
    const int chunk = blockIdx.x % S.gsplit, b = j.x, h0 = j.y * S.hw, g0 = chunk * S.gch;
    const int tid = threadIdx.x, cnt = j.w - j.z + 1, heads = min(S.gch, A.G - g0);
    const int lane = tid % kLanes, grp = tid / kLanes;
    // rows: hw heads of gch query heads, of which `heads` exist
    auto out = [&](int row, float4 a, float top, float sum) {
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
        const int64_t to = (int64_t)b * A.Hq + (h0 + row / S.gch) * A.G + g0 + row % S.gch;
        put4<T>(static_cast<T *>(A.out) + to * D + lane * 4,
                make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
        if (A.lse && lane == 0) A.lse[to] = (top + log2f(sum)) * kLn2;
    };
    if (cnt <= kFew) {
        if (blockIdx.y) return;
        for (int row = grp; row < S.rows; row += kGroups) {
            if (row % S.gch >= heads) continue;
            float top = -INFINITY, sum = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < cnt; i0 += 4) {
                float4 x[4];
                float2 y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = i0 + k;
                    const int64_t at = (((int64_t)(j.z + i) * S.gsplit + chunk) * 2 + (i == 0)) * S.rows + row;
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    y[k] = make_float2(-INFINITY, 0.f);
                    if (i < cnt) {
                        x[k] = *reinterpret_cast<const float4 *>(S.part + at * D + lane * 4);
                        y[k] = S.ml[at];
                    }
                }
                const float up = fmaxf(fmaxf(fmaxf(y[0].x, y[1].x), fmaxf(y[2].x, y[3].x)), top);
                const float ref = up == -INFINITY ? 0.f : up, f0 = ex2(top - ref);
                top = up;
                sum *= f0;
                a.x *= f0, a.y *= f0, a.z *= f0, a.w *= f0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f = ex2(y[k].x - ref);
                    sum = fmaf(y[k].y, f, sum);
                    a.x = fmaf(x[k].x, f, a.x), a.y = fmaf(x[k].y, f, a.y);
                    a.z = fmaf(x[k].z, f, a.z), a.w = fmaf(x[k].w, f, a.w);
                }
            }
            out(row, a, top, sum);
        }
        return;
    }
    const int row = blockIdx.y;
    if (row % S.gch >= heads) return;
    auto at = [&](int i) {
        return (((int64_t)(j.z + i) * S.gsplit + chunk) * 2 + (i == 0)) * S.rows + row;
    };
    // the first kAhead parts of a thread are on their way while the weights are formed
    float4 x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = grp + k * kGroups;
        x[k] = i < cnt ? *reinterpret_cast<const float4 *>(S.part + at(i) * D + lane * 4)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = -INFINITY;
    for (int i = tid; i < cnt; i += kJoinThreads) {
        const float2 y = S.ml[at(i)];
        w[i] = y;
        top = fmaxf(top, y.x);
    }
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, red[i]);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = grp + k * kGroups;
        const float f = i < cnt ? ex2(w[i].x - ref) : 0.f;
        a.x = fmaf(x[k].x, f, a.x), a.y = fmaf(x[k].y, f, a.y);
        a.z = fmaf(x[k].z, f, a.z), a.w = fmaf(x[k].w, f, a.w);
    }
#pragma unroll 4
    for (int i = grp + kAhead * kGroups; i < cnt; i += kGroups) {
        const float4 y = *reinterpret_cast<const float4 *>(S.part + at(i) * D + lane * 4);
        const float f = ex2(w[i].x - ref);
        a.x = fmaf(y.x, f, a.x), a.y = fmaf(y.y, f, a.y);
        a.z = fmaf(y.z, f, a.z), a.w = fmaf(y.w, f, a.w);
    }
    acc[grp][lane] = a;
    if (tid < 32) {
        float s = 0.f;
        for (int i = tid; i < cnt; i += 32) s = fmaf(w[i].y, ex2(w[i].x - ref), s);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) sum_s = s;
    }
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 y = acc[i][lane];
        a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
    }
    out(row, a, top, sum_s);
}

Split make_split(int B, int Hq, int Hkv, int D, int dtype) {
    Split S = {};
    const int G = Hq / Hkv, most = dtype == HGA_F32 ? 8 : D == 64 ? 32 : 16;
    // Runs of 256 bytes: bf16 heads of 64 are taken in pairs (64 x 16K tokens of 8
    // heads: 366 us one by one, 320 in pairs); for rows of 256 bytes and more one head
    // a CTA is faster, as four times the parts cost more than longer runs give (16 x
    // 64K tokens of 4 heads of 128: 316 us against 326 for four heads).
    S.hw = D * (dtype == HGA_BF16 ? 2 : 4) < 256 && Hkv % 2 == 0 ? 2 : 1;
    // More query heads than registers hold rows for (bf16 heads of 64: 32, of 128: 16;
    // fp32: 8) are cut into chunks; the CTAs of a range's chunks run side by side, so
    // that the second reads K and V from L2.
    S.gsplit = (G + most - 1) / most;
    S.gch = (G + S.gsplit - 1) / S.gsplit;
    S.gsplit = (G + S.gch - 1) / S.gch;
    S.items = Hkv / S.hw;
    S.rows = S.hw * S.gch;
    S.by_item = (long long)B * S.items * S.gsplit <= kMaxCtas;
    return S;
}

// CTAs of a call at most: two per SM, and at least one range
inline int max_ctas(const Split &S) { return std::max(kMaxCtas, S.gsplit); }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename Tile, int D, int kRows, int kHw>
hga_status run(const PagedArgs &A, const Split &S, cudaStream_t st) {
    auto *k = k_paged_decode<Tile, D, kRows, kHw>;
    const size_t smem = smem_bytes<Tile, D>();
    cudaError_t e = ensure_smem((const void *)k, smem);
    if (e != cudaSuccess) return cuda_status(e);
    e = launch_dependent(k, dim3(S.n * S.gsplit), dim3(kThreads), smem, st, A, S);
    if (e != cudaSuccess) return cuda_status(e);
    const int entries = (S.by_item ? A.B * S.items : S.n) * S.gsplit;
    return cuda_status(launch_dependent(k_paged_join<typename Tile::T, D>, dim3(entries, S.rows),
                                        dim3(kJoinThreads), 0, st, A, S));
}

}  // namespace

size_t paged_decode_workspace_bytes(int B, int Hq, int Hkv, int D, int dtype) {
    const Split S = make_split(B, Hq, Hkv, D, dtype);
    const size_t rows = (size_t)max_ctas(S) * 2 * S.rows;
    return up256(rows * D * 4) + up256(rows * sizeof(float2)) + up256(max_ctas(S) * sizeof(int4));
}

hga_status launch_paged_decode(const PagedArgs &A, int dtype, int D, void *ws, cudaStream_t st) {
    Split S = make_split(A.B, A.Hq, A.Hkv, D, dtype);
    const size_t rows = (size_t)max_ctas(S) * 2 * S.rows;
    char *p = static_cast<char *>(ws);
    S.part = reinterpret_cast<float *>(p);
    p += up256(rows * D * 4);
    S.ml = reinterpret_cast<float2 *>(p);
    p += up256(rows * sizeof(float2));
    S.join = reinterpret_cast<int4 *>(p);
    // no more CTAs than there can be units: the longest row a sequence may have
    long long most = (long long)A.max_pages << A.log2_page;
    if (A.window > 0) most = std::min(most, (long long)A.window + A.sinks);
    const int uk = kUnitTiles * (kTileBytes / (D * (dtype == HGA_BF16 ? 2 : 4)));
    const long long units = (most + uk - 1) / uk * S.items * A.B;
    if (units > 0x7fffffffLL) return HGA_ERR_UNSUPPORTED;       // the kernel counts them in 32 bits
    S.n = (int)std::max(1ll, std::min(units, (long long)std::min(2 * sm_count(), kMaxCtas) / S.gsplit));
    if (dtype == HGA_BF16) {
        if (D == 128)
            return S.gch > 8 ? run<TileBf16<128, 16>, 128, 16, 1>(A, S, st)
                             : run<TileBf16<128, 8>, 128, 8, 1>(A, S, st);
        if (S.hw == 2)
            return S.gch > 24   ? run<TileBf16<64, 32>, 64, 32, 2>(A, S, st)
                   : S.gch > 16 ? run<TileBf16<64, 24>, 64, 24, 2>(A, S, st)
                   : S.gch > 8  ? run<TileBf16<64, 16>, 64, 16, 2>(A, S, st)
                                : run<TileBf16<64, 8>, 64, 8, 2>(A, S, st);
        return S.gch > 24   ? run<TileBf16<64, 32>, 64, 32, 1>(A, S, st)
               : S.gch > 16 ? run<TileBf16<64, 24>, 64, 24, 1>(A, S, st)
               : S.gch > 8  ? run<TileBf16<64, 16>, 64, 16, 1>(A, S, st)
                            : run<TileBf16<64, 8>, 64, 8, 1>(A, S, st);
    }
    if (D == 128)
        return S.gch > 4 ? run<TileF32<128, 8>, 128, 8, 1>(A, S, st)
                         : run<TileF32<128, 4>, 128, 4, 1>(A, S, st);
    return S.gch > 4 ? run<TileF32<64, 8>, 64, 8, 1>(A, S, st)
                     : run<TileF32<64, 4>, 64, 4, 1>(A, S, st);
}

cudaError_t paged_error_word(int **word) { return cudaGetSymbolAddress((void **)word, g_paged_error); }

}  // namespace hga
