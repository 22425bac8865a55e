// How a warp of the paged attention steps over the keys of a segment: tiles of
// `keys` keys, every `step`-th key on.  Plain C++ as well as CUDA, so that the CPU
// tests compile it too.
#pragma once

#ifdef __CUDACC__
#define HGA_WALK_HD __host__ __device__ __forceinline__
#else
#define HGA_WALK_HD inline
#endif

namespace hga {

// Keys are numbered in unsigned: an end is below 2^31 (a row's capacity is) and a step
// at most 128, so that what lies a step or a lane beyond the end does not wrap.
struct KeyWalk {
    unsigned at, end, step;          // first key of the next tile
    HGA_WALK_HD bool more() const { return at < end; }
    HGA_WALK_HD void next() { at += step; }
    // the key of a lane of the tile; live: it is one of the segment's
    HGA_WALK_HD unsigned key(int lane, bool &live) const {
        const unsigned k = at + (unsigned)lane;
        live = k < end;
        return k;
    }
};

// Units of uk keys that n keys take (n + uk need not fit 31 bits).
HGA_WALK_HD int units_of(int n, int uk) { return n / uk + (n % uk != 0); }

// The tiles of warp ksub (of kw that take turns) in units [u, u + cnt) of a row of n
// keys in nu units.
HGA_WALK_HD KeyWalk key_walk(int u, int cnt, int nu, int n, int uk, int ksub, int kw, int keys) {
    KeyWalk w;
    w.at = (unsigned)u * (unsigned)uk + (unsigned)(ksub * keys);
    w.end = u + cnt >= nu ? (unsigned)n : (unsigned)(u + cnt) * (unsigned)uk;
    w.step = (unsigned)(keys * kw);
    return w;
}

}  // namespace hga
