// Block tables, slot map and positions of a serving step, from the requests'
// lengths alone (hga_paged_plan).
//
// Whole-number prefix sums over the requests: of their new tokens (where each
// request's tokens lie in the packed batch) and of the pages they need (which
// entries of the free stack are theirs).  Bound by latency: a step of 256
// requests touches a few KB, so one CTA scans the requests and, up to
// kFillHere tokens, also fills the map; beyond that the fill is a grid of its
// own, a programmatic dependent (8 bytes written per token).
#include "paged_internal.cuh"

namespace hga {

__device__ int g_plan_error = 0;

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kFillHere = 2048;   // tokens the scanning CTA fills itself (4.5 us; 5.0 with a grid; 8192: 9.0, 4.9)
constexpr int kRun = 16;          // table entries a thread gives back at a time

__device__ __forceinline__ void bad() { atomicExch(&g_plan_error, (int)HGA_ERR_BOUNDS); }

// Exclusive sum of x over the CTA; total: the sum of all.  part: [kWarps + 1].
__device__ long long scan(long long x, long long *part, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += y;
    }
    __syncthreads();                       // the last call's part is read
    if (lane == 31) part[warp] = in;
    __syncthreads();
    if (warp == 0) {
        const long long w = part[lane];
        long long s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        part[lane] = s - w;
        if (lane == 31) part[kWarps] = s;
    }
    __syncthreads();
    total = part[kWarps];
    return part[warp] + in - x;
}
static_assert(kWarps == 32, "scan() sums the warps' totals with one warp");

// First index of [0, n) whose entry of the ascending list a (entry i + 1 is the
// end of i) lies beyond t; n if none.
__device__ __forceinline__ int find(const int32_t *a, int n, int t) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The same over the kThreads rows of `ends` (ends[0] = 0), without a branch, so that
// several searches run side by side.
__device__ __forceinline__ int find_row(const int32_t *ends, int e) {
    int lo = 0;
#pragma unroll
    for (int s = kThreads / 2; s > 0; s >>= 1) lo += ends[lo + s] <= e ? s : 0;
    return lo;
}

// Slot and position of packed token t, and the table entry if it opens a page.
// cu: cu_tokens, in shared memory where it fits.
__device__ __forceinline__ void fill(const PlanArgs &a, const int32_t *cu, int t) {
    const int b = find(cu, a.B, t);
    int slot = -1, pos = 0;
    if (b < a.B) {
        const int got = a.io.granted[b], at = a.io.lens_out[b] - got;
        pos = (int)((unsigned)at + (unsigned)(t - cu[b]));
        if (got > 0) {
            const int page = pos >> a.log2_page;
            const int held = (int)(((long long)at + (1 << a.log2_page) - 1) >> a.log2_page);
            int32_t *entry = a.io.block_table + (int64_t)b * a.max_pages + page;
            int id = page < held ? *entry : a.io.free_pages[a.first[b] - (page - held)];
            if ((unsigned)id >= (unsigned)a.num_pages) {
                id = -1;
                bad();
            }
            const int off = pos & ((1 << a.log2_page) - 1);
            if (page >= held && off == 0) *entry = id;
            if (id >= 0) slot = (id << a.log2_page) + off;
        }
    }
    a.io.slot[t] = slot;
    a.io.pos[t] = pos;
}

__global__ void __launch_bounds__(kThreads) k_plan_scan(const PlanArgs a, int fill_here) {
    __shared__ long long part[kWarps + 1];
    __shared__ int32_t ends[kThreads + 1];
    __shared__ int taken;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lg = a.log2_page, mask = (1 << lg) - 1;
    const long long cap = (long long)a.max_pages << lg;
    long long stack = *a.io.free_count, total;
    if (stack < 0 || stack > a.num_pages) {
        if (tid == 0) bad();
        stack = stack < 0 ? 0 : a.num_pages;
    }
    // ---- released rows give their pages back: the rows' entries in one line, kRun of
    // it a thread
    if (a.io.release)
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + tid;
            int give = 0;
            if (b < a.B && a.io.release[b]) {
                const int len = a.io.lens[b];
                if (len >= 0 && len <= cap) give = (int)(((long long)len + mask) >> lg);
            }
            const long long before = scan(give, part, total);
            ends[tid + 1] = (int)(before + give);
            if (tid == 0) ends[0] = 0;
            __syncthreads();
            const unsigned n = (unsigned)total;    // below 2^31, but n + a step is not
            auto entry = [&](int row, int e) {
                return a.io.block_table[(int64_t)(b0 + row) * a.max_pages + e - ends[row]];
            };
            for (unsigned e0 = 0; e0 < n; e0 += kThreads * kRun) {
                // a warp takes 32 kRun entries in a row: few rows, so one search and then
                // a look at the row's end
                const unsigned w0 = e0 + (tid >> 5) * 32 * kRun + (tid & 31);
                int ids[kRun], row = find_row(ends, (int)min(w0, n - 1));
                bool good = true;
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    const int e = (int)min(w0 + i * 32, n - 1);
                    if (ends[row + 1] <= e) row = find_row(ends, e);
                    ids[i] = entry(row, e);
                }
#pragma unroll
                for (int i = 0; i < kRun; ++i) good &= (unsigned)ids[i] < (unsigned)a.num_pages;
                const int many = (int)min(n - e0, (unsigned)(kThreads * kRun));
                if (__syncthreads_and(good) && stack + many <= a.num_pages) {
#pragma unroll
                    for (int i = 0; i < kRun; ++i)
                        if (w0 + i * 32 < n) a.io.free_pages[stack + (w0 - e0) + i * 32] = ids[i];
                    stack += many;
                    continue;
                }
                // bad ids are left out, and what the stack has no room for
                for (int i = 0; i < kRun; ++i) {
                    const unsigned e = e0 + i * kThreads + tid;
                    const int id = e < n ? entry(find_row(ends, (int)e), (int)e) : -1;
                    const bool ok = (unsigned)id < (unsigned)a.num_pages;
                    long long all, at = stack + scan(ok ? 1 : 0, part, all);
                    if (ok && at < a.num_pages) a.io.free_pages[at] = id;
                    if (e < n && (!ok || at >= a.num_pages)) bad();
                    stack = stack + all < a.num_pages ? stack + all : a.num_pages;
                }
            }
            __syncthreads();
        }
    // ---- tokens and pages of each row
    long long tokens = 0, pages = 0;
    if (tid == 0) taken = 0;             // read after the scans' barriers
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        int len = 0, add = 0, given = 0;
        bool fits = false;
        if (b < a.B) {
            len = a.io.lens[b];
            add = a.io.new_tokens[b];
            if (len < 0 || len > cap || add < 0) bad();
            else fits = true;
            if (a.io.release && a.io.release[b] && len >= 0 && len <= cap) len = 0;
            add = add < 0 ? 0 : add;
        }
        const long long begin = tokens + scan(add, part, total), end = begin + add;
        tokens += total;
        fits = fits && (long long)len + add <= cap && end <= a.n_slots;
        const long long held = ((long long)len + mask) >> lg;
        const long long need = fits ? (((long long)len + add + mask) >> lg) - held : 0;
        const long long from = pages + scan(need, part, total);
        pages += total;
        const bool ok = fits && (need == 0 || from + need <= stack);
        given = ok ? add : 0;
        // the rows served are the first of those that need pages, so what they take
        // ends where the last of them does
        if (ok && need) atomicMax(&taken, (int)(from + need));
        if (b < a.B) {
            a.io.lens_out[b] = len + given;
            a.io.granted[b] = given;
            a.first[b] = (int)(stack - 1 - from);
            const int32_t cu = (int32_t)(end < 0x7fffffffLL ? end : 0x7fffffffLL);
            a.io.cu_tokens[b + 1] = cu;
            if (b0 == 0) ends[tid + 1] = cu;
        }
    }
    __syncthreads();
    if (tid == 0) {
        a.io.cu_tokens[0] = 0;
        *a.io.free_count_out = (int32_t)(stack - taken);
        ends[0] = 0;
    }
    if (!fill_here) return;
    __syncthreads();
    const int32_t *cu = a.B <= kThreads ? ends : a.io.cu_tokens;
    for (int t = tid; t < a.n_slots; t += kThreads) fill(a, cu, t);
}

__global__ void __launch_bounds__(256) k_plan_fill(const PlanArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t < a.n_slots) fill(a, a.io.cu_tokens, t);
}

}  // namespace

size_t plan_workspace_bytes(int B, int) { return ((size_t)B * 4 + 255) & ~(size_t)255; }

hga_status launch_paged_plan(const PlanArgs &a, cudaStream_t st) {
    const bool here = a.n_slots <= kFillHere;
    const cudaError_t e =
        launch_dependent(k_plan_scan, dim3(1), dim3(kThreads), 0, st, a, here ? 1 : 0);
    if (e != cudaSuccess || here) return cuda_status(e);
    return cuda_status(launch_dependent(k_plan_fill, dim3((unsigned)((a.n_slots + 255LL) / 256)),
                                        dim3(256), 0, st, a));
}

cudaError_t plan_error_word(int **word) { return cudaGetSymbolAddress((void **)word, g_plan_error); }

}  // namespace hga
