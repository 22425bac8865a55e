// Internal declarations of the paged-cache operators: what paged_api.cu hands
// to the kernels after checking the arguments.
#pragma once

#include "hga_internal.cuh"

namespace hga {

// The rotation of one call: 64-bit turn rates of the pairs (as in Rope) and
// the magnitude.  Passed by value as a kernel parameter.
struct PairRope {
    unsigned long long turn[kMaxHalf];
    float magnitude;
    int R;             // rotary_dim
    int interleaved;
};

struct PlanArgs {
    int B, num_pages, log2_page, max_pages, n_slots;
    hga_paged_plan_io io;
    int32_t *first;    // [B] stack index of each row's first new page
};

struct QkArgs {
    int64_t tokens;
    int Hq, Hkv;
    hga_qk_io io;
    PairRope rope;
};

struct QkGradArgs {
    int64_t tokens;
    int Hq, Hkv;
    hga_qk_grad_io io;
    PairRope rope;
    float *part;       // [CTAs][2][D] partial sums of the weights' gradients
};

struct PagedArgs {
    int B, Hq, Hkv, G, num_pages, log2_page, max_pages;
    int window, sinks;
    float scale_log2;  // softmax scale * log2(e)
    const void *q, *k, *v;
    const int32_t *table, *lens;
    void *out;
    float *lse;
};

int sm_count();        // of the current device (0 without one)

size_t plan_workspace_bytes(int B, int n_slots);
hga_status launch_paged_plan(const PlanArgs &a, cudaStream_t st);
hga_status launch_qk_norm_rope(const QkArgs &a, int dtype, int D, cudaStream_t st);
size_t qk_grad_workspace_bytes(int D);
hga_status launch_qk_norm_rope_backward(const QkGradArgs &a, int dtype, int D, cudaStream_t st);
size_t paged_decode_workspace_bytes(int B, int Hq, int Hkv, int D, int dtype);
hga_status launch_paged_decode(const PagedArgs &a, int dtype, int D, void *ws, cudaStream_t st);

cudaError_t plan_error_word(int **word);
cudaError_t qk_error_word(int **word);
cudaError_t paged_error_word(int **word);

// Launch as a programmatic dependent of whatever precedes on the stream: the grid may
// start when that kernel's CTAs have all allowed it (or ended), and every kernel
// launched so waits (griddepcontrol.wait: the kernel before has completed and its
// writes are visible) before it touches global memory, so only its launch overlaps.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*k)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t st, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace hga
