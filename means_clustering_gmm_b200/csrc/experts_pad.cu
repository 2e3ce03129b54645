// Zero-padded copies for 16-bit arrays whose widths are not multiples of 8.
//
// The tensor-core kernels read rows of whole 16-byte units.  With every width
// rounded up and zeros in the new rows and columns the padded problem has the
// same results in the old ones: padded contraction indices add products of
// zeros on both sides, and what a hidden unit that does not exist would get
// (0 times an infinity of the point is not 0) is set to 0 by the epilogue that
// forms it.  Only experts in use are copied.
// Bound by the copies: about three passes over the used weights, where the
// CUDA-core form of such a call multiplies 64-row tiles for a few points.
#include "experts.h"

namespace gmmb {

// A warp per line of the wide form, a lane per element: both sides are read
// and written in runs of 64 bytes.  (16 bytes a lane on the wide side left the
// other side with 2-byte accesses 16 bytes apart: a call that writes 800 MB of
// weight gradients took 1.93 ms, and takes 1.06.)
template <bool BACK>
__global__ void __launch_bounds__(256) exp_pad_kernel(PadJobs jobs) {
    exp_enter();
    const PadJob j = jobs.j[blockIdx.y];
    const int lane = threadIdx.x & 31;
    const int64_t lines = (int64_t)j.planes * j.rows_to;
    for (int64_t l = blockIdx.x * 8 + (threadIdx.x >> 5); l < lines; l += gridDim.x * 8) {
        const int plane = (int)(l / j.rows_to), row = (int)(l - (int64_t)plane * j.rows_to);
        uint16_t *wide = (uint16_t *)j.wide + l * j.cols_to;
        uint16_t *narrow = (uint16_t *)j.narrow + ((int64_t)plane * j.rows + row) * j.cols;
        if (BACK) {
            if (row >= j.rows) continue;
#pragma unroll 8
            for (int c = lane; c < j.cols; c += 32) narrow[c] = wide[c];
        } else {
            if (j.per_expert && jobs.cnt && jobs.cnt[plane / j.per_expert] == 0) continue;
            const int cols = row < j.rows ? j.cols : 0;
#pragma unroll 8
            for (int c = lane; c < j.cols_to; c += 32) wide[c] = c < cols ? narrow[c] : 0;
        }
    }
}

cudaError_t launch_exp_pad(const PadJobs &jobs, bool back, cudaStream_t s) {
    if (jobs.n == 0) return cudaSuccess;
    const dim3 grid(148 * 8, jobs.n);
    return back ? exp_launch(exp_pad_kernel<true>, grid, 256, 0, s, jobs)
                : exp_launch(exp_pad_kernel<false>, grid, 256, 0, s, jobs);
}

}  // namespace gmmb
