// Internal interface of the experts' products (experts*.cu): sizes, workspace
// views, and the routing that turns ids [N x r] into one segment of rows per
// expert.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace gmmb {

// Rows of one expert's segment start at a multiple of kExpTile, so that a
// tile of rows belongs to one expert.
constexpr int kExpTile = 128;
// Pairs per histogram of the routing's sort: short runs for latency, longer
// ones with many experts, so that the histograms stay within four words a pair.
inline int exp_chunk(int K) { return K < 256 ? 64 : K < 1024 ? 256 : 1024; }

struct ExpShape {
    int64_t N, P;   // points; (point, entry) pairs, N * max(r, 1)
    int d, h, o, K, r, gh;   // gh: rows of W1 (2h when gated)
    gmm_dtype dt;
    int act;
    bool gated, mlp, dense;
    // one entry per point: a pair's row of the last product is the point's
    // row of the result, and no sum over entries follows
    __host__ __device__ bool direct() const { return r <= 1; }
    __host__ __device__ int first() const { return mlp ? gh : o; }   // width of the first product
};

// Rows per expert from which a product's tile is two 128-row tiles of one
// segment on a pair of CTAs.
constexpr int64_t kExpPairRows = 384;

// Device view of the routing.  Tile t of 128 rows holds rows 128 t .. of its
// expert; a tile of 256 rows is two of those, the second possibly past the
// segment.
struct ExpRoute {
    int *cnt;           // [K + 1] pairs of each expert; [K]: points without any (direct only)
    int *seg;           // [K + 2] first row of each segment
    int4 *tile_at;      // [max_tiles] expert, first row, valid rows of each 128-row tile
    int4 *pair_at;      // [max_tiles] the same of each 256-row tile
    int *ntiles;        // [2] 128-row and 256-row tiles
    int *row_pair;      // [max rows] pair of each valid row
    int *hist;          // [chunks x (K + 1)]
    int chunk;          // pairs per chunk, a multiple of 64
    const int32_t *ids; // NULL: dense
    int64_t N, P;
    int K, r;
    int max_tiles;      // of 128 rows
    int tile_rows;      // of the products' tiles

    struct Tile { int expert, valid; int64_t row0; };
    __device__ __forceinline__ int tiles(int rows = kExpTile) const {
        return ids ? ntiles[rows == kExpTile ? 0 : 1] : (int)((N + rows - 1) / rows);
    }
    // a tile's entry, loaded, and what it says
    __device__ __forceinline__ int4 tile_entry(int t, int rows = kExpTile) const {
        if (ids) return rows == kExpTile ? tile_at[t] : pair_at[t];
        const int64_t left = N - (int64_t)t * rows;
        return make_int4(0, t * rows, left < rows ? (int)left : rows, 0);
    }
    __device__ __forceinline__ Tile tile(int t, int rows = kExpTile) const {
        const int4 e = tile_entry(t, rows);
        return Tile{e.x, e.z, e.y};
    }
    __device__ __forceinline__ int64_t pair(int64_t row) const {
        return ids ? row_pair[row] : row;
    }
    // pairs of more than one entry a point fit 31 bits
    __device__ __forceinline__ int64_t token(int64_t p) const {
        return r > 1 ? (uint32_t)p / (uint32_t)r : p;
    }
    __device__ __forceinline__ bool used(int64_t p) const {
        return !ids || (ids[p] >= 0 && ids[p] < K);
    }
};

// Everything a launch needs: the caller's arrays and the workspace views.
// The first layer's arrays are those of gmm_expert_linear too.
struct ExpCall {
    ExpShape s;
    ExpRoute rt;
    int *err;
    const void *x, *dy, *w1, *b1, *w2, *b2, *res;
    const float *resp;
    void *y, *dx, *dw1, *db1, *dw2, *db2;
    float *dresp;
    // workspace: rows of the hidden vector (forward) or of resp * h
    // (backward), of the first layer's pre-activation gradient, per-pair
    // results before the sum over entries, and partial sums of dresp
    void *hid, *da;
    // rows of X and dY sorted by expert, zeros past each segment (tensor
    // cores; the arrays themselves in the dense form), and how many
    void *xrows, *dyrows;
    int64_t point_rows;
    int64_t da_rows;    // rows of da's array
    // linear form without activation and weights: the pre-activations'
    // gradient is dY itself, and nothing has to be computed again
    __host__ __device__ bool plain_da() const {
        return !s.mlp && s.act == GMM_ACT_NONE && !resp;
    }
    float *slots, *rpart, *colpart;
    int64_t max_rows;
    int nrpart;         // partial sums of dresp per pair
    size_t esize;       // bytes per element of hid and da
    int units;          // hidden units that exist (padded copies have more); linear: no limit
};

// The activation and its derivative.
template <int ACT> __device__ __forceinline__ void act_both(float z, float &f, float &df) {
    if (ACT == GMM_ACT_RELU) {
        f = z > 0.f ? z : (z <= 0.f ? 0.f : z);   // NaN stays NaN
        df = z > 0.f ? 1.f : 0.f;
    } else if (ACT == GMM_ACT_GELU) {
        const float cdf = 0.5f * erfcf(-0.70710678f * z);
        f = z * cdf;
        df = fmaf(z, 0.39894228f * expf(-0.5f * z * z), cdf);
    } else if (ACT == GMM_ACT_SILU) {
        const float p = 1.f / (1.f + expf(-z));
        f = z * p;
        df = p * fmaf(z, 1.f - p, 1.f);
    } else {
        f = z;
        df = 1.f;
    }
}
template <int ACT> __device__ __forceinline__ float act_of(float z) {
    float f, df;
    act_both<ACT>(z, f, df);
    return f;
}

// The same to fp32 precision of z rather than of f, for results that are
// rounded to 16 bits, two at a time (packed fp32 arithmetic): hardware
// exponential and reciprocal (2^-21), and for gelu erfc by Abramowitz and
// Stegun 7.1.26 (absolute error 1.5e-7), whose exponential is the density's
// too.  erfcf and expf take about 55 instructions an element, this 4 (silu)
// to 9 (gelu); a 4096 x 1024 x 4096 gelu map took 92 us with them and 73
// with scalar code of this form.
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_pair(float2 x) {
    float2 y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
    return y;
}
__device__ __forceinline__ float2 rcp_pair(float2 x) {
    float2 y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
    return y;
}
template <int ACT> __device__ __forceinline__ void act_pair(float2 z, float2 &f, float2 &df) {
    if (ACT == GMM_ACT_GELU) {
        const float2 az = make_float2(fabsf(z.x), fabsf(z.y));
        const float2 t = rcp_pair(__ffma2_rn(splat(0.3275911f * 0.70710678f), az, splat(1.f)));
        float2 p = __ffma2_rn(splat(1.061405429f), t, splat(-1.453152027f));
        p = __ffma2_rn(p, t, splat(1.421413741f));
        p = __ffma2_rn(p, t, splat(-0.284496736f));
        p = __ffma2_rn(p, t, splat(0.254829592f));
        // e = exp(-z^2 / 2); the tail 1 - Phi(|z|) = p t e / 2
        const float2 e = ex2_pair(__fmul2_rn(__fmul2_rn(z, splat(-0.72134752f)), z));
        const float2 tail = __fmul2_rn(__fmul2_rn(p, t), __fmul2_rn(e, splat(0.5f)));
        const float2 cdf = make_float2(z.x >= 0.f ? 1.f - tail.x : tail.x,
                                       z.y >= 0.f ? 1.f - tail.y : tail.y);
        f = __fmul2_rn(z, cdf);
        df = __ffma2_rn(z, __fmul2_rn(e, splat(0.39894228f)), cdf);
    } else if (ACT == GMM_ACT_SILU) {
        const float2 p = rcp_pair(__fadd2_rn(ex2_pair(__fmul2_rn(z, splat(-1.44269504f))),
                                             splat(1.f)));
        f = __fmul2_rn(z, p);
        // p (1 + z (1 - p)) = p + f - f p
        df = __fadd2_rn(p, __ffma2_rn(__fmul2_rn(f, splat(-1.f)), p, f));
    } else {
        act_both<ACT>(z.x, f.x, df.x);
        act_both<ACT>(z.y, f.y, df.y);
    }
}
template <int ACT> __device__ __forceinline__ float act_fast(float z) {
    float2 f, df;
    act_pair<ACT>(splat(z), f, df);
    return f.x;
}

template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_float<__half>(float v) {
    return __float2half_rn(v);
}
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// Every kernel of a call starts under the tail of the one before it
// (programmatic dependent launch) and waits here for all of it; what it does
// before this touches no memory of the call.
__device__ __forceinline__ void exp_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void exp_enter() {
    exp_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t exp_launch(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t s,
                       const A &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    note_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// experts_route.cu
cudaError_t launch_exp_route(const ExpCall &c, cudaStream_t s);
// the rows of X (and dY) sorted by expert (16-bit types, 16-byte rows)
cudaError_t launch_exp_gather(const ExpCall &c, bool backward, cudaStream_t s);
// forward: y_n = sum_i g_ni slots_ni (+ residual_n); backward: dx_n = sum_i
// slots_ni, and dresp from its partial sums (and <dy, b2>)
cudaError_t launch_exp_combine(const ExpCall &c, bool backward, cudaStream_t s);
// column sums of da and g dy
cudaError_t launch_exp_bias_grads(const ExpCall &c, cudaStream_t s);
int exp_colsum_slices(const ExpShape &s);
// experts_pad.cu: copies between [planes x rows x cols] and its zero-padded
// form [planes x rows_to x cols_to] (16-bit elements, cols_to a multiple of 8)
struct PadJob {
    void *narrow, *wide;
    int planes, rows, cols, rows_to, cols_to;
    int per_expert;   // planes of an expert: planes of unused ones are left; 0: all
};
struct PadJobs {
    PadJob j[8];
    int n;
    const int *cnt;   // rows of each expert, NULL: all are used
};
cudaError_t launch_exp_pad(const PadJobs &jobs, bool back, cudaStream_t s);
// experts_simt.cu: the products on CUDA cores
cudaError_t launch_exp_simt(const ExpCall &c, bool backward, cudaStream_t s);
// experts_tc.cu: on the tensor cores (16-bit types, widths multiples of 8)
cudaError_t launch_exp_tc(const ExpCall &c, bool backward, cudaStream_t s);
// experts_few.cu: the whole forward call for few points
cudaError_t launch_exp_few(const ExpCall &c, cudaStream_t s);
// Points up to which that form runs: its sums of 16 outputs of every point
// stay in shared memory.
constexpr int64_t kExpFewPoints = 64;
int exp_tc_resp_parts(const ExpShape &s);

}  // namespace gmmb
