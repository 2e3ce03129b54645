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

// Device view of the routing.  Tile t holds rows [128 t, 128 t + valid).
struct ExpRoute {
    int *cnt;           // [K + 1] pairs of each expert; [K]: points without any (direct only)
    int *seg;           // [K + 2] first row of each segment
    int *tile_expert;   // [max tiles]
    int *ntiles;        // [1]
    int *row_pair;      // [max rows] pair of each valid row
    int *hist;          // [chunks x (K + 1)]
    const int32_t *ids; // NULL: dense
    int64_t N, P;
    int K, r;
    int max_tiles;

    struct Tile { int expert, valid; int64_t row0, seg_end; };
    __device__ __forceinline__ int tiles() const {
        return ids ? *ntiles : (int)((N + kExpTile - 1) / kExpTile);
    }
    __device__ __forceinline__ Tile tile(int t) const {
        Tile x;
        x.row0 = (int64_t)t * kExpTile;
        x.expert = ids ? tile_expert[t] : 0;
        x.seg_end = ids ? (int64_t)seg[x.expert] + cnt[x.expert] : N;
        const int64_t v = x.seg_end - x.row0;
        x.valid = v < kExpTile ? (int)v : kExpTile;
        return x;
    }
    __device__ __forceinline__ int64_t pair(int64_t row) const {
        return ids ? row_pair[row] : row;
    }
    __device__ __forceinline__ int64_t token(int64_t p) const { return r > 1 ? p / r : p; }
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
    float *slots, *rpart;
    int64_t max_rows;
    int nrpart;         // partial sums of dresp per row
    size_t esize;       // bytes per element of hid and da
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

// An ordinary load: the compiler keeps it behind the test that guards it,
// which it need not do with the inline assembly behind __ldg of 16-bit types.
template <typename T> __device__ __forceinline__ float value_at(const T *p) {
    return to_float(*p);
}
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_float<__half>(float v) {
    return __float2half_rn(v);
}
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// experts_route.cu
cudaError_t launch_exp_route(const ExpCall &c, cudaStream_t s);
// the rows of X (and dY) sorted by expert (16-bit types, 16-byte rows)
cudaError_t launch_exp_gather(const ExpCall &c, bool backward, cudaStream_t s);
// y_n = sum_i g_ni slots_ni (+ residual_n); dx_n = sum_i slots_ni
cudaError_t launch_exp_combine(const ExpCall &c, bool backward, cudaStream_t s);
// dresp from its partial sums (and <dy, b2>); column sums of da and g dy
cudaError_t launch_exp_dresp(const ExpCall &c, cudaStream_t s);
cudaError_t launch_exp_bias_grads(const ExpCall &c, cudaStream_t s);
// experts_simt.cu: the products on CUDA cores
cudaError_t launch_exp_simt(const ExpCall &c, bool backward, cudaStream_t s);
// experts_tc.cu: on the tensor cores (16-bit types, widths multiples of 8)
cudaError_t launch_exp_tc(const ExpCall &c, bool backward, cudaStream_t s);
int exp_tc_resp_parts(const ExpShape &s);

}  // namespace gmmb
