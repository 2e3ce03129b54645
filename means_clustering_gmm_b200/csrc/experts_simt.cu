// The experts' products on CUDA cores, for fp32 and for widths or pointers
// the tensor-core kernels do not take.  Every product is a 64 x 64 tile with
// a 4 x 4 micro tile per thread, fp32 throughout; what one product hands to
// the next stays fp32 in the workspace.
#include "experts.h"

namespace gmmb {

constexpr int kB = 64, kBK = 16;

struct SimtSmem {
    float a[kBK][kB + 4], b[kBK][kB + 4];
};

// acc[i][j] += sum_k A(ty * 4 + i, k) B(tx * 4 + j, k).  la / lb return one
// element (0 outside); AK / BK: whether k is the operand's contiguous axis
// (only the order of the loads depends on it).
template <bool AK, bool BK, class LA, class LB>
__device__ __forceinline__ void simt_mma(SimtSmem &sh, float (&acc)[4][4], int64_t K, LA la,
                                         LB lb) {
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    for (int64_t k0 = 0; k0 < K; k0 += kBK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kB * kBK / 256; ++i) {
            const int e = tid + i * 256;
            const int ka = AK ? e % kBK : e / kB, m = AK ? e / kBK : e % kB;
            sh.a[ka][m] = k0 + ka < K ? la(m, k0 + ka) : 0.f;
            const int kb = BK ? e % kBK : e / kB, n = BK ? e / kBK : e % kB;
            sh.b[kb][n] = k0 + kb < K ? lb(n, k0 + kb) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            const float4 av = *reinterpret_cast<const float4 *>(&sh.a[k][ty * 4]);
            const float4 bv = *reinterpret_cast<const float4 *>(&sh.b[k][tx * 4]);
            const float a[4] = {av.x, av.y, av.z, av.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
    }
}

// Operands: one element each, 0 outside.
template <typename E> struct GatherRows {   // row tok[m] of [. x ld], column k
    const E *p;
    const int64_t *tok;
    int valid, ld;
    __device__ __forceinline__ float operator()(int m, int64_t k) const {
        return m < valid ? value_at(p + tok[m] * ld + k) : 0.f;
    }
};
struct OwnRows {   // row m of the block's fp32 rows, column k
    const float *p;
    int valid, ld;
    __device__ __forceinline__ float operator()(int m, int64_t k) const {
        return m < valid ? p[(int64_t)m * ld + k] : 0.f;
    }
};
template <typename E> struct WeightRows {   // W[n0 + n][k]
    const E *p;
    int n0, rows, ld;
    __device__ __forceinline__ float operator()(int n, int64_t k) const {
        return n0 + n < rows ? value_at(p + (size_t)(n0 + n) * ld + k) : 0.f;
    }
};
template <typename E> struct WeightCols {   // W[k][n0 + n]
    const E *p;
    int n0, ld;
    __device__ __forceinline__ float operator()(int n, int64_t k) const {
        return n0 + n < ld ? value_at(p + (size_t)k * ld + n0 + n) : 0.f;
    }
};
template <typename E> struct PointCols {   // column c0 + m of the segment's k-th point
    const E *p;
    ExpRoute rt;
    int64_t row0;
    int c0, ld;
    __device__ __forceinline__ float operator()(int m, int64_t k) const {
        return c0 + m < ld ? value_at(p + rt.token(rt.pair(row0 + k)) * ld + c0 + m) : 0.f;
    }
};
struct OwnCols {   // column c0 + m of the segment's k-th fp32 row
    const float *p;
    int c0, ld;
    __device__ __forceinline__ float operator()(int m, int64_t k) const {
        return c0 + m < ld ? p[k * ld + c0 + m] : 0.f;
    }
};

__device__ __forceinline__ void zero(float (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
}

// A block's 64 rows: half of a routing tile, with each row's pair and point.
struct SimtRows {
    int expert, valid;
    int64_t row0;
    bool null_expert;
    __device__ __forceinline__ bool load(const ExpRoute &rt, int64_t *tok, int64_t *pair) {
        const int t = blockIdx.x >> 1, half = blockIdx.x & 1;
        if (t >= rt.tiles()) return false;
        const auto x = rt.tile(t);
        expert = x.expert;
        null_expert = expert >= rt.K;
        row0 = x.row0 + half * kB;
        valid = x.valid - half * kB;
        if (valid > kB) valid = kB;
        if (valid <= 0) return false;
        if (threadIdx.x < kB) {
            const int m = threadIdx.x < valid ? threadIdx.x : 0;
            const int64_t p = rt.pair(row0 + m);
            pair[threadIdx.x] = p;
            tok[threadIdx.x] = rt.token(p);
        }
        __syncthreads();
        return true;
    }
};

// The last product's epilogue: the point's result itself (direct), or the
// pair's row of slots.
template <typename T>
__device__ __forceinline__ void store_result(const ExpCall &c, int64_t pair, int64_t tok, int col,
                                             float v, bool null_expert) {
    if (c.s.direct()) {
        float r = null_expert ? 0.f : v * (c.resp ? c.resp[pair] : 1.f);
        if (c.res) r += to_float(((const T *)c.res)[tok * c.s.o + col]);
        ((T *)c.y)[tok * c.s.o + col] = from_float<T>(r);
    } else {
        c.slots[pair * c.s.o + col] = v;
    }
}

// First product: f(W1 x + b1) (gated: f(a) u) to the hidden rows, or, for
// the linear form, to the result.
template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(256) simt_first_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem sh;
    __shared__ int64_t tok[kB], pair[kB];
    SimtRows rows;
    if (!rows.load(c.rt, tok, pair)) return;
    const int d = c.s.d, width = c.s.mlp ? c.s.h : c.s.o, n0 = blockIdx.y * kB;
    const T *x = (const T *)c.x;
    if (rows.null_expert && c.s.mlp) return;
    float acc[2][4][4];
    zero(acc[0]);
    zero(acc[1]);
    if (!rows.null_expert) {
        const GatherRows<T> la{x, tok, rows.valid, d};
#pragma unroll
        for (int half = 0; half < (GATED ? 2 : 1); ++half) {
            const T *w = (const T *)c.w1 + ((size_t)rows.expert * c.s.first() +
                                            (size_t)half * width) * d;
            simt_mma<true, true>(sh, acc[half], d, la, WeightRows<T>{w, n0, width, d});
        }
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const T *b = c.b1 ? (const T *)c.b1 + (size_t)rows.expert * c.s.first() : nullptr;
    for (int i = 0; i < 4; ++i) {
        const int m = ty * 4 + i;
        if (m >= rows.valid) break;
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + tx * 4 + j;
            if (col >= width) break;
            float v = 0.f;
            if (!rows.null_expert) {
                v = act_of<ACT>(acc[0][i][j] + (b ? value_at(b + col) : 0.f));
                if (GATED) v *= acc[1][i][j] + (b ? value_at(b + width + col) : 0.f);
            }
            if (c.s.mlp)
                ((float *)c.hid)[(rows.row0 + m) * width + col] = v;
            else
                store_result<T>(c, pair[m], tok[m], col, v, rows.null_expert);
        }
    }
}

// Second product: W2 h + b2.
template <typename T>
__global__ void __launch_bounds__(256) simt_second_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem sh;
    __shared__ int64_t tok[kB], pair[kB];
    SimtRows rows;
    if (!rows.load(c.rt, tok, pair)) return;
    const int h = c.s.h, o = c.s.o, n0 = blockIdx.y * kB;
    const float *hid = (const float *)c.hid;
    float acc[4][4];
    zero(acc);
    if (!rows.null_expert) {
        const T *w = (const T *)c.w2 + (size_t)rows.expert * o * h;
        simt_mma<true, true>(sh, acc, h, OwnRows{hid + rows.row0 * h, rows.valid, h},
                             WeightRows<T>{w, n0, o, h});
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i) {
        const int m = ty * 4 + i;
        if (m >= rows.valid) break;
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + tx * 4 + j;
            if (col >= o) break;
            float v = acc[i][j];
            if (c.b2 && !rows.null_expert)
                v += value_at((const T *)c.b2 + (size_t)rows.expert * o + col);
            store_result<T>(c, pair[m], tok[m], col, v, rows.null_expert);
        }
    }
}

// Backward, up to the first layer's pre-activations: recomputes them, forms
// the hidden gradient (mlp: q = W2^T dy; linear: dy itself), and writes
// da = d loss / d (W1 x + b1), resp * h for dW2, and this block's part of
// dresp = <q, h> (mlp) or <dy, f(z)> (linear).
template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(256) simt_da_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem sh;
    __shared__ int64_t tok[kB], pair[kB];
    SimtRows rows;
    if (!rows.load(c.rt, tok, pair) || rows.null_expert) return;
    const int d = c.s.d, o = c.s.o, width = c.s.mlp ? c.s.h : c.s.o, n0 = blockIdx.y * kB;
    const T *x = (const T *)c.x, *dy = (const T *)c.dy;
    float acc[2][4][4], q[4][4];
    zero(acc[0]);
    zero(acc[1]);
    zero(q);
#pragma unroll
    for (int half = 0; half < (GATED ? 2 : 1); ++half) {
        const T *w = (const T *)c.w1 + ((size_t)rows.expert * c.s.first() +
                                        (size_t)half * width) * d;
        simt_mma<true, true>(sh, acc[half], d, GatherRows<T>{x, tok, rows.valid, d},
                             WeightRows<T>{w, n0, width, d});
    }
    if (c.s.mlp) {
        const T *w = (const T *)c.w2 + (size_t)rows.expert * o * width;
        simt_mma<true, false>(sh, q, o, GatherRows<T>{dy, tok, rows.valid, o},
                              WeightCols<T>{w, n0, width});
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const T *b = c.b1 ? (const T *)c.b1 + (size_t)rows.expert * c.s.first() : nullptr;
    float *da = (float *)c.da, *hs = (float *)c.hid;
    for (int i = 0; i < 4; ++i) {
        const int m = ty * 4 + i;
        const bool ok = m < rows.valid;
        const int64_t row = rows.row0 + m;
        float part = 0.f;
        for (int j = 0; j < 4 && ok; ++j) {
            const int col = n0 + tx * 4 + j;
            if (col >= width) break;
            const float g = c.resp ? c.resp[pair[m]] : 1.f;
            float f, df;
            act_both<ACT>(acc[0][i][j] + (b ? value_at(b + col) : 0.f), f, df);
            const float up = GATED ? acc[1][i][j] + (b ? value_at(b + width + col) : 0.f) : 1.f;
            const float qq = c.s.mlp ? q[i][j] : value_at(dy + tok[m] * o + col);
            part = fmaf(qq, f * up, part);
            da[row * c.s.first() + col] = g * qq * up * df;
            if (GATED) da[row * c.s.first() + width + col] = g * qq * f;
            if (c.s.mlp) hs[row * width + col] = g * f * up;
        }
        // the 16 lanes of a row
#pragma unroll
        for (int s = 8; s; s >>= 1) part += __shfl_xor_sync(0xffffffffu, part, s);
        if (tx == 0 && ok && c.dresp) c.rpart[row * c.nrpart + blockIdx.y] = part;
    }
}

// dx (or its per-pair part) = da W1.
template <typename T>
__global__ void __launch_bounds__(256) simt_dx_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem sh;
    __shared__ int64_t tok[kB], pair[kB];
    SimtRows rows;
    if (!rows.load(c.rt, tok, pair)) return;
    const int d = c.s.d, first = c.s.first(), n0 = blockIdx.y * kB;
    const float *da = (const float *)c.da;
    float acc[4][4];
    zero(acc);
    if (!rows.null_expert) {
        const T *w = (const T *)c.w1 + (size_t)rows.expert * first * d;
        simt_mma<true, false>(sh, acc, first, OwnRows{da + rows.row0 * first, rows.valid, first},
                              WeightCols<T>{w, n0, d});
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i) {
        const int m = ty * 4 + i;
        if (m >= rows.valid) break;
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + tx * 4 + j;
            if (col >= d) break;
            if (c.s.direct())
                ((T *)c.dx)[tok[m] * d + col] = from_float<T>(acc[i][j]);
            else
                c.slots[pair[m] * d + col] = acc[i][j];
        }
    }
}

// Weight gradient of one expert: out[m][n] = sum over its rows of
// A(row, m) B(row, n).  SECOND: A = dy (gathered), B = resp * h; otherwise
// A = da, B = x (gathered).
template <typename T, bool SECOND>
__global__ void __launch_bounds__(256) simt_dw_kernel(ExpCall c, int mtiles) {
    __shared__ __align__(16) SimtSmem sh;
    const int e = blockIdx.x / mtiles, m0 = (blockIdx.x % mtiles) * kB, n0 = blockIdx.y * kB;
    const int M = SECOND ? c.s.o : c.s.first(), N = SECOND ? c.s.h : c.s.d;
    const int64_t row0 = c.rt.ids ? c.rt.seg[e] : 0;
    const int64_t cnt = c.rt.ids ? c.rt.cnt[e] : c.rt.N;
    const float *own = (const float *)(SECOND ? c.hid : c.da);
    const T *points = (const T *)(SECOND ? c.dy : c.x);
    const int pw = SECOND ? c.s.o : c.s.d, ow = SECOND ? c.s.h : c.s.first();
    float acc[4][4];
    zero(acc);
    const PointCols<T> pc{points, c.rt, row0, SECOND ? m0 : n0, pw};
    const OwnCols oc{own + row0 * ow, SECOND ? n0 : m0, ow};
    if (SECOND) simt_mma<false, false>(sh, acc, cnt, pc, oc);
    else simt_mma<false, false>(sh, acc, cnt, oc, pc);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    T *out = (T *)(SECOND ? c.dw2 : c.dw1) + (size_t)e * M * N;
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i;
        if (m >= M) break;
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= N) break;
            out[(size_t)m * N + n] = from_float<T>(acc[i][j]);
        }
    }
}

static unsigned tiles_of(int64_t n) { return (unsigned)((n + kB - 1) / kB); }

template <typename T, int ACT, bool GATED>
static void simt_run(const ExpCall &c, bool backward, cudaStream_t s) {
    const ExpShape &p = c.s;
    const unsigned rows = 2u * (unsigned)c.rt.max_tiles;
    const int width = p.mlp ? p.h : p.o;
    if (!backward) {
        simt_first_kernel<T, ACT, GATED><<<dim3(rows, tiles_of(width)), 256, 0, s>>>(c);
        if (p.mlp) simt_second_kernel<T><<<dim3(rows, tiles_of(p.o)), 256, 0, s>>>(c);
        note_launches(p.mlp ? 2 : 1);
        return;
    }
    simt_da_kernel<T, ACT, GATED><<<dim3(rows, tiles_of(width)), 256, 0, s>>>(c);
    simt_dx_kernel<T><<<dim3(rows, tiles_of(p.d)), 256, 0, s>>>(c);
    const unsigned m1 = tiles_of(p.first());
    simt_dw_kernel<T, false><<<dim3(m1 * p.K, tiles_of(p.d)), 256, 0, s>>>(c, (int)m1);
    if (p.mlp) {
        const unsigned m2 = tiles_of(p.o);
        simt_dw_kernel<T, true><<<dim3(m2 * p.K, tiles_of(p.h)), 256, 0, s>>>(c, (int)m2);
    }
    note_launches(p.mlp ? 4 : 3);
}

template <typename T, int ACT>
static void simt_gate(const ExpCall &c, bool backward, cudaStream_t s) {
    if (c.s.gated) simt_run<T, ACT, true>(c, backward, s);
    else simt_run<T, ACT, false>(c, backward, s);
}

template <typename T> static void simt_act(const ExpCall &c, bool backward, cudaStream_t s) {
    switch (c.s.act) {
        case GMM_ACT_RELU: simt_gate<T, GMM_ACT_RELU>(c, backward, s); break;
        case GMM_ACT_GELU: simt_gate<T, GMM_ACT_GELU>(c, backward, s); break;
        case GMM_ACT_SILU: simt_gate<T, GMM_ACT_SILU>(c, backward, s); break;
        default: simt_gate<T, GMM_ACT_NONE>(c, backward, s);
    }
}

cudaError_t launch_exp_simt(const ExpCall &c, bool backward, cudaStream_t s) {
    switch (c.s.dt) {
        case GMM_F32: simt_act<float>(c, backward, s); break;
        case GMM_BF16: simt_act<__nv_bfloat16>(c, backward, s); break;
        default: simt_act<__half>(c, backward, s);
    }
    return cudaGetLastError();
}

}  // namespace gmmb
