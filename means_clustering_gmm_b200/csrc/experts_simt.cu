// The experts' products on CUDA cores, for fp32 and GMM_FLAG_FORCE_SIMT.  Every product is a tile of 16 R x 64
// with an R x 4 micro tile per thread (forward calls of a few rows per expert: a
// dot product per warp), fp32 throughout; what one product hands to the next
// stays fp32 in the workspace.  Bound by the FMA pipes and what
// feeds them from shared memory: 35 TFLOP/s at 4096 x 512 x 512 (R = 8; 30 with
// R = 4, 23 with R = 2), 25 in a backward pass of 8192 pairs of 512-512-512.
#include <type_traits>

#include "experts.h"

namespace gmmb {

constexpr int kB = 64, kBK = 32, kSms = 148;

// Column m of contraction index k sits at m ^ 4 (k / 4 % 8): four indices of a
// row stored one by one meet 32 banks, and four columns stay together.
__device__ __forceinline__ int at_col(int k, int m) { return m ^ ((k >> 2 & 7) << 2); }

// A tile has 16 R rows, R per thread, and kB columns, four per thread.
template <int R> struct SimtSmem {
    float a[2][kBK][16 * R], b[2][kBK][kB];
};

// Operands.  KROW: row(m) is the array's row of tile row m (NULL outside),
// contiguous along the contraction; otherwise row(k) is the row of
// contraction index k, contiguous along the tile's rows, of which `cols` from
// column c0 exist.
template <typename E_> struct GatherRows {   // the segment's m-th point of [. x ld]
    using E = E_;
    static constexpr bool KROW = true;
    const E *p;
    ExpRoute rt;
    int64_t row0;
    int valid, ld;
    __device__ __forceinline__ const E *row(int m) const {
        return m < valid ? p + rt.token(rt.pair(row0 + m)) * ld : nullptr;
    }
};
template <typename E_> struct PlainRows {    // rows m0 + m of [rows x ld]
    using E = E_;
    static constexpr bool KROW = true;
    const E *p;
    int m0, rows, ld;
    __device__ __forceinline__ const E *row(int m) const {
        return m0 + m < rows ? p + (size_t)(m0 + m) * ld : nullptr;
    }
};
template <typename E_> struct PlainCols {    // columns of rows k of [. x ld]
    using E = E_;
    static constexpr bool KROW = false;
    const E *p;
    int c0, ld;
    __device__ __forceinline__ int cols() const { return ld - c0; }
    __device__ __forceinline__ const E *row(int64_t k) const { return p + k * ld + c0; }
};
template <typename E_> struct PointCols {    // columns of the segment's k-th point
    using E = E_;
    static constexpr bool KROW = false;
    const E *p;
    ExpRoute rt;
    int64_t row0;
    int c0, ld;
    __device__ __forceinline__ int cols() const { return ld - c0; }
    __device__ __forceinline__ const E *row(int64_t k) const {
        return p + rt.token(rt.pair(row0 + k)) * ld + c0;
    }
};

// A thread's W / 8 elements of a W x 32 operand tile, between global and
// shared memory.  VEC (fp32, rows of whole 16-byte units): in float4.
template <class OP, int W, bool VEC> struct Part {
    static constexpr int kN = W / (VEC ? 32 : 8);    // loads
    static constexpr int kCols = VEC ? W / 4 : W;    // threads along a row of the tile
    float r[W / 8];
    const typename OP::E *p[OP::KROW ? kN : 1];
    __device__ __forceinline__ void begin(const OP &op) {
        const int tid = threadIdx.x;
        if constexpr (OP::KROW)
#pragma unroll
            for (int i = 0; i < kN; ++i)
                p[i] = op.row(VEC ? (tid >> 3) + 32 * i : (tid >> 5) + 8 * i);
    }
    __device__ __forceinline__ void load(const OP &op, int64_t k0, int64_t K) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if constexpr (VEC) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if constexpr (OP::KROW) {
                    const int64_t k = k0 + (tid & 7) * 4;
                    if (p[i] && k < K) v = *reinterpret_cast<const float4 *>(p[i] + k);
                } else {
                    const int64_t k = k0 + tid / kCols + 256 / kCols * i;
                    const int n = tid % kCols * 4;
                    if (k < K && n < op.cols())
                        v = *reinterpret_cast<const float4 *>(op.row(k) + n);
                }
                r[4 * i] = v.x;
                r[4 * i + 1] = v.y;
                r[4 * i + 2] = v.z;
                r[4 * i + 3] = v.w;
            } else if constexpr (OP::KROW) {
                const int64_t k = k0 + (tid & 31);
                r[i] = p[i] && k < K ? load_elem(p[i] + k) : 0.f;
            } else {
                const int64_t k = k0 + tid / kCols + 256 / kCols * i;
                const int n = tid % kCols;
                r[i] = k < K && n < op.cols() ? load_elem(op.row(k) + n) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(float (&sh)[kBK][W]) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if constexpr (VEC && OP::KROW) {
                const int k = (tid & 7) * 4, m = (tid >> 3) + 32 * i;
#pragma unroll
                for (int j = 0; j < 4; ++j) sh[k + j][at_col(k, m)] = r[4 * i + j];
            } else if constexpr (VEC) {
                const int k = tid / kCols + 256 / kCols * i;
                *reinterpret_cast<float4 *>(&sh[k][at_col(k, tid % kCols * 4)]) =
                    make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            } else {
                const int k = OP::KROW ? tid & 31 : tid / kCols + 256 / kCols * i;
                const int m = OP::KROW ? (tid >> 5) + 8 * i : tid % kCols;
                sh[k][at_col(k, m)] = r[i];
            }
        }
    }
};

// A thread's R x 4 sums, two rows to a register pair: the packed fma leaves
// every other issue slot to the loads from shared memory.
template <int R> struct Acc {
    float2 v[R / 2][4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < R / 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = make_float2(0.f, 0.f);
    }
    __device__ __forceinline__ float at(int i, int j) const {
        return i & 1 ? v[i >> 1][j].y : v[i >> 1][j].x;
    }
};

// acc(i, j) += sum_k A(ty * R + i, k) B(tx * 4 + j, k).  The next 32 indices
// are on their way into registers while these are multiplied, and shared
// memory is double-buffered: one barrier a step.
template <bool VEC, int R, class A, class B>
__device__ __forceinline__ void simt_mma(SimtSmem<R> &sh, Acc<R> &acc, int64_t K, const A &opa,
                                         const B &opb) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    Part<A, 16 * R, VEC> pa;
    Part<B, kB, VEC> pb;
    pa.begin(opa);
    pb.begin(opb);
    pa.load(opa, 0, K);
    pb.load(opb, 0, K);
    __syncthreads();   // the product before has read both buffers
    int buf = 0;
    for (int64_t k0 = 0; k0 < K; k0 += kBK, buf ^= 1) {
        pa.store(sh.a[buf]);
        pb.store(sh.b[buf]);
        __syncthreads();
        if (k0 + kBK < K) {
            pa.load(opa, k0 + kBK, K);
            pb.load(opb, k0 + kBK, K);
        }
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            float2 a[R / 2];
            if constexpr (R == 2) {
                a[0] = *reinterpret_cast<const float2 *>(&sh.a[buf][k][at_col(k, ty * 2)]);
            } else {
#pragma unroll
                for (int i = 0; i < R; i += 4) {
                    const float4 v =
                        *reinterpret_cast<const float4 *>(&sh.a[buf][k][at_col(k, ty * R + i)]);
                    a[i / 2] = make_float2(v.x, v.y);
                    a[i / 2 + 1] = make_float2(v.z, v.w);
                }
            }
            const float4 bv = *reinterpret_cast<const float4 *>(&sh.b[buf][k][at_col(k, tx * 4)]);
            const float b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc.v[i][j] = __ffma2_rn(a[i], make_float2(b[j], b[j]), acc.v[i][j]);
        }
    }
}

// A block's 16 R rows: a part of a routing tile.
template <int R> struct SimtRows {
    int expert, valid;
    int64_t row0;
    bool null_expert;
    __device__ __forceinline__ bool load(const ExpRoute &rt) {
        constexpr int kParts = 8 / R;
        const int t = blockIdx.x / kParts, part = blockIdx.x % kParts;
        if (t >= rt.tiles()) return false;
        const auto x = rt.tile(t);
        expert = x.expert;
        null_expert = expert >= rt.K;
        row0 = x.row0 + part * (16 * R);
        valid = x.valid - part * (16 * R);
        if (valid > 16 * R) valid = 16 * R;
        return valid > 0;
    }
    // The pairs of this thread's rows: on their way while it multiplies, but
    // with eight rows only after that (8 registers more than 128 cost the
    // second block of an SM: 145 us against 119 for 8192 x 512 x 512).
    static constexpr bool kEarly = R < 8;
    __device__ __forceinline__ void own(const ExpRoute &rt, int (&pair)[R]) const {
        const int m = (threadIdx.x >> 4) * R;
#pragma unroll
        for (int i = 0; i < R; ++i) pair[i] = m + i < valid ? (int)rt.pair(row0 + m + i) : 0;
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
template <typename T, int ACT, bool GATED, bool V, int R>
__global__ void __launch_bounds__(256) simt_first_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem<R> sh;
    SimtRows<R> rows;
    exp_wait();
    if (!rows.load(c.rt)) return;
    const int d = c.s.d, width = c.s.mlp ? c.s.h : c.s.o, n0 = blockIdx.y * kB;
    const T *x = (const T *)c.x;
    if (rows.null_expert && c.s.mlp) return;
    int own[R] = {};
    if (rows.kEarly && !c.s.mlp) rows.own(c.rt, own);
    Acc<R> acc[2];
    acc[0].zero();
    acc[1].zero();
    if (!rows.null_expert) {
        const GatherRows<T> la{x, c.rt, rows.row0, rows.valid, d};
#pragma unroll
        for (int half = 0; half < (GATED ? 2 : 1); ++half) {
            const T *w = (const T *)c.w1 + ((size_t)rows.expert * c.s.first() +
                                            (size_t)half * width) * d;
            simt_mma<V>(sh, acc[half], d, la, PlainRows<T>{w, n0, width, d});
        }
    }
    if (!rows.kEarly && !c.s.mlp) rows.own(c.rt, own);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const T *b = c.b1 ? (const T *)c.b1 + (size_t)rows.expert * c.s.first() : nullptr;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int m = ty * R + i;
        if (m >= rows.valid) continue;
        const int64_t pair = own[i], tok = c.rt.token(pair);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + tx * 4 + j;
            if (col >= width) continue;
            float v = 0.f;
            if (!rows.null_expert) {
                v = act_of<ACT>(acc[0].at(i, j) + (b ? load_elem(b + col) : 0.f));
                if (GATED) v *= acc[1].at(i, j) + (b ? load_elem(b + width + col) : 0.f);
            }
            if (c.s.mlp)
                ((float *)c.hid)[(rows.row0 + m) * width + col] = v;
            else
                store_result<T>(c, pair, tok, col, v, rows.null_expert);
        }
    }
}

// Second product: W2 h + b2.
template <typename T, bool V, int R>
__global__ void __launch_bounds__(256) simt_second_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem<R> sh;
    SimtRows<R> rows;
    exp_wait();
    if (!rows.load(c.rt)) return;
    const int h = c.s.h, o = c.s.o, n0 = blockIdx.y * kB;
    const float *hid = (const float *)c.hid;
    int own[R];
    if (rows.kEarly) rows.own(c.rt, own);
    Acc<R> acc;
    acc.zero();
    if (!rows.null_expert) {
        const T *w = (const T *)c.w2 + (size_t)rows.expert * o * h;
        simt_mma<V>(sh, acc, h, PlainRows<float>{hid + rows.row0 * h, 0, rows.valid, h},
                    PlainRows<T>{w, n0, o, h});
    }
    if (!rows.kEarly) rows.own(c.rt, own);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int m = ty * R + i;
        if (m >= rows.valid) continue;
        const int64_t pair = own[i], tok = c.rt.token(pair);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + tx * 4 + j;
            if (col >= o) continue;
            float v = acc.at(i, j);
            if (c.b2 && !rows.null_expert)
                v += load_elem((const T *)c.b2 + (size_t)rows.expert * o + col);
            store_result<T>(c, pair, tok, col, v, rows.null_expert);
        }
    }
}

// ----------------------------------------------- few rows per expert, forward
// sums[i] = sum_k A(m0 + i, k) w[k] for kFewRows rows, by one warp along k, in
// every lane.  Rows past the segment are NULL and give 0.
constexpr int kFewRows = 4;
template <bool VEC, class A, typename T>
__device__ __forceinline__ void dots(float (&sums)[kFewRows], const A &opa, int m0, int K,
                                     const T *w) {
    const int lane = threadIdx.x & 31;
    const typename A::E *a[kFewRows];
#pragma unroll
    for (int i = 0; i < kFewRows; ++i) {
        a[i] = opa.row(m0 + i);
        sums[i] = 0.f;
    }
    if constexpr (VEC) {
#pragma unroll 4
        for (int k = lane * 4; k < K; k += 128) {
            const float4 b = *reinterpret_cast<const float4 *>(w + k);
#pragma unroll
            for (int i = 0; i < kFewRows; ++i)
                if (a[i]) {
                    const float4 v = *reinterpret_cast<const float4 *>(a[i] + k);
                    sums[i] = fmaf(v.x, b.x, sums[i]);
                    sums[i] = fmaf(v.y, b.y, sums[i]);
                    sums[i] = fmaf(v.z, b.z, sums[i]);
                    sums[i] = fmaf(v.w, b.w, sums[i]);
                }
        }
    } else {
#pragma unroll 4
        for (int k = lane; k < K; k += 32) {
            const float b = load_elem(w + k);
#pragma unroll
            for (int i = 0; i < kFewRows; ++i)
                if (a[i]) sums[i] = fmaf(load_elem(a[i] + k), b, sums[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kFewRows; ++i)
#pragma unroll
        for (int o = 16; o; o >>= 1) sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], o);
}

// One layer where the experts' segments hold few rows: a warp takes one output
// column of a tile and multiplies that row of the weight, read coalesced, with
// four points' rows at a time (from L1: the block's eight warps share them; the
// weight's row is read again for every four).  Bound by the weights' read for
// a row or two, then by L1.
template <typename T, int ACT, bool GATED, bool SECOND, bool V>
__global__ void __launch_bounds__(256) simt_few_kernel(ExpCall c) {
    exp_wait();
    SimtRows<8> rows;
    const int n = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int width = c.s.mlp && !SECOND ? c.s.h : c.s.o;
    if (!rows.load(c.rt) || n >= width) return;
    const bool last = SECOND || !c.s.mlp;
    if (rows.null_expert && !last) return;
    const int depth = SECOND ? c.s.h : c.s.d, first = SECOND ? c.s.o : c.s.first();
    const size_t at = (size_t)rows.expert * first + n;
    const T *w = (const T *)(SECOND ? c.w2 : c.w1) + at * depth;
    const T *b = (const T *)(SECOND ? c.b2 : c.b1);
    for (int m0 = 0; m0 < rows.valid; m0 += kFewRows) {
        float z[kFewRows] = {}, u[kFewRows] = {};
        if (!rows.null_expert) {
            if constexpr (SECOND) {
                const PlainRows<float> a{(const float *)c.hid + rows.row0 * depth, 0, rows.valid,
                                         depth};
                dots<V>(z, a, m0, depth, w);
            } else {
                const GatherRows<T> a{(const T *)c.x, c.rt, rows.row0, rows.valid, depth};
                dots<V>(z, a, m0, depth, w);
                if constexpr (GATED) dots<V>(u, a, m0, depth, w + (size_t)width * depth);
            }
        }
        // row m0 + i in lane i
        float v = z[0], up = u[0];
#pragma unroll
        for (int i = 1; i < kFewRows; ++i)
            if (lane == i) {
                v = z[i];
                up = u[i];
            }
        const int m = m0 + lane;
        if (lane >= kFewRows || m >= rows.valid) continue;
        if (!rows.null_expert) {
            if (b) v += load_elem(b + at);
            if constexpr (!SECOND) {
                v = act_of<ACT>(v);
                if constexpr (GATED) v *= up + (b ? load_elem(b + at + width) : 0.f);
            }
        }
        if (last) {
            const int64_t pair = c.rt.pair(rows.row0 + m);
            store_result<T>(c, pair, c.rt.token(pair), n, v, rows.null_expert);
        } else {
            ((float *)c.hid)[(rows.row0 + m) * width + n] = v;
        }
    }
}

// Backward, up to the first layer's pre-activations: recomputes them, forms
// the hidden gradient (mlp: q = W2^T dy; linear: dy itself), and writes
// da = d loss / d (W1 x + b1), resp * h for dW2, and this block's part of
// dresp = <q, h> (mlp) or <dy, f(z)> (linear).
template <typename T, int ACT, bool GATED, bool V, int R>
__global__ void __launch_bounds__(256) simt_da_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem<R> sh;
    SimtRows<R> rows;
    exp_wait();
    if (!rows.load(c.rt) || rows.null_expert) return;
    const int d = c.s.d, o = c.s.o, width = c.s.mlp ? c.s.h : c.s.o, n0 = blockIdx.y * kB;
    const T *x = (const T *)c.x, *dy = (const T *)c.dy;
    int own[R];
    rows.own(c.rt, own);
    Acc<R> acc[2], q;
    acc[0].zero();
    acc[1].zero();
    q.zero();
#pragma unroll
    for (int half = 0; half < (GATED ? 2 : 1); ++half) {
        const T *w = (const T *)c.w1 + ((size_t)rows.expert * c.s.first() +
                                        (size_t)half * width) * d;
        simt_mma<V>(sh, acc[half], d, GatherRows<T>{x, c.rt, rows.row0, rows.valid, d},
                    PlainRows<T>{w, n0, width, d});
    }
    if (c.s.mlp) {
        const T *w = (const T *)c.w2 + (size_t)rows.expert * o * width;
        simt_mma<V>(sh, q, o, GatherRows<T>{dy, c.rt, rows.row0, rows.valid, o},
                    PlainCols<T>{w, n0, width});
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const T *b = c.b1 ? (const T *)c.b1 + (size_t)rows.expert * c.s.first() : nullptr;
    float *da = (float *)c.da, *hs = (float *)c.hid;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int m = ty * R + i;
        const bool ok = m < rows.valid;
        const int64_t row = rows.row0 + m, pair = own[i], tok = c.rt.token(pair);
        const float g = ok && c.resp ? c.resp[pair] : 1.f;
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + tx * 4 + j;
            if (!ok || col >= width) continue;
            float f, df;
            act_both<ACT>(acc[0].at(i, j) + (b ? load_elem(b + col) : 0.f), f, df);
            const float up = GATED ? acc[1].at(i, j) + (b ? load_elem(b + width + col) : 0.f) : 1.f;
            const float qq = c.s.mlp ? q.at(i, j) : load_elem(dy + tok * o + col);
            part = fmaf(qq, f * up, part);
            da[row * c.s.first() + col] = g * qq * up * df;
            if (GATED) da[row * c.s.first() + width + col] = g * qq * f;
            if (c.s.mlp) hs[row * width + col] = g * f * up;
        }
        // the 16 lanes of a row
#pragma unroll
        for (int s = 8; s; s >>= 1) part += __shfl_xor_sync(0xffffffffu, part, s);
        if (tx == 0 && ok && c.dresp) c.rpart[pair * c.nrpart + blockIdx.y] = part;
    }
}

// dx (or its per-pair part) = da W1.
template <typename T, bool V, int R>
__global__ void __launch_bounds__(256) simt_dx_kernel(ExpCall c) {
    __shared__ __align__(16) SimtSmem<R> sh;
    SimtRows<R> rows;
    exp_wait();
    if (!rows.load(c.rt)) return;
    const int d = c.s.d, first = c.s.first(), n0 = blockIdx.y * kB;
    const float *da = (const float *)c.da;
    int own[R];
    if (rows.kEarly) rows.own(c.rt, own);
    Acc<R> acc;
    acc.zero();
    if (!rows.null_expert) {
        const T *w = (const T *)c.w1 + (size_t)rows.expert * first * d;
        simt_mma<V>(sh, acc, first, PlainRows<float>{da + rows.row0 * first, 0, rows.valid, first},
                    PlainCols<T>{w, n0, d});
    }
    if (!rows.kEarly) rows.own(c.rt, own);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int m = ty * R + i;
        if (m >= rows.valid) continue;
        const int64_t pair = own[i], tok = c.rt.token(pair);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + tx * 4 + j;
            if (col >= d) continue;
            if (c.s.direct())
                ((T *)c.dx)[tok * d + col] = from_float<T>(acc.at(i, j));
            else
                c.slots[pair * d + col] = acc.at(i, j);
        }
    }
}

// Weight gradient of one expert: out[m][n] = sum over its rows of
// A(row, m) B(row, n).  SECOND: A = dy (gathered), B = resp * h; otherwise
// A = da, B = x (gathered).
template <typename T, bool SECOND, bool V>
__global__ void __launch_bounds__(256) simt_dw_kernel(ExpCall c, int mtiles) {
    __shared__ __align__(16) SimtSmem<4> sh;
    constexpr int R = 4;
    const int e = blockIdx.x / mtiles, m0 = (blockIdx.x % mtiles) * (16 * R), n0 = blockIdx.y * kB;
    const int M = SECOND ? c.s.o : c.s.first(), N = SECOND ? c.s.h : c.s.d;
    exp_wait();
    const int64_t row0 = c.rt.ids ? c.rt.seg[e] : 0;
    const int64_t cnt = c.rt.ids ? c.rt.cnt[e] : c.rt.N;
    const float *own = (const float *)(SECOND ? c.hid : c.da);
    const T *points = (const T *)(SECOND ? c.dy : c.x);
    const int pw = SECOND ? c.s.o : c.s.d, ow = SECOND ? c.s.h : c.s.first();
    Acc<R> acc;
    acc.zero();
    const PointCols<T> pc{points, c.rt, row0, SECOND ? m0 : n0, pw};
    const PlainCols<float> oc{own + row0 * ow, SECOND ? n0 : m0, ow};
    if constexpr (SECOND) simt_mma<V>(sh, acc, cnt, pc, oc);
    else simt_mma<V>(sh, acc, cnt, oc, pc);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    T *out = (T *)(SECOND ? c.dw2 : c.dw1) + (size_t)e * M * N;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int m = m0 + ty * R + i;
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= N) continue;
            out[(size_t)m * N + n] = from_float<T>(acc.at(i, j));
        }
    }
}

static int64_t tiles_of(int64_t n, int w) { return (n + w - 1) / w; }

// Mean rows per expert up to which a forward call takes simt_few_kernel.  One
// dense 1024-4096 map: 1 point 4.9 us against 52 in tiles, 8 points 10 against
// 53; 16 points, r = 4 of 64 experts 512-1024-512 67 against 176; with 9 rows
// an expert (300 points, r = 2 of 64 experts 512-512-512) 137 against 125.  The
// mean says nothing of the lengths: with 8 rows an expert, 512-512-512, 64
// experts take 90 us against 122 in tiles when used evenly, 193 against 123
// when half of the points are one expert's, 167 against 87 when all are; 256
// experts 321 against 378, 458 against 423 and 331 against 122.
constexpr int64_t kFewMean = 8;

// Rows per thread of a product over the points' rows, with `cols` column
// tiles: the most that the experts' segments fill and that leaves every SM
// work.  8 against 4: 238 us against 266 for 8192 pairs of 8 experts 512-512-512;
// with 64 pairs an expert 256 against 228, with 144 blocks 57 against 52.  2
// against 4: 125 us against 142 with 9 pairs an expert, 266 against 228 with 64.
// What keeps two or three arrays of sums (da) lost with 8 (312 us against 286:
// one block an SM), and so did the weight gradients (235 against 185: the
// experts' lengths differ, and large tiles even them out less).
static int rows_per_thread(const ExpShape &p, int64_t cols) {
    const int64_t mean = p.P / p.K;
    if (mean <= 32) return 2;
    return mean >= 128 && tiles_of(p.P, 128) * cols >= 3 * kSms / 2 ? 8 : 4;
}

// fn(integral_constant<R>) for R = min(r, MAX); odd widths and the 16-bit
// types (which come here only where they are forced to) always take 4.
template <bool V, int MAX, class F> static cudaError_t with_rows(int r, F fn) {
    if constexpr (V) {
        if constexpr (MAX == 8)
            if (r == 8) return fn(std::integral_constant<int, 8>());
        if (r == 2) return fn(std::integral_constant<int, 2>());
    }
    return fn(std::integral_constant<int, 4>());
}

template <typename T, int ACT, bool GATED, bool V>
static cudaError_t simt_products(const ExpCall &c, bool backward, cudaStream_t s) {
    const ExpShape &p = c.s;
    const int width = p.mlp ? p.h : p.o;
    // a product over the points' rows, with n columns
    const auto rows = [&](auto most, int n, auto launch) {
        const unsigned cols = (unsigned)tiles_of(n, kB);
        return with_rows<V, most()>(rows_per_thread(p, cols), [&](auto r) {
            return launch(r, dim3(8u / r() * (unsigned)c.rt.max_tiles, cols));
        });
    };
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    cudaError_t e;
    if constexpr (sizeof(T) == 4)
        if (!backward && p.P <= kFewMean * (int64_t)p.K) {
            const auto grid = [&](int n) {
                return dim3((unsigned)c.rt.max_tiles, (unsigned)tiles_of(n, 8));
            };
            e = exp_launch(simt_few_kernel<T, ACT, GATED, false, V>, grid(width), 256, 0, s, c);
            if (e == cudaSuccess && p.mlp)
                e = exp_launch(simt_few_kernel<T, GMM_ACT_NONE, false, true, V>, grid(p.o), 256, 0,
                               s, c);
            return e;
        }
    if (!backward) {
        e = rows(eight, width, [&](auto r, dim3 g) {
            return exp_launch(simt_first_kernel<T, ACT, GATED, V, r()>, g, 256, 0, s, c);
        });
        if (e == cudaSuccess && p.mlp)
            e = rows(eight, p.o, [&](auto r, dim3 g) {
                return exp_launch(simt_second_kernel<T, V, r()>, g, 256, 0, s, c);
            });
        return e;
    }
    e = rows(four, width, [&](auto r, dim3 g) {
        return exp_launch(simt_da_kernel<T, ACT, GATED, V, r()>, g, 256, 0, s, c);
    });
    if (e == cudaSuccess)
        e = rows(eight, p.d, [&](auto r, dim3 g) {
            return exp_launch(simt_dx_kernel<T, V, r()>, g, 256, 0, s, c);
        });
    const unsigned m1 = (unsigned)tiles_of(p.first(), kB), m2 = (unsigned)tiles_of(p.o, kB);
    if (e == cudaSuccess)
        e = exp_launch(simt_dw_kernel<T, false, V>, dim3(m1 * p.K, (unsigned)tiles_of(p.d, kB)),
                       256, 0, s, c, (int)m1);
    if (e == cudaSuccess && p.mlp)
        e = exp_launch(simt_dw_kernel<T, true, V>, dim3(m2 * p.K, (unsigned)tiles_of(p.h, kB)),
                       256, 0, s, c, (int)m2);
    return e;
}

template <typename T, int ACT, bool GATED>
static cudaError_t simt_run(const ExpCall &c, bool backward, cudaStream_t s) {
    const ExpShape &p = c.s;
    // rows of whole 16-byte units in every array that is read along them
    if constexpr (sizeof(T) == 4)
        if (p.d % 4 == 0 && p.h % 4 == 0 && (p.o % 4 == 0 || !backward))
            return simt_products<T, ACT, GATED, true>(c, backward, s);
    return simt_products<T, ACT, GATED, false>(c, backward, s);
}

template <typename T, int ACT>
static cudaError_t simt_gate(const ExpCall &c, bool backward, cudaStream_t s) {
    return c.s.gated ? simt_run<T, ACT, true>(c, backward, s)
                     : simt_run<T, ACT, false>(c, backward, s);
}

template <typename T> static cudaError_t simt_act(const ExpCall &c, bool backward, cudaStream_t s) {
    switch (c.s.act) {
        case GMM_ACT_RELU: return simt_gate<T, GMM_ACT_RELU>(c, backward, s);
        case GMM_ACT_GELU: return simt_gate<T, GMM_ACT_GELU>(c, backward, s);
        case GMM_ACT_SILU: return simt_gate<T, GMM_ACT_SILU>(c, backward, s);
        default: return simt_gate<T, GMM_ACT_NONE>(c, backward, s);
    }
}

cudaError_t launch_exp_simt(const ExpCall &c, bool backward, cudaStream_t s) {
    switch (c.s.dt) {
        case GMM_F32: return simt_act<float>(c, backward, s);
        case GMM_BF16: return simt_act<__nv_bfloat16>(c, backward, s);
        default: return simt_act<__half>(c, backward, s);
    }
}

}  // namespace gmmb
