// The experts' products for few points (16-bit types, widths multiples of 8,
// at most GMM_EXPERT_FEW_PAIRS pairs): each used expert's weights are read
// once, and that read is the bound.
//
//   few_first_kernel   a block is 16 or 32 rows of one expert's first weight;
//                      the blocks of a pair whose expert an earlier pair
//                      names leave at once.  All points of the expert are the
//                      columns of one product.
//   few_second_kernel  a cluster is 16 rows of the output for all points;
//                      (expert, slice of h) units are dealt to its warps,
//                      whose weighted sums are added up in a fixed order
//                      through shared and distributed shared memory, with b2
//                      and the residual: no array of per-pair results and no
//                      third kernel.
//
// Weights go from global memory straight into mma.sync fragments (a lane
// holds 8 consecutive elements of rows g and g + 8, 16 bytes each; the
// contraction index is permuted the same way in both operands), because with
// 1 to 32 columns the tensor cores wait for memory whatever form is used, and
// a register fragment needs neither shared memory nor barriers on the way.
#include "experts.h"
#include "tc_ptx.cuh"

namespace gmmb {
namespace {

using namespace tc;

constexpr int kPairs = GMM_EXPERT_FEW_PAIRS;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
static_assert(kPairs == kThreads, "one thread looks at one pair");

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                     uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes of weights, read once: not kept in L1.
__device__ __forceinline__ uint4 stream16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// acc[nt] += 16 weight rows x 8 points, over the 32-wide chunks c0, c0 + step,
// .. of a contraction of K.  w0 / w1: rows g and g + 8 (NULL: zeros); x[nt]:
// the row of point 8 nt + g (NULL: zeros).
template <typename T, int NT, int U>
__device__ __forceinline__ void stream_rows(float (&acc)[NT][4], const T *w0, const T *w1,
                                            const T *const (&x)[NT], int K, int c0, int step,
                                            int chunks) {
    const int t8 = (threadIdx.x & 3) * 8;
    for (int c = c0; c < chunks; c += step * U) {
        uint4 a0[U], a1[U], b[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cc = c + u * step, k = cc * 32 + t8;
            const bool in = cc < chunks && k < K;
            a0[u] = a1[u] = make_uint4(0u, 0u, 0u, 0u);
            if (in && w0) a0[u] = stream16(w0 + k);
            if (in && w1) a1[u] = stream16(w1 + k);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                b[u][n] = make_uint4(0u, 0u, 0u, 0u);
                if (in && x[n]) b[u][n] = *reinterpret_cast<const uint4 *>(x[n] + k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t lo[4] = {a0[u].x, a1[u].x, a0[u].y, a1[u].y};
            const uint32_t hi[4] = {a0[u].z, a1[u].z, a0[u].w, a1[u].w};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16<T>(acc[n], lo, b[u][n].x, b[u][n].y);
                mma16<T>(acc[n], hi, b[u][n].z, b[u][n].w);
            }
        }
    }
}

// First weight.  grid (row tiles, pairs); R: 16-row groups of a block (gated:
// gate rows and up rows); the other warps split the contraction.
template <typename T, int ACT, bool GATED, int R>
__global__ void __launch_bounds__(kThreads, 2) few_first_kernel(ExpCall c) {
    constexpr int KS = kWarps / R, COLS = 32;
    __shared__ float part[KS][R * 16][COLS + 1];
    __shared__ int list[kPairs];    // pairs of this block's expert
    __shared__ int wcount[kWarps];
    const ExpShape &s = c.s;
    const int P = (int)s.P, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int width = s.mlp ? s.h : s.o;
    const int rows = GATED ? 16 : R * 16, n0 = blockIdx.x * rows;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int e = 0;
    int total = P;
    if (s.dense) {
        if ((int)threadIdx.x < P) list[threadIdx.x] = threadIdx.x;
        __syncthreads();
    } else {
        const int p = blockIdx.y;
        e = c.rt.ids[p];
        if (e >= s.K) {
            if (threadIdx.x == 0 && blockIdx.x == 0) set_error(c.err, GMM_ERR_RANGE);
            e = -1;
        }
        if (e < 0) {
            // a point without an expert: what the sum over none gives
            if (!s.mlp && s.direct())
                for (int i = threadIdx.x; i < rows && n0 + i < width; i += kThreads) {
                    const size_t at = (size_t)p * width + n0 + i;
                    ((T *)c.y)[at] = c.res ? ((const T *)c.res)[at] : from_float<T>(0.f);
                }
            return;
        }
        const bool mine = (int)threadIdx.x < P && c.rt.ids[threadIdx.x] == e;
        const unsigned votes = __ballot_sync(0xffffffffu, mine);
        if (lane == 0) wcount[warp] = __popc(votes);
        if (__syncthreads_or(mine && (int)threadIdx.x < p)) return;
        int at = __popc(votes & ((1u << lane) - 1));
        total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += wcount[w];
            total += wcount[w];
        }
        if (mine) list[at] = threadIdx.x;
        __syncthreads();
    }
    const T *x = (const T *)c.x, *w = (const T *)c.w1 + (size_t)e * s.first() * s.d;
    const T *b = c.b1 ? (const T *)c.b1 + (size_t)e * s.first() : nullptr;
    const int g = lane >> 2, t = lane & 3, grp = warp % R, ks = warp / R;
    // this lane's two weight rows
    const int r0 = GATED ? n0 + g : n0 + grp * 16 + g, r1 = r0 + 8;
    const T *base = w + (GATED ? (size_t)grp * width * s.d : 0);
    const T *w0 = r0 < width ? base + (size_t)r0 * s.d : nullptr;
    const T *w1 = r1 < width ? base + (size_t)r1 * s.d : nullptr;
    const int chunks = (s.d + 31) / 32;
    for (int col0 = 0; col0 < total; col0 += COLS) {
        float acc[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
        const T *xp[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int at = col0 + n * 8 + g;
            xp[n] = at < total ? x + c.rt.token(list[at]) * s.d : nullptr;
        }
        if (total - col0 <= 8) {
            float one[1][4] = {{0.f, 0.f, 0.f, 0.f}};
            const T *const x1[1] = {xp[0]};
            stream_rows<T, 1, 4>(one, w0, w1, x1, s.d, ks, KS, chunks);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][i] = one[0][i];
        } else {
            stream_rows<T, 4, 2>(acc, w0, w1, xp, s.d, ks, KS, chunks);
        }
        __syncthreads();   // the parts of the columns before are read
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[ks][grp * 16 + g + (i >> 1) * 8][n * 8 + t * 2 + (i & 1)] = acc[n][i];
        }
        __syncthreads();
        const int cols = total - col0 < COLS ? total - col0 : COLS;
        for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
            const int row = i % rows, col = i / rows, out = n0 + row;
            if (out >= width) continue;
            float v = 0.f, u = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                v += part[k][row][col];
                if (GATED) u += part[k][16 + row][col];
            }
            float f, df;
            act_fast<ACT>(v + (b ? value_at(b + out) : 0.f), f, df);
            if (GATED) f *= u + (b ? value_at(b + width + out) : 0.f);
            const int64_t p = list[col0 + col];
            if (s.mlp) {
                // rounded to the type: the second product's operand
                ((T *)c.hid)[p * width + out] = from_float<T>(f);
            } else if (s.direct()) {
                f *= c.resp ? c.resp[p] : 1.f;
                if (c.res) f += to_float(((const T *)c.res)[p * width + out]);
                ((T *)c.y)[p * width + out] = from_float<T>(f);
            } else {
                c.slots[p * width + out] = f;
            }
        }
    }
}

// Second weight.  grid (16-row tiles x C) in clusters of C blocks; dynamic
// shared memory: kWarps + 1 sums of [N x 16].
constexpr int kSecondCols = 32;
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) few_second_kernel(ExpCall c, int C) {
    extern __shared__ float sums[];
    __shared__ int expert[kPairs];               // the used experts, in the order of their first pair
    __shared__ __align__(16) int ids[kPairs];
    __shared__ float resp[kPairs];
    __shared__ int wcount[kWarps];
    __shared__ uint8_t lists[kWarps][kPairs];    // per warp: points of a unit
    const ExpShape &s = c.s;
    const int P = (int)s.P, N = (int)s.N, r = c.rt.r, warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = blockIdx.x % C, n0 = blockIdx.x / C * 16;
    const int tid = threadIdx.x;
    float *mine = sums + warp * N * 16, *block = sums + kWarps * N * 16;
    // ids and weights do not depend on the first kernel
    int id = -1;
    float weight = 0.f;
    if (tid < P) {
        id = s.dense ? 0 : c.rt.ids[tid];
        if (id >= s.K) id = -1;
        weight = c.resp ? c.resp[tid] : 1.f;
    }
    ids[tid] = id;
    resp[tid] = weight;
    for (int i = lane; i < N * 16; i += 32) mine[i] = 0.f;
    __syncthreads();
    bool lead = id >= 0;
    const int4 *all = reinterpret_cast<const int4 *>(ids);
#pragma unroll 8
    for (int q = 0; q <= (tid | 31) / 4; ++q) {   // the same trip count for a warp
        const int4 v = all[q];
        lead = lead && !((v.x == id && 4 * q < tid) || (v.y == id && 4 * q + 1 < tid) ||
                         (v.z == id && 4 * q + 2 < tid) || (v.w == id && 4 * q + 3 < tid));
    }
    const unsigned votes = __ballot_sync(0xffffffffu, lead);
    if (lane == 0) wcount[warp] = __popc(votes);
    __syncthreads();
    int at = __popc(votes & ((1u << lane) - 1)), E = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += wcount[w];
        E += wcount[w];
    }
    if (lead) expert[at] = id;
    __syncthreads();
    // slices of h per expert: as many as the cluster's warps can take at
    // once, of 128 indices at least
    const int warps = kWarps * C, chunks = (s.h + 31) / 32;
    int KS = E > 0 ? warps / E : 1;
    if (KS > (chunks + 3) / 4) KS = (chunks + 3) / 4;
    if (KS < 1) KS = 1;
    const int g = lane >> 2, t = lane & 3;
    const T *hid = (const T *)c.hid;
    uint8_t *list = lists[warp];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int unit = warp * C + rank; unit < E * KS; unit += warps) {
        const int i = unit / KS, ks = unit - i * KS, e = expert[i];
        // the expert's points; one that lists it twice once, with both weights
        int total = 0;
        for (int p0 = 0; p0 < P; p0 += 32) {
            const int p = p0 + lane;
            bool in = p < P && ids[p] == e;
            if (in)
                for (int q = p / r * r; q < p; ++q) in = in && ids[q] != e;
            const unsigned v = __ballot_sync(0xffffffffu, in);
            if (in) list[total + __popc(v & ((1u << lane) - 1))] = (uint8_t)p;
            total += __popc(v);
        }
        __syncwarp();
        const T *w = (const T *)c.w2 + (size_t)e * s.o * s.h;
        const T *w0 = n0 + g < s.o ? w + (size_t)(n0 + g) * s.h : nullptr;
        const T *w1 = n0 + g + 8 < s.o ? w + (size_t)(n0 + g + 8) * s.h : nullptr;
        for (int col0 = 0; col0 < total; col0 += kSecondCols) {
            float acc[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[n][k] = 0.f;
            const T *xp[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int l = col0 + n * 8 + g;
                xp[n] = l < total ? hid + (size_t)list[l] * s.h : nullptr;
            }
            if (total - col0 <= 8) {
                float one[1][4] = {{0.f, 0.f, 0.f, 0.f}};
                const T *const x1[1] = {xp[0]};
                stream_rows<T, 1, 4>(one, w0, w1, x1, s.h, ks, KS, chunks);
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[0][k] = one[0][k];
            } else {
                stream_rows<T, 4, 2>(acc, w0, w1, xp, s.h, ks, KS, chunks);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int l = col0 + n * 8 + t * 2 + (k & 1);
                    if (l >= total) continue;
                    const int p = list[l], tok = p / r;
                    float gw = 0.f;
                    for (int q = p; q < (tok + 1) * r; ++q)
                        if (ids[q] == e) gw += resp[q];
                    mine[tok * 16 + g + (k >> 1) * 8] += gw * acc[n][k];
                }
        }
        __syncwarp();
    }
    __syncthreads();
    for (int i = tid; i < N * 16; i += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sums[w * N * 16 + i];
        block[i] = v;
    }
    cluster_sync_all();
    for (int i = rank * kThreads + tid; i < N * 16; i += C * kThreads) {
        const int tok = i / 16, out = n0 + i % 16;
        if (out >= s.o) continue;
        float v = 0.f;
        for (int k = 0; k < C; ++k) {
            float x;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_u32(block + i, k)));
            v += x;
        }
        if (c.b2)
            for (int q = tok * r; q < (tok + 1) * r; ++q)
                if (ids[q] >= 0)
                    v = fmaf(resp[q], value_at((const T *)c.b2 + (size_t)ids[q] * s.o + out), v);
        const size_t y = (size_t)tok * s.o + out;
        if (c.res) v += to_float(((const T *)c.res)[y]);
        ((T *)c.y)[y] = from_float<T>(v);
    }
    cluster_sync_all();   // no block leaves while another reads its sums
}

template <typename T, int ACT, bool GATED, int R>
cudaError_t launch_first(const ExpCall &c, cudaStream_t st) {
    const int rows = GATED ? 16 : R * 16, width = c.s.mlp ? c.s.h : c.s.o;
    const dim3 grid((width + rows - 1) / rows, c.s.dense ? 1 : (unsigned)c.s.P);
    few_first_kernel<T, ACT, GATED, R><<<grid, kThreads, 0, st>>>(c);
    note_launches(1);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_second(const ExpCall &c, cudaStream_t st) {
    const int tiles = (c.s.o + 15) / 16;
    // about four blocks an SM
    int C = 8;
    while (C > 1 && tiles * C > 4 * 148) C /= 2;
    const size_t smem = (size_t)(kWarps + 1) * c.s.N * 16 * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(few_second_kernel<T>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // starts under the first kernel's tail; its wait is for all of it
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)C, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, few_second_kernel<T>, c, C);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, int ACT> cudaError_t first_act(const ExpCall &c, cudaStream_t st) {
    if (c.s.gated) return launch_first<T, ACT, true, 2>(c, st);
    // 16-row blocks until they fill the SMs
    const int width = c.s.mlp ? c.s.h : c.s.o;
    const int64_t experts = c.s.dense ? 1 : c.s.P < c.s.K ? c.s.P : c.s.K;
    return experts * ((width + 31) / 32) >= 4 * 148 ? launch_first<T, ACT, false, 2>(c, st)
                                                    : launch_first<T, ACT, false, 1>(c, st);
}

template <typename T> cudaError_t few_t(const ExpCall &c, cudaStream_t st) {
    cudaError_t e;
    switch (c.s.act) {
        case GMM_ACT_RELU: e = first_act<T, GMM_ACT_RELU>(c, st); break;
        case GMM_ACT_GELU: e = first_act<T, GMM_ACT_GELU>(c, st); break;
        case GMM_ACT_SILU: e = first_act<T, GMM_ACT_SILU>(c, st); break;
        default: e = first_act<T, GMM_ACT_NONE>(c, st);
    }
    if (e != cudaSuccess) return e;
    if (c.s.mlp) return launch_second<T>(c, st);
    return c.s.direct() ? cudaSuccess : launch_exp_combine(c, false, st);
}

}  // namespace

cudaError_t launch_exp_few(const ExpCall &c, cudaStream_t s) {
    return c.s.dt == GMM_BF16 ? few_t<__nv_bfloat16>(c, s) : few_t<__half>(c, s);
}

}  // namespace gmmb
