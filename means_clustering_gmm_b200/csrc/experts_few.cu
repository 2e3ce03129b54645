// The experts' products for few points (16-bit types, widths multiples of 8,
// at most kExpFewPoints points and GMM_EXPERT_FEW_PAIRS pairs): each used
// expert's weights are read once for every 32 of its points, and that read is
// the bound.
//
//   few_first_kernel   a block is 16 or 32 rows of one expert's first weight;
//                      the blocks of a pair whose expert an earlier pair
//                      names leave at once.  All points of the expert are the
//                      columns of one product.
//   few_second_kernel  a cluster is 16 rows of the output for all points; its
//                      warps share out the contraction indices of all used
//                      experts evenly, and their weighted sums are added up
//                      in a fixed order through shared and distributed shared
//                      memory, with b2 and the residual: no array of per-pair
//                      results and no third kernel.  It is launched under the
//                      first one's tail and prefetches its part of W2 there.
//
// Weights go from global memory straight into mma.sync fragments (a lane
// holds 8 consecutive elements of rows g and g + 8, 16 bytes each; the
// contraction index is permuted the same way in both operands): with 1 to 32
// columns the tensor cores wait for memory whatever form is used, and a
// register fragment needs neither shared memory nor barriers on the way.  A
// ring of TMA stages was built instead and was slower (one point, 8 gated
// experts of 2048-1024-2048: 33 us against 25): its stream alone, with the
// products taken out, ran at 5.4 TB/s where coalesced loads run at 6.3.
#include "experts.h"
#include "tc_ptx.cuh"

namespace gmmb {
namespace {

using namespace tc;

constexpr int kPairs = GMM_EXPERT_FEW_PAIRS;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 32;                     // points of one expert per pass
constexpr int kSegs = kPairs + kPairs / kCols;
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
// acc[nt] += 16 weight rows x 8 points over the contraction indices [k0, k1)
// (k0 a multiple of 32).  w0 / w1: rows g and g + 8; x[nt]: the row of point
// 8 nt + g.  All are rows that exist (a lane without one of its own repeats
// another's; its sums are not used), so whole chunks need no tests and cost
// three loads and two products each.
template <typename T, int NT, int U>
__device__ __forceinline__ void stream_rows(float (&acc)[4][4], const T *w0, const T *w1,
                                            const T *const (&x)[4], int k0, int k1) {
    const int t8 = (threadIdx.x & 3) * 8;
    auto products = [&](const uint4 &a0, const uint4 &a1, const uint4 (&b)[NT]) {
        const uint32_t lo[4] = {a0.x, a1.x, a0.y, a1.y};
        const uint32_t hi[4] = {a0.z, a1.z, a0.w, a1.w};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma16<T>(acc[n], lo, b[n].x, b[n].y);
            mma16<T>(acc[n], hi, b[n].z, b[n].w);
        }
    };
    int k = k0 + t8;
    const int end = k1 + t8;
    for (; k + 32 * U <= end; k += 32 * U) {
        uint4 a0[U], a1[U], b[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a0[u] = *reinterpret_cast<const uint4 *>(w0 + k + u * 32);
            a1[u] = *reinterpret_cast<const uint4 *>(w1 + k + u * 32);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                b[u][n] = *reinterpret_cast<const uint4 *>(x[n] + k + u * 32);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) products(a0[u], a1[u], b[u]);
    }
    for (; k < end; k += 32) {
        uint4 a0 = make_uint4(0u, 0u, 0u, 0u), a1 = a0, b[NT];
        const bool in = k < k1;
        if (in) {
            a0 = *reinterpret_cast<const uint4 *>(w0 + k);
            a1 = *reinterpret_cast<const uint4 *>(w1 + k);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            b[n] = make_uint4(0u, 0u, 0u, 0u);
            if (in) b[n] = *reinterpret_cast<const uint4 *>(x[n] + k);
        }
        products(a0, a1, b);
    }
}

// What the pairs name, in shared memory: the entries (pairs) sorted by expert
// and, per run of at most 32 entries of one expert, a segment.
struct Lists {
    int ids[kPairs];        // expert of each pair, or -1
    int start[kPairs];      // of a pair that names its expert first: its first entry
    float weight[kPairs];   // of an entry
    int2 seg[kSegs];        // expert, first entry | entries << 16
    int16_t pair[kPairs];   // of an entry
    int wsum[kWarps];
    int segs;
};

// (what every kernel may use without a limit of its own)
static_assert((kWarps + 1) * kExpFewPoints * 16 * sizeof(float) + sizeof(Lists) <= 48 * 1024,
              "sums of the points and the lists");

// One thread per pair.  A pair that repeats its point's expert has no entry of
// its own; its weight goes to the first one's.
__device__ __forceinline__ void make_lists(const ExpCall &c, Lists &L) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = (int)c.s.P, r = c.rt.r;
    int id = -1;
    float own = 0.f;
    if (tid < P) {
        id = c.s.dense ? 0 : c.rt.ids[tid];
        own = c.resp ? c.resp[tid] : 1.f;
        if (id >= c.s.K) {
            if (blockIdx.x == 0) set_error(c.err, GMM_ERR_RANGE);
            id = -1;
        }
        if (id < 0) id = -1;
    }
    if (P <= 32) {   // one warp, no barriers on the way
        if (warp == 0) {
            const unsigned same = __match_any_sync(0xffffffffu, id);
            // this pair's point's entries, before it and from it on
            const int p0 = lane / r * r;
            const unsigned point = ((1u << r) - 1) << p0;
            const bool repeat = (same & point & ((1u << lane) - 1)) != 0;
            float weight = own;
            for (int i = 1; i < r; ++i) {
                const float w = __shfl_down_sync(0xffffffffu, own, i);
                if (lane + i < p0 + r && lane + i < 32 && (same >> (lane + i) & 1)) weight += w;
            }
            const unsigned entries = __ballot_sync(0xffffffffu, id >= 0 && !repeat);
            const unsigned mine = same & entries;
            const int rank = __popc(mine & ((1u << lane) - 1)), count = __popc(mine);
            const bool entry = entries >> lane & 1, lead = entry && rank == 0;
            const unsigned leads = __ballot_sync(0xffffffffu, lead);
            int x = lead ? count : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            // (a lead's first entry, for the others of its expert)
            const int e0 = __shfl_sync(0xffffffffu, x - (lead ? count : 0),
                                       mine ? __ffs(mine) - 1 : lane);
            if (lead) L.seg[__popc(leads & ((1u << lane) - 1))] = make_int2(id, e0 | count << 16);
            if (entry) {
                L.pair[e0 + rank] = (int16_t)lane;
                L.weight[e0 + rank] = weight;
            }
            L.ids[lane] = id;
            if (lane == 0) L.segs = __popc(leads);
        }
        __syncthreads();
        return;
    }
    L.ids[tid] = id;
    L.weight[tid] = own;
    __syncthreads();
    float weight = 0.f;
    if (id >= 0) {
        const int p0 = tid / r * r;
        for (int q = p0; q < p0 + r; ++q) {
            const bool same = L.ids[q] == id;
            if (same && q < tid) id = -1;
            if (same && q >= tid) weight += L.weight[q];
        }
    }
    __syncthreads();
    L.ids[tid] = id;
    __syncthreads();
    int first = kPairs, rank = 0, count = 0;
    if (id >= 0) {
        const int4 *all = reinterpret_cast<const int4 *>(L.ids);
#pragma unroll 4
        for (int q = 0; q < (P + 3) / 4; ++q) {
            const int4 v = all[q];
            const int e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool same = e[i] == id;
                const int at = 4 * q + i;
                count += same;
                rank += same && at < tid;
                first = same && at < first ? at : first;
            }
        }
    }
    // entries and segments before this expert's: a scan over the pairs that
    // name an expert first
    const bool lead = id >= 0 && first == tid;
    const int segs = lead ? (count + kCols - 1) / kCols : 0;
    const int v = lead ? count | segs << 16 : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) L.wsum[warp] = x;
    __syncthreads();
    int before = x - v, total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += L.wsum[w];
        total += L.wsum[w];
    }
    if (lead) {
        const int e0 = before & 0xffff, s0 = before >> 16;
        L.start[tid] = e0;
        for (int i = 0; i < segs; ++i) {
            const int n = count - i * kCols < kCols ? count - i * kCols : kCols;
            L.seg[s0 + i] = make_int2(id, (e0 + i * kCols) | n << 16);
        }
    }
    if (tid == 0) L.segs = total >> 16;
    __syncthreads();
    if (id >= 0) {
        const int at = L.start[first] + rank;
        L.pair[at] = (int16_t)tid;
        L.weight[at] = weight;
    }
    __syncthreads();
}

// First weight.  grid (row tiles, pairs); R: 16-row groups of a block (gated:
// gate rows and up rows); the other warps split the contraction.
template <typename T, int ACT, bool GATED, int R>
__global__ void __launch_bounds__(kThreads, 4) few_first_kernel(ExpCall c) {
    constexpr int KS = kWarps / R;
    __shared__ float part[KS][R * 16][kCols + 1];
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
    // this lane's two weight rows, and this warp's slice of the contraction
    const int r0 = min(GATED ? n0 + g : n0 + grp * 16 + g, width - 1);
    const int r1 = min(GATED ? n0 + g + 8 : n0 + grp * 16 + g + 8, width - 1);
    const T *base = w + (GATED ? (size_t)grp * width * s.d : 0);
    const T *w0 = base + (size_t)r0 * s.d, *w1 = base + (size_t)r1 * s.d;
    const int chunks = (s.d + 31) / 32;
    const int k0 = chunks * ks / KS * 32, k1 = min(chunks * (ks + 1) / KS * 32, s.d);
    // (the biases of the row this thread finishes, on their way meanwhile)
    const int own = min(n0 + (int)threadIdx.x % rows, width - 1);
    const float bias = b ? load_elem(b + own) : 0.f;
    const float bias_up = GATED && b ? load_elem(b + width + own) : 0.f;
    for (int col0 = 0; col0 < total; col0 += kCols) {
        const int cols = min(total - col0, kCols);
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) (&acc[0][0])[i] = 0.f;
        auto point = [&](int at) {
            return x + c.rt.token(list[col0 + (at < cols ? at : 0)]) * s.d;
        };
        if (cols <= 8) {
            const T *const xp[4] = {point(g)};
            stream_rows<T, 1, 4>(acc, w0, w1, xp, k0, k1);
        } else {
            const T *const xp[4] = {point(g), point(g + 8), point(g + 16), point(g + 24)};
            stream_rows<T, 4, 1>(acc, w0, w1, xp, k0, k1);
        }
        if (col0) __syncthreads();   // the parts of the columns before are read
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n * 8 >= cols) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[ks][grp * 16 + g + (i >> 1) * 8][n * 8 + t * 2 + (i & 1)] = acc[n][i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
            const int row = i % rows, col = i / rows, out = n0 + row;
            if (out >= width) continue;
            float v = 0.f, u = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                v += part[k][row][col];
                if (GATED) u += part[k][16 + row][col];
            }
            float f = act_fast<ACT>(v + bias);   // (row is the same for every i)
            if (GATED) f *= u + bias_up;
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
template <typename T>
__global__ void __launch_bounds__(kThreads, 3) few_second_kernel(ExpCall c, int C) {
    extern __shared__ float sums[];
    __shared__ __align__(16) Lists L;
    const ExpShape &s = c.s;
    const int N = (int)s.N, r = c.rt.r, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % C, n0 = blockIdx.x / C * 16;
    float *mine = sums + warp * N * 16, *block = sums + kWarps * N * 16;
    for (int i = tid; i < kWarps * N * 16; i += kThreads) sums[i] = 0.f;
    // ids and weights do not depend on the first kernel
    make_lists(c, L);
    // this warp's part of the segments' 32-index chunks, laid end to end
    const int per = (s.h + 31) / 32, total = L.segs * per;
    const int w = rank * kWarps + warp, warps = C * kWarps;
    const int beg = (int)((int64_t)total * w / warps), end = (int)((int64_t)total * (w + 1) / warps);
    // its weights start for L2 while the first kernel ends
    for (int i = beg; i < end;) {
        const int sg = i / per, stop = min(end, (sg + 1) * per), row = lane & 15;
        const int k1 = min((stop - sg * per) * 32, s.h);
        const T *p = (const T *)c.w2 + ((size_t)L.seg[sg].x * s.o + min(n0 + row, s.o - 1)) * s.h;
        for (int k = (i - sg * per) * 32 + (lane >> 4) * 64; k < k1; k += 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + k));
        i = stop;
    }
    const int g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = beg; i < end;) {
        const int sg = i / per, stop = min(end, (sg + 1) * per);
        const int k0 = (i - sg * per) * 32, k1 = min((stop - sg * per) * 32, s.h);
        const int2 seg = L.seg[sg];
        const int e0 = seg.y & 0xffff, cnt = seg.y >> 16;
        const T *wr = (const T *)c.w2 + (size_t)seg.x * s.o * s.h;
        const T *w0 = wr + (size_t)min(n0 + g, s.o - 1) * s.h;
        const T *w1 = wr + (size_t)min(n0 + g + 8, s.o - 1) * s.h;
        const T *xp[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int at = n * 8 + g;
            xp[n] = (const T *)c.hid + (size_t)L.pair[e0 + (at < cnt ? at : 0)] * s.h;
        }
        float acc[4][4];
#pragma unroll
        for (int n = 0; n < 16; ++n) (&acc[0][0])[n] = 0.f;
        if (cnt <= 8) stream_rows<T, 1, 4>(acc, w0, w1, xp, k0, k1);
        else stream_rows<T, 4, 1>(acc, w0, w1, xp, k0, k1);
        // to the points' sums: no two lanes have a point and a row in common
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n * 8 >= cnt) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = n * 8 + t * 2 + (j & 1);
                if (at < cnt)
                    mine[(L.pair[e0 + at] / r) * 16 + g + (j >> 1) * 8] +=
                        L.weight[e0 + at] * acc[n][j];
            }
        }
        __syncwarp();
        i = stop;
    }
    __syncthreads();
    for (int i = tid; i < N * 16; i += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += sums[k * N * 16 + i];
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
            for (int q = tok * r; q < (tok + 1) * r; ++q) {
                const int id = s.dense ? 0 : c.rt.ids[q];
                if (id >= 0 && id < s.K)
                    v = fmaf(c.resp ? c.resp[q] : 1.f,
                             load_elem((const T *)c.b2 + (size_t)id * s.o + out), v);
            }
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
    // one wave at three blocks an SM
    int C = 8;
    while (C > 1 && tiles * C > 3 * 148) C /= 2;
    const size_t smem = (size_t)(kWarps + 1) * c.s.N * 16 * sizeof(float);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, few_second_kernel<T>, c, C);
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
    return launch_exp_combine(c, false, st);
}

}  // namespace

cudaError_t launch_exp_few(const ExpCall &c, cudaStream_t s) {
    return c.s.dt == GMM_BF16 ? few_t<__nv_bfloat16>(c, s) : few_t<__half>(c, s);
}

}  // namespace gmmb
