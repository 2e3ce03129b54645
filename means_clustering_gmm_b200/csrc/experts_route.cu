// Routing of the experts' products and the sums around them.
//
// Routing is a stable counting sort of the (point, entry) pairs by expert,
// as the k-means update sorts points by cluster: histograms of chunks of 64 to
// 1024 pairs (one warp each), a scan over the chunks per expert, a scan over the
// experts with every segment rounded up to whole 128-row tiles, a stable
// scatter.  No floating-point atomics and no order that depends on
// scheduling, so every later sum over a segment is reproducible.
#include "experts.h"

namespace gmmb {

constexpr int kKeys = 2;   // pairs a lane loads at once

// Key of a pair: its expert, or K where it has none.
__device__ __forceinline__ int pair_key(const int32_t *ids, int64_t p, int K, int *err) {
    const int id = ids[p];
    if (id >= K) set_error(err, GMM_ERR_RANGE);
    return id < 0 || id >= K ? K : id;
}

__global__ void __launch_bounds__(128)
exp_hist_kernel(ExpRoute rt, int *err) {
    extern __shared__ int sh[];
    exp_enter();
    const int KK = rt.K + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *row = sh + warp * KK;
    const int64_t chunk = (int64_t)blockIdx.x * 4 + warp;
    const int64_t beg = chunk * rt.chunk, end = min(beg + rt.chunk, rt.P);
    if (beg >= rt.P) return;
    for (int e = lane; e < KK; e += 32) row[e] = 0;
    __syncwarp();
    for (int64_t p0 = beg; p0 < end; p0 += 32 * kKeys) {
        int key[kKeys];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int64_t p = p0 + u * 32 + lane;
            key[u] = p < end ? pair_key(rt.ids, p, rt.K, err) : -1;
        }
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const unsigned same = __match_any_sync(0xffffffffu, key[u]);
            if (key[u] >= 0 && lane == __ffs(same) - 1) row[key[u]] += __popc(same);
            __syncwarp();
        }
    }
    for (int e = lane; e < KK; e += 32) rt.hist[chunk * KK + e] = row[e];
}

// One block per key: exclusive scan of its counts over the chunks, in place.
__global__ void __launch_bounds__(1024)
exp_scan_kernel(ExpRoute rt, int64_t nch) {
    exp_enter();
    __shared__ int wsum[32];
    const int KK = rt.K + 1, e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    int total = 0;
    for (int64_t c0 = 0; c0 < nch; c0 += blockDim.x) {
        const int64_t c = c0 + threadIdx.x;
        const int v = c < nch ? rt.hist[c * KK + e] : 0;
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) x += wsum[w];
            all += wsum[w];
        }
        if (c < nch) rt.hist[c * KK + e] = total + x - v;
        total += all;
        __syncthreads();
    }
    // points without an expert make rows only where the last product writes
    // the result itself
    if (threadIdx.x == 0) rt.cnt[e] = e < rt.K || rt.r <= 1 ? total : 0;
}

// One block of 1024: segment starts (whole tiles) and the tables of 128-row
// and 256-row tiles, from the counts.  sh: [2 x (KK + 1)] ints.
__device__ __forceinline__ void make_tiles(const ExpRoute &rt, const int *cnt, int *sh) {
    __shared__ int wsum[2][32];
    const int KK = rt.K + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *first1 = sh, *first2 = sh + KK + 1;   // first tile of each segment
    const int per = (KK + 1023) / 1024;
    int mine1 = 0, mine2 = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e < KK) {
            mine1 += (cnt[e] + kExpTile - 1) / kExpTile;
            mine2 += (cnt[e] + 2 * kExpTile - 1) / (2 * kExpTile);
        }
    }
    int x1 = mine1, x2 = mine2;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y1 = __shfl_up_sync(0xffffffffu, x1, o);
        const int y2 = __shfl_up_sync(0xffffffffu, x2, o);
        if (lane >= o) {
            x1 += y1;
            x2 += y2;
        }
    }
    if (lane == 31) {
        wsum[0][warp] = x1;
        wsum[1][warp] = x2;
    }
    __syncthreads();
    if (warp < 2) {
        int w = wsum[warp][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        wsum[warp][lane] = w;
    }
    __syncthreads();
    int t1 = x1 - mine1 + (warp ? wsum[0][warp - 1] : 0);
    int t2 = x2 - mine2 + (warp ? wsum[1][warp - 1] : 0);
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e < KK) {
            first1[e] = t1;
            first2[e] = t2;
            rt.seg[e] = t1 * kExpTile;
            t1 += (cnt[e] + kExpTile - 1) / kExpTile;
            t2 += (cnt[e] + 2 * kExpTile - 1) / (2 * kExpTile);
        }
    }
    const int total1 = wsum[0][31], total2 = wsum[1][31];
    if (tid == 0) {
        rt.seg[KK] = total1 * kExpTile;
        rt.ntiles[0] = total1;
        rt.ntiles[1] = total2;
    }
    __syncthreads();
    for (int i = tid; i < total1 + total2; i += 1024) {
        const bool two = i >= total1;
        const int t = two ? i - total1 : i;
        const int *f = two ? first2 : first1;
        int lo = 0, hi = KK;   // last e with f[e] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (f[mid] <= t) lo = mid; else hi = mid;
        }
        const int rows = two ? 2 * kExpTile : kExpTile, before = (t - f[lo]) * rows;
        const int left = cnt[lo] - before;
        (two ? rt.pair_at : rt.tile_at)[t] =
            make_int4(lo, first1[lo] * kExpTile + before, left < rows ? left : rows, 0);
    }
}

__global__ void __launch_bounds__(1024)
exp_tiles_kernel(ExpRoute rt) {
    extern __shared__ int sh[];
    exp_enter();
    make_tiles(rt, rt.cnt, sh);
}

// The whole sort in one block, for up to kOneBlockPairs pairs: warp w takes
// the w-th run of pairs, twice (counts, then places).
constexpr int kOneBlockPairs = 4096;
constexpr int kOneBlockKeys = 1024;
__global__ void __launch_bounds__(1024)
exp_route_kernel(ExpRoute rt, int *err) {
    extern __shared__ int sh[];
    exp_enter();
    const int KK = rt.K + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *counts = sh;                    // [32][KK]
    int *cnt = sh + 32 * KK;             // [KK]
    int *tiles = cnt + KK;               // [2 x (KK + 1)]
    int *row = counts + warp * KK;
    const int P = (int)rt.P;
    const int run = ((P + 1023) / 1024) * 32;   // pairs of a warp
    const int beg = warp * run, end = min(beg + run, P);
    for (int i = tid; i < 32 * KK; i += 1024) counts[i] = 0;
    __syncthreads();
    for (int p0 = beg; p0 < end; p0 += 256) {
        int key[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int p = p0 + u * 32 + lane;
            key[u] = p < end ? pair_key(rt.ids, p, rt.K, err) : -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const unsigned same = __match_any_sync(0xffffffffu, key[u]);
            if (key[u] >= 0 && lane == __ffs(same) - 1) row[key[u]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = tid; e < KK; e += 1024) {
        int t = 0;
        for (int w = 0; w < 32; ++w) {
            const int v = counts[w * KK + e];
            counts[w * KK + e] = t;
            t += v;
        }
        // points without an expert make rows only where the last product
        // writes the result itself
        if (e == rt.K && rt.r > 1) t = 0;
        cnt[e] = t;
        rt.cnt[e] = t;
    }
    __syncthreads();
    make_tiles(rt, cnt, tiles);
    __syncthreads();
    for (int p0 = beg; p0 < end; p0 += 256) {
        int key[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int p = p0 + u * 32 + lane;
            key[u] = p < end ? pair_key(rt.ids, p, rt.K, nullptr) : -1;
            if (key[u] == rt.K && rt.r > 1) key[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const unsigned same = __match_any_sync(0xffffffffu, key[u]);
            const int rank = __popc(same & ((1u << lane) - 1));
            const int base = key[u] >= 0 ? row[key[u]] : 0;
            __syncwarp();
            if (key[u] >= 0) {
                rt.row_pair[tiles[key[u]] * kExpTile + base + rank] = p0 + u * 32 + lane;
                if (rank == 0) row[key[u]] = base + __popc(same);
            }
            __syncwarp();
        }
    }
}

__global__ void __launch_bounds__(128)
exp_scatter_kernel(ExpRoute rt) {
    extern __shared__ int sh[];
    exp_enter();
    const int KK = rt.K + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *row = sh + warp * KK;   // next row of each expert for this chunk
    const int64_t chunk = (int64_t)blockIdx.x * 4 + warp;
    const int64_t beg = chunk * rt.chunk, end = min(beg + rt.chunk, rt.P);
    if (beg >= rt.P) return;
    for (int e = lane; e < KK; e += 32) row[e] = rt.seg[e] + rt.hist[chunk * KK + e];
    __syncwarp();
    for (int64_t p0 = beg; p0 < end; p0 += 32 * kKeys) {
        int key[kKeys];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const int64_t p = p0 + u * 32 + lane;
            key[u] = p < end ? pair_key(rt.ids, p, rt.K, nullptr) : -1;
            if (key[u] == rt.K && rt.r > 1) key[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const unsigned same = __match_any_sync(0xffffffffu, key[u]);
            const int rank = __popc(same & ((1u << lane) - 1));
            const int base = key[u] >= 0 ? row[key[u]] : 0;
            __syncwarp();
            if (key[u] >= 0) {
                rt.row_pair[base + rank] = (int)(p0 + u * 32 + lane);
                if (rank == 0) row[key[u]] = base + __popc(same);
            }
            __syncwarp();
        }
    }
}

// A kernel's limit of dynamic shared memory belongs to the function, not to a
// launch: it is always set to what the largest call needs, so that calls of
// other sizes on other threads cannot lower it between this and their launch.
template <typename F> static cudaError_t allow_smem(F kernel, size_t bytes, size_t most) {
    return bytes <= 40 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kernel,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     (int)most);
}

cudaError_t launch_exp_route(const ExpCall &c, cudaStream_t s) {
    const ExpRoute &rt = c.rt;
    if (!rt.ids) return cudaSuccess;
    const int KK = rt.K + 1;
    cudaError_t e;
    if (rt.P <= kOneBlockPairs && KK <= kOneBlockKeys) {
        const auto size = [](int keys) { return (35 * keys + 2) * sizeof(int); };
        e = allow_smem(exp_route_kernel, size(KK), size(kOneBlockKeys));
        if (e != cudaSuccess) return e;
        return exp_launch(exp_route_kernel, dim3(1), 1024, size(KK), s, rt, c.err);
    }
    const int64_t nch = (rt.P + rt.chunk - 1) / rt.chunk;
    const unsigned blocks = (unsigned)((nch + 3) / 4);
    const size_t smem = 4 * KK * sizeof(int), most = 4 * (GMM_EXPERT_MAX_K + 1) * sizeof(int);
    e = allow_smem(exp_hist_kernel, smem, most);
    if (e == cudaSuccess) e = allow_smem(exp_scatter_kernel, smem, most);
    if (e != cudaSuccess) return e;
    e = exp_launch(exp_hist_kernel, dim3(blocks), 128, smem, s, rt, c.err);
    if (e == cudaSuccess)
        e = exp_launch(exp_scan_kernel, dim3(KK), nch > 256 ? 1024 : 256, 0, s, rt, nch);
    if (e == cudaSuccess)
        e = exp_launch(exp_tiles_kernel, dim3(1), 1024, 2 * (KK + 1) * sizeof(int), s, rt);
    if (e == cudaSuccess) e = exp_launch(exp_scatter_kernel, dim3(blocks), 128, smem, s, rt);
    return e;
}

// -------------------------------------------------------------- gather
// The rows of the segments' tiles: copies of their points' rows, zeros past a
// segment (the weight gradients contract over whole tiles).  A warp takes four
// rows at once, so that their loads are under way together; bound by HBM.
__global__ void __launch_bounds__(256)
exp_gather_kernel(ExpRoute rt, const uint4 *__restrict__ x, uint4 *__restrict__ xrows, int xu,
                  const uint4 *__restrict__ dy, uint4 *__restrict__ dyrows, int dyu) {
    exp_enter();
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)rt.tiles() * kExpTile;
    const uint4 *src = blockIdx.y ? dy : x;
    uint4 *dst = blockIdx.y ? dyrows : xrows;
    const int u = blockIdx.y ? dyu : xu;
    for (int64_t row = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4; row < rows;
         row += gridDim.x * 32) {
        const int4 p4 = *reinterpret_cast<const int4 *>(rt.row_pair + row);
        const int pairs[4] = {p4.x, p4.y, p4.z, p4.w};
        const auto t = rt.tile((int)(row / kExpTile));
        const int left = (int)(t.row0 + t.valid - row);   // rows of the segment from here
        const uint4 *p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = k < left ? src + rt.token(pairs[k]) * u : nullptr;
        for (int i = lane; i < u; i += 32) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = p[k] ? p[k][i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k) dst[(row + k) * u + i] = v[k];
        }
    }
}

cudaError_t launch_exp_gather(const ExpCall &c, bool backward, cudaStream_t s) {
    const int64_t want = (c.max_rows + 31) / 32;
    // (the linear form's gradients read dY through the pairs instead, or take
    // its rows as they are)
    const bool dy = backward && (c.s.mlp || c.plain_da());
    const dim3 grid((unsigned)(want < 148 * 8 ? want : 148 * 8), dy ? 2 : 1);
    return exp_launch(exp_gather_kernel, grid, 256, 0, s, c.rt, (const uint4 *)c.x,
                      (uint4 *)c.xrows, c.s.d / 8, (const uint4 *)c.dy, (uint4 *)c.dyrows,
                      c.s.o / 8);
}

// ------------------------------------------------------------- combine
// The sum of a point's entries: reads r rows of slots and writes one result;
// bound by HBM.  A thread takes V columns (8: float4 reads, one 16- or
// 32-byte write; 1: odd widths or a residual that is not 16-byte aligned).
template <typename T, bool BWD, int V>
__device__ __forceinline__ void combine_rows(const ExpRoute &rt, const float *slots,
                                             const float *resp, const T *res, T *out, int width,
                                             int blocks) {
    const int units = width / V;
    const int64_t total = rt.N * units;
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total;
         i += (int64_t)blocks * 256) {
        const int64_t n = i / units;
        const int col = (int)(i - n * units) * V;
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
        for (int e = 0; e < rt.r; ++e) {
            const int64_t p = n * rt.r + e;
            if (!rt.used(p)) continue;
            const float g = BWD || !resp ? 1.f : resp[p];
            const float *s = slots + p * width + col;
            float x[V];
            if constexpr (V == 8) {
                const float4 lo = __ldcs(reinterpret_cast<const float4 *>(s));
                const float4 hi = __ldcs(reinterpret_cast<const float4 *>(s) + 1);
                x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
                x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
            } else {
                x[0] = *s;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = BWD ? acc[v] + x[v] : fmaf(g, x[v], acc[v]);
        }
        __align__(16) T o[V];
        if (!BWD && res) {
            __align__(16) T b[V];
            if constexpr (V == 8) {
                const uint4 *w = reinterpret_cast<const uint4 *>(res + n * width + col);
                uint4 *d = reinterpret_cast<uint4 *>(b);
#pragma unroll
                for (int k = 0; k < (int)(V * sizeof(T) / 16); ++k) d[k] = w[k];
            } else {
                b[0] = res[n * width + col];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += to_float(b[v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = from_float<T>(acc[v]);
        if constexpr (V == 8) {
            uint4 *w = reinterpret_cast<uint4 *>(out + n * width + col);
            const uint4 *d = reinterpret_cast<const uint4 *>(o);
#pragma unroll
            for (int k = 0; k < (int)(V * sizeof(T) / 16); ++k) w[k] = d[k];
        } else {
            out[n * width + col] = o[0];
        }
    }
}


// One warp per pair: its partial sums in order, then <dy, b2>; 0 for an entry
// without an expert.
template <typename T>
__device__ __forceinline__ void dresp_rows(const ExpCall &c, int block, int blocks) {
    const int lane = threadIdx.x & 31, o = c.s.o;
    for (int64_t p = block * 8 + (threadIdx.x >> 5); p < c.rt.P; p += blocks * 8) {
        float acc = 0.f;
        if (c.rt.used(p)) {
            for (int i = lane; i < c.nrpart; i += 32) acc += c.rpart[p * c.nrpart + i];
            if (c.b2) {
                const T *g = (const T *)c.dy + c.rt.token(p) * o;
                const T *b = (const T *)c.b2 + (size_t)c.rt.ids[p] * o;
                for (int i = lane; i < o; i += 32) acc = fmaf(to_float(g[i]), to_float(b[i]), acc);
            }
#pragma unroll
            for (int m = 16; m; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
        }
        if (lane == 0) c.dresp[p] = acc;
    }
}

// Blocks below `blocks` sum entries, the others (backward) finish dresp.
template <typename T, bool BWD, int V>
__global__ void __launch_bounds__(256) exp_combine_kernel(ExpCall c, int width, int blocks) {
    exp_enter();
    if (BWD && (int)blockIdx.x >= blocks)
        dresp_rows<T>(c, blockIdx.x - blocks, gridDim.x - blocks);
    else
        combine_rows<T, BWD, V>(c.rt, c.slots, BWD ? nullptr : c.resp,
                                BWD ? nullptr : (const T *)c.res, (T *)(BWD ? c.dx : c.y), width,
                                blocks);
}

template <typename T, bool BWD, int V>
static cudaError_t combine_v(const ExpCall &c, cudaStream_t s) {
    const int width = BWD ? c.s.d : c.s.o;
    const int64_t want = c.s.direct() ? 0 : (c.s.N * (width / V) + 255) / 256;
    const int blocks = (int)(want < 148 * 16 ? want : 148 * 16);
    const int64_t rows = BWD && c.dresp ? (c.s.P + 7) / 8 : 0;
    const int more = (int)(rows < 148 * 8 ? rows : 148 * 8);
    return exp_launch(exp_combine_kernel<T, BWD, V>, dim3(blocks + more), 256, 0, s, c, width,
                      blocks);
}

template <typename T> static cudaError_t combine_t(const ExpCall &c, bool backward, cudaStream_t s) {
    if (backward) return c.s.d % 8 == 0 ? combine_v<T, true, 8>(c, s) : combine_v<T, true, 1>(c, s);
    return c.s.o % 8 == 0 && ((uintptr_t)c.res & 15) == 0 ? combine_v<T, false, 8>(c, s)
                                                          : combine_v<T, false, 1>(c, s);
}

cudaError_t launch_exp_combine(const ExpCall &c, bool backward, cudaStream_t s) {
    if (c.s.direct() && !(backward && c.dresp)) return cudaSuccess;
    switch (c.s.dt) {
        case GMM_F32: return combine_t<float>(c, backward, s);
        case GMM_BF16: return combine_t<__nv_bfloat16>(c, backward, s);
        default: return combine_t<__half>(c, backward, s);
    }
}

// ------------------------------------------------------ bias gradients
// Column sums over each expert's rows, for both biases in one launch: 32
// columns x 8 row lanes per block, the first w1 columns' blocks from da, the
// rest from dy's rows by index, weighted by resp.  The segment's rows are
// split into gridDim.z slices when the experts alone make too few blocks:
// fixed-order partial sums in c.colpart, added by exp_colsum_join_kernel.
// 8192 pairs of 8 experts, two biases of 512: 132 us unsplit, 18 split.
template <typename T>
__global__ void __launch_bounds__(256)
exp_colsum_kernel(ExpCall c, int w1, int w2) {
    exp_enter();
    __shared__ float sh[8][33];
    const ExpRoute &rt = c.rt;
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, S = gridDim.z, b1 = (w1 + 31) / 32;
    const bool second = (int)blockIdx.x >= b1;
    const int width = second ? w2 : w1;
    const int e = blockIdx.y, col = (blockIdx.x - (second ? b1 : 0)) * 32 + lane;
    const int64_t seg = rt.ids ? rt.seg[e] : 0, cnt = rt.ids ? rt.cnt[e] : rt.N;
    const int64_t per = (cnt + S - 1) / S;
    const int64_t beg = seg + blockIdx.z * per;
    const int64_t end = seg + (cnt < (blockIdx.z + 1) * per ? cnt : (blockIdx.z + 1) * per);
    float acc = 0.f;
    if (col < width && second) {
        const T *dy = (const T *)c.dy;
#pragma unroll 4
        for (int64_t row = beg + ty; row < end; row += 8) {
            const int64_t p = rt.pair(row);
            acc = fmaf(c.resp ? c.resp[p] : 1.f, load_elem(dy + rt.token(p) * width + col), acc);
        }
    } else if (col < width) {
        const float *da = (const float *)c.da;
#pragma unroll 4
        for (int64_t row = beg + ty; row < end; row += 8) acc += da[row * width + col];
    }
    sh[ty][lane] = acc;
    __syncthreads();
    if (ty == 0 && col < width) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sh[i][lane];
        float *part = c.colpart + (second ? (size_t)S * gridDim.y * w1 : 0);
        if (S == 1) ((T *)(second ? c.db2 : c.db1))[(size_t)e * width + col] = from_float<T>(t);
        else part[((size_t)blockIdx.z * gridDim.y + e) * width + col] = t;
    }
}

// The same over 16-bit rows of whole 16-byte units (copies in segment order):
// 64 columns x 32 row lanes per block.  One dense expert of 8192 x 4096 took
// 94 us unsplit, reading 64 MB; 14 split.
template <typename T>
__global__ void __launch_bounds__(256)
exp_colsum16_kernel(ExpCall c, int w1, int w2) {
    __shared__ float sh[32][65];
    const ExpRoute &rt = c.rt;
    const int cx = threadIdx.x & 7, ty = threadIdx.x >> 3, S = gridDim.z, b1 = (w1 + 63) / 64;
    const bool second = (int)blockIdx.x >= b1;
    const int width = second ? w2 : w1, c0 = (blockIdx.x - (second ? b1 : 0)) * 64;
    const int e = blockIdx.y, col = c0 + cx * 8;
    const T *rows = (const T *)(second ? c.dyrows : c.da);
    const float *resp = second ? c.resp : nullptr;
    T *out = (T *)(second ? c.db2 : c.db1);
    float *part = c.colpart + (second ? (size_t)S * gridDim.y * w1 : 0);
    exp_enter();
    const int64_t seg = rt.ids ? rt.seg[e] : 0, cnt = rt.ids ? rt.cnt[e] : rt.N;
    const int64_t per = (cnt + S - 1) / S;
    const int64_t beg = seg + blockIdx.z * per;
    const int64_t end = seg + (cnt < (blockIdx.z + 1) * per ? cnt : (blockIdx.z + 1) * per);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (col < width) {
#pragma unroll 4
        for (int64_t row = beg + ty; row < end; row += 32) {
            const uint4 w = *reinterpret_cast<const uint4 *>(rows + row * width + col);
            const float g = resp ? resp[rt.pair(row)] : 1.f;
            const T *v = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(g, to_float(v[i]), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sh[ty][cx * 8 + i] = acc[i];
    __syncthreads();
    const int cc = threadIdx.x & 63, q = threadIdx.x >> 6;   // quarter of the row lanes
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sh[q * 8 + i][cc];
    __syncthreads();
    sh[q][cc] = t;
    __syncthreads();
    const int oc = c0 + cc;
    if (q == 0 && oc < width) {
        const float v = sh[0][cc] + sh[1][cc] + sh[2][cc] + sh[3][cc];
        if (S == 1) out[(size_t)e * width + oc] = from_float<T>(v);
        else part[((size_t)blockIdx.z * gridDim.y + e) * width + oc] = v;
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
exp_colsum_join_kernel(ExpCall c, int S, int64_t n1, int64_t n2) {
    exp_enter();
    int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (i >= n1 + n2) return;
    const bool second = i >= n1;
    const float *part = c.colpart + (second ? S * n1 : 0);
    if (second) i -= n1;
    const int64_t n = second ? n2 : n1;
    float t = 0.f;
    for (int k = 0; k < S; ++k) t += part[k * n + i];
    ((T *)(second ? c.db2 : c.db1))[i] = from_float<T>(t);
}

// Slices of a segment: about four blocks an SM, at least 64 rows a slice.
int exp_colsum_slices(const ExpShape &s) {
    const int width = s.first() + (s.mlp ? s.o : 0);
    const int64_t blocks = (int64_t)s.K * ((width + 63) / 64);
    int64_t S = (4 * 148 + blocks - 1) / blocks;
    const int64_t most = s.P / s.K / 64;
    if (S > most) S = most;
    return (int)(S < 1 ? 1 : S > 32 ? 32 : S);
}

template <typename T> static cudaError_t bias_t(const ExpCall &c, cudaStream_t s) {
    const int w1 = c.db1 ? c.s.first() : 0, w2 = c.db2 ? c.s.o : 0, S = exp_colsum_slices(c.s);
    if (w1 + w2 == 0) return cudaSuccess;
    const auto grid = [&](int w) {
        return dim3((w1 + w - 1) / w + (w2 + w - 1) / w, c.s.K, S);
    };
    cudaError_t e;
    if (sizeof(T) == 2 && c.esize == 2) {
        if constexpr (sizeof(T) == 2)
            e = exp_launch(exp_colsum16_kernel<T>, grid(64), 256, 0, s, c, w1, w2);
    } else {
        e = exp_launch(exp_colsum_kernel<T>, grid(32), 256, 0, s, c, w1, w2);
    }
    const int64_t n1 = (int64_t)c.s.K * w1, n2 = (int64_t)c.s.K * w2;
    if (e == cudaSuccess && S > 1)
        e = exp_launch(exp_colsum_join_kernel<T>, dim3((unsigned)((n1 + n2 + 255) / 256)), 256, 0,
                       s, c, S, n1, n2);
    return e;
}

cudaError_t launch_exp_bias_grads(const ExpCall &c, cudaStream_t s) {
    switch (c.s.dt) {
        case GMM_F32: return bias_t<float>(c, s);
        case GMM_BF16: return bias_t<__nv_bfloat16>(c, s);
        default: return bias_t<__half>(c, s);
    }
}

}  // namespace gmmb
