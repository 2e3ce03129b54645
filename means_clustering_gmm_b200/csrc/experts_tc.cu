// The experts' products on the tensor cores (16-bit types, widths that are
// multiples of 8): one persistent kernel template, one CTA per SM, for every
// product of both directions.
//
//   warp 0       TMA producer.  Rows of X and dY come from copies sorted by
//                expert (the arrays themselves in the dense form).  Fetching
//                them in place by index (tile::gather4) was built first and
//                bounded every product that used it: a gather of four rows
//                takes an SM's TMA unit about 40 ns, 1.3 us for a stage whose
//                products take 0.27 us (8192 points, 2048-4096 gated: 1266 us
//                against 238 us a half-sized product from boxes), where the
//                copy costs two passes over the rows.  Rows, columns and
//                contraction indices past an edge arrive as zeros from the
//                tensor map.
//   warp 1       tcgen05.mma, M = 128, N up to 256, fp32 accumulators in
//                TMEM, two buffers of 256 columns: the epilogue of one tile
//                runs under the products of the next.
//   warps 2..9   epilogue, two warps per TMEM lane quadrant, each half of
//                the tile's columns; a thread owns one row.
//
// Operands are used as they lie in memory: a contraction over an array's
// contiguous axis reads it K-major, one over its rows (the weights in the
// backward pass, all operands of the weight gradients) MN-major, so nothing
// is transposed.
#include "experts.h"
#include "tc_ptx.cuh"

#include <cuda.h>

namespace gmmb {
namespace {

using namespace tc;

constexpr int kSms = 148;
constexpr int kThreads = 320;
constexpr int kRowsA = 128;          // rows of a tile (points, or weight rows of dW)
constexpr int kStepK = 64;           // contraction indices per stage
constexpr int kBytesA = kRowsA * kStepK * 2;
constexpr int kBlk = 64 * 128;       // one MN-major block: 64 columns x 64 rows

enum Kind {
    kFirst,    // f(W1 x + b1) -> hidden rows, or the linear form's result
    kSecond,   // W2 h + b2 -> result
    kDaLin,    // W x + b again; da from dY
    kDaMlp,    // W1 x + b1 again and W2^T dY; da, resp * h
    kDx,       // da W1 -> dx
    kDw1,      // da^T x
    kDw2       // dY^T (resp * h)
};

// Output columns per tile, MMA widths of the (up to two) phases, bytes of a
// stage's B part and the number of stages.  kDaMlp keeps the pre-activations
// and q = W2^T dY side by side in one accumulator buffer, so its tile is
// narrower: 64 columns gated (64 + 64 + 64), 128 otherwise (128 + 128).
template <int KIND, bool GATED> struct Cfg {
    static constexpr bool kGrad = KIND == kDw1 || KIND == kDw2;
    static constexpr int NB = KIND == kDaMlp ? (GATED ? 64 : 128)
                              : (KIND == kFirst && GATED) ? 128 : 256;
    static constexpr int N1 = KIND == kDaMlp ? 128 : 256;
    static constexpr int N2 = KIND == kDaMlp ? NB : 0;
    static constexpr int kBytesB = N1 * kStepK * 2;
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kStages = 192 * 1024 / kStage;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 256;
    static constexpr bool kAMn = kGrad;
    static constexpr bool kBMn = kGrad || KIND == kDx;
};

struct Args {
    ExpCall c;
    CUtensorMap a, b, a2, b2;   // phase 1 and phase 2 operands
    int ntn, ntm;               // column tiles; row tiles of one expert's dW
    int vec_bias, vec_res;      // biases / residual may be read 16 bytes at a time
};

struct Bars {
    uint64_t full[8], empty[8], accfull[2], accfree[2], done;
};

// One tile: which expert, which rows and columns, how many contraction steps.
struct Job {
    int expert, valid, col0, m0, steps1, steps2;
    int64_t row0, seg_end;
};

template <int KIND, bool GATED>
__device__ __forceinline__ int total_jobs(const Args &a) {
    return Cfg<KIND, GATED>::kGrad ? a.c.s.K * a.ntm * a.ntn : a.c.rt.tiles() * a.ntn;
}

template <int KIND, bool GATED>
__device__ __forceinline__ Job job_of(const Args &a, int idx) {
    using C = Cfg<KIND, GATED>;
    Job j;
    const ExpShape &s = a.c.s;
    const int t = idx / a.ntn;
    j.col0 = (idx - t * a.ntn) * C::NB;
    if constexpr (C::kGrad) {
        j.expert = t / a.ntm;
        j.m0 = (t - j.expert * a.ntm) * kRowsA;
        const int64_t cnt = a.c.rt.ids ? a.c.rt.cnt[j.expert] : a.c.rt.N;
        j.row0 = a.c.rt.ids ? a.c.rt.seg[j.expert] : 0;
        j.seg_end = j.row0 + cnt;
        j.valid = kRowsA;
        j.steps1 = (int)((cnt + kStepK - 1) / kStepK);
        j.steps2 = 0;
    } else {
        const auto x = a.c.rt.tile(t);
        j.expert = x.expert;
        j.valid = x.valid;
        j.row0 = x.row0;
        j.seg_end = x.seg_end;
        j.m0 = 0;
        const int k1 = KIND == kSecond ? s.h : KIND == kDx ? s.first() : s.d;
        const bool none = x.expert >= s.K;
        j.steps1 = none ? 0 : (k1 + kStepK - 1) / kStepK;
        j.steps2 = KIND == kDaMlp && !none ? (s.o + kStepK - 1) / kStepK : 0;
    }
    return j;
}

// Eight consecutive elements as floats.
template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float (&v)[8]) {
    if (vec) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_float(p[i]);
    }
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float x, float y);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                               pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

template <typename T, int KIND, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) exp_tc_kernel(const __grid_constant__ Args a) {
    using C = Cfg<KIND, GATED>;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    Bars *bars = reinterpret_cast<Bars *>(sm + (size_t)C::kStages * C::kStage);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert(sizeof(Bars) + 8 <= 256, "barrier block");

    const ExpCall &c = a.c;
    const ExpShape &s = c.s;
    const ExpRoute &rt = c.rt;
    (void)rt;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->accfull[i], 1);
            mbar_init(&bars->accfree[i], 8);
        }
        mbar_init(&bars->done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&a.a);
        prefetch_tensormap(&a.b);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = total_jobs<KIND, GATED>(a);

    if (warp == 0) {
        // ================================================ TMA producer
        uint32_t fill = 0;   // stages filled so far
        if (lane == 0) {
            bool ok = true;
            for (int idx = blockIdx.x; idx < total && ok; idx += gridDim.x) {
                const Job j = job_of<KIND, GATED>(a, idx);
                const int steps = j.steps1 + j.steps2, row = (int)j.row0;
                for (int st = 0; st < steps; ++st, ++fill) {
                    const int slot = fill % C::kStages;
                    ok = mbar_wait(&bars->empty[slot], ((fill / C::kStages) & 1) ^ 1, c.err,
                                   abort_flag);
                    if (!ok) break;
                    uint8_t *A = sm + (size_t)slot * C::kStage, *B = A + kBytesA;
                    uint64_t *bar = &bars->full[slot];
                    const bool second = KIND == kDaMlp && st >= j.steps1;
                    mbar_arrive_expect_tx(
                        bar, kBytesA + (second ? C::N2 * kStepK * 2 : C::N1 * kStepK * 2));
                    const int k = (second ? st - j.steps1 : st) * kStepK;
                    if constexpr (C::kGrad) {
#pragma unroll
                        for (int i = 0; i < kRowsA / 64; ++i)
                            tma_g2s_2d(A + i * kBlk, &a.a, j.m0 + i * 64, row + k, bar);
#pragma unroll
                        for (int i = 0; i < C::NB / 64; ++i)
                            tma_g2s_2d(B + i * kBlk, &a.b, j.col0 + i * 64, row + k, bar);
                    } else {
                        tma_g2s_2d(A, second ? &a.a2 : &a.a, k, row, bar);
                        if (KIND == kDx || second) {
                            constexpr int n = (KIND == kDx ? C::N1 : C::N2) / 64;
#pragma unroll
                            for (int i = 0; i < n; ++i)
                                tma_g2s_3d(B + i * kBlk, second ? &a.b2 : &a.b, j.col0 + i * 64, k,
                                           j.expert, bar);
                        } else if constexpr (GATED) {
                            // the tile's gate rows, then its up rows
                            tma_g2s_3d(B, &a.b, k, j.col0, j.expert, bar);
                            tma_g2s_3d(B + C::kBytesB / 2, &a.b, k, j.col0 + s.h, j.expert, bar);
                        } else {
                            tma_g2s_3d(B, &a.b, k, j.col0, j.expert, bar);
                        }
                    }
                }
            }
        }
        // no copy in flight at teardown
        for (uint32_t f = fill > (uint32_t)C::kStages ? fill - C::kStages : 0; f < fill; ++f)
            mbar_wait_drain(&bars->full[f % C::kStages], (f / C::kStages) & 1, c.err);
    } else if (warp == 1) {
        // ================================================ MMA issuer
        if (lane == 0) {
            constexpr bool kBf = sizeof(T) == 2 && !__is_same(T, __half);
            constexpr uint32_t id1 = kBf ? idesc_bf16(128, C::N1, C::kAMn, C::kBMn)
                                         : idesc_f16(128, C::N1, C::kAMn, C::kBMn);
            constexpr uint32_t id2 = kBf ? idesc_bf16(128, C::N2 ? C::N2 : 64, false, true)
                                         : idesc_f16(128, C::N2 ? C::N2 : 64, false, true);
            const uint64_t dA = smem_desc(smem_u32(sm), C::kAMn ? kBlk : 16, 1024, kSwz128);
            const uint64_t dB1 = smem_desc(smem_u32(sm + kBytesA), C::kBMn ? kBlk : 16, 1024,
                                           kSwz128);
            const uint64_t dB2 = smem_desc(smem_u32(sm + kBytesA), kBlk, 1024, kSwz128);
            uint32_t use = 0, tile = 0;
            bool ok = true;
            int idx = blockIdx.x;
            Job nxt = idx < total ? job_of<KIND, GATED>(a, idx) : Job{};
            for (; idx < total && ok; idx += gridDim.x, ++tile) {
                const Job j = nxt;
                if (idx + (int)gridDim.x < total) nxt = job_of<KIND, GATED>(a, idx + gridDim.x);
                const int buf = tile & 1;
                if (!mbar_wait(&bars->accfree[buf], ((tile >> 1) & 1) ^ 1, c.err, abort_flag)) break;
                tc_fence_after();
                const uint32_t acc = tmem + buf * 256;
                const int steps = j.steps1 + j.steps2;
                for (int st = 0; st < steps; ++st, ++use) {
                    const int slot = use % C::kStages;
                    if (!mbar_wait(&bars->full[slot], (use / C::kStages) & 1, c.err, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t off = (uint32_t)(slot * C::kStage) >> 4;
                    const bool second = KIND == kDaMlp && st >= j.steps1;
                    const bool fresh = st == 0 || (KIND == kDaMlp && st == j.steps1);
#pragma unroll
                    for (int kk = 0; kk < kStepK / 16; ++kk) {
                        const uint64_t da = dA + off + (uint32_t)(kk * (C::kAMn ? 2048 : 32) >> 4);
                        if (second)
                            mma_f16(acc + C::N1, da, dB2 + off + (uint32_t)(kk * 2048 >> 4), id2,
                                    fresh && kk == 0 ? 0u : 1u);
                        else
                            mma_f16(acc, da,
                                    dB1 + off + (uint32_t)(kk * (C::kBMn ? 2048 : 32) >> 4), id1,
                                    fresh && kk == 0 ? 0u : 1u);
                    }
                    mma_commit(&bars->empty[slot]);
                }
                if (ok) mma_commit(&bars->accfull[buf]);
            }
            mma_commit(&bars->done);
            mbar_wait_drain(&bars->done, 0, c.err);   // no MMA in flight at teardown
        }
    } else {
        // ================================================ epilogue
        const int q = warp & 3, hf = (warp - 2) >> 2, m = q * 32 + lane;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        uint32_t tile = 0;
        for (int idx = blockIdx.x; idx < total; idx += gridDim.x, ++tile) {
            const Job j = job_of<KIND, GATED>(a, idx);
            const int buf = tile & 1;
            const bool none = !C::kGrad && j.expert >= s.K;
            const bool valid = m < j.valid;
            const int64_t row = j.row0 + m;
            int64_t pair = 0, tok = 0;
            float g = 1.f;
            if (!C::kGrad && valid) {
                pair = rt.pair(row);
                tok = rt.token(pair);
                if (c.resp) g = c.resp[pair];
            }
            __syncwarp();
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->accfull[buf], (tile >> 1) & 1, c.err,
                                                   abort_flag)))
                break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * 256 + lane_base;
            const bool has = j.steps1 > 0;   // otherwise the accumulators were not written
            float part = 0.f;
            constexpr int kHalf = C::NB / 2;
#pragma unroll 1
            for (int c0 = hf * kHalf; c0 < (hf + 1) * kHalf; c0 += 32) {
                uint32_t r0[32], r1[32], r2[32];
                __syncwarp();   // the loads below are warp-wide
                tmem_ld32(acc + c0, r0);
                if constexpr (KIND == kFirst && GATED) tmem_ld32(acc + 128 + c0, r1);
                if constexpr (KIND == kDaMlp && GATED) tmem_ld32(acc + 64 + c0, r1);
                if constexpr (KIND == kDaMlp) tmem_ld32(acc + C::N1 + c0, r2);
                tmem_ld_wait();
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int col = j.col0 + c0 + v * 8;
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = has ? __uint_as_float(r0[v * 8 + i]) : 0.f;
                    if constexpr (C::kGrad) {
                        const int M = KIND == kDw2 ? s.o : s.first();
                        const int N = KIND == kDw2 ? s.h : s.d;
                        T *out = (T *)(KIND == kDw2 ? c.dw2 : c.dw1);
                        if (j.m0 + m < M && col < N)
                            store8(out + ((size_t)j.expert * M + j.m0 + m) * N + col, x);
                    } else if constexpr (KIND == kDx) {
                        if (valid && col < s.d) {
                            if (s.direct()) {
                                store8((T *)c.dx + tok * s.d + col, x);
                            } else {
                                float4 *o = reinterpret_cast<float4 *>(c.slots + pair * s.d + col);
                                o[0] = make_float4(x[0], x[1], x[2], x[3]);
                                o[1] = make_float4(x[4], x[5], x[6], x[7]);
                            }
                        }
                    } else if constexpr (KIND == kDaLin || KIND == kDaMlp) {
                        const int width = s.mlp ? s.h : s.o;
                        if (none || col >= width) continue;
                        T *da = (T *)c.da + row * s.first() + col;
                        T *hs = (T *)c.hid + row * s.h + col;
                        float d1[8], d2[8], h8[8];
                        if (valid) {
                            float b8[8] = {}, u8[8] = {}, q8[8];
                            const T *b = (const T *)c.b1 + (size_t)j.expert * s.first() + col;
                            if (c.b1) {
                                load8(b, a.vec_bias, b8);
                                if (GATED) load8(b + width, a.vec_bias, u8);
                            }
                            if constexpr (KIND == kDaLin)
                                load8((const T *)c.dy + tok * s.o + col, true, q8);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float f, df;
                                act_both<ACT>(x[i] + b8[i], f, df);
                                float up = 1.f, qq;
                                if constexpr (KIND == kDaMlp) qq = __uint_as_float(r2[v * 8 + i]);
                                else qq = q8[i];
                                if constexpr (GATED) up = __uint_as_float(r1[v * 8 + i]) + u8[i];
                                const float gq = g * qq, fu = f * up;
                                part = fmaf(qq, fu, part);
                                d1[i] = gq * up * df;
                                d2[i] = gq * f;
                                h8[i] = g * fu;
                            }
                        } else {
                            // rows past the segment are zeros: the weight
                            // gradients contract over them
#pragma unroll
                            for (int i = 0; i < 8; ++i) d1[i] = d2[i] = h8[i] = 0.f;
                        }
                        store8(da, d1);
                        if constexpr (KIND == kDaMlp) {
                            if constexpr (GATED) store8(da + width, d2);
                            store8(hs, h8);
                        }
                    } else {
                        const int width = KIND == kSecond ? s.o : s.mlp ? s.h : s.o;
                        if (!valid || col >= width) continue;
                        if (KIND == kFirst && s.mlp && none) continue;
                        const T *b = (const T *)(KIND == kSecond ? c.b2 : c.b1);
                        if (b && !none) {
                            b += (size_t)j.expert * (KIND == kSecond ? s.o : s.first()) + col;
                            float b8[8];
                            load8(b, a.vec_bias, b8);
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] += b8[i];
                        }
                        if constexpr (KIND == kFirst) {
                            if (!none) {
                                if constexpr (GATED) {
                                    float u8[8] = {};
                                    if (b) load8(b + width, a.vec_bias, u8);
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        x[i] = act_of<ACT>(x[i]) *
                                               (__uint_as_float(r1[v * 8 + i]) + u8[i]);
                                } else {
#pragma unroll
                                    for (int i = 0; i < 8; ++i) x[i] = act_of<ACT>(x[i]);
                                }
                            }
                            if (s.mlp) {
                                // rounded to the type: the second product's operand
                                store8((T *)c.hid + row * width + col, x);
                                continue;
                            }
                        }
                        if (s.direct()) {
                            float r8[8] = {};
                            if (c.res) load8((const T *)c.res + tok * width + col, a.vec_res, r8);
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = none ? r8[i] : fmaf(g, x[i], r8[i]);
                            store8((T *)c.y + tok * width + col, x);
                        } else {
                            float4 *o = reinterpret_cast<float4 *>(c.slots + pair * width + col);
                            o[0] = make_float4(x[0], x[1], x[2], x[3]);
                            o[1] = make_float4(x[4], x[5], x[6], x[7]);
                        }
                    }
                }
            }
            if constexpr (KIND == kDaLin || KIND == kDaMlp) {
                if (valid && !none && c.dresp)
                    c.rpart[row * c.nrpart + (j.col0 / C::NB) * 2 + hf] = part;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->accfree[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------- host side
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeFn)p;
    }();
    return fn;
}

struct Maps {
    gmm_dtype dt;
    bool ok = true;
    // [planes x] rows x cols, boxes of 64 columns x box_rows
    void make(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t planes,
              int box_rows) {
        const EncodeFn fn = encode_fn();
        if (!fn) {
            ok = false;
            return;
        }
        const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
        const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * rows * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
        const cuuint32_t one[3] = {1, 1, 1};
        ok = ok && fn(m, dt == GMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      planes ? 3 : 2, const_cast<void *>(base), dims, strides, box, one,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
};

template <typename T, int KIND, int ACT, bool GATED>
cudaError_t launch_kind(const ExpCall &c, cudaStream_t st) {
    using C = Cfg<KIND, GATED>;
    const ExpShape &s = c.s;
    Args a;
    a.c = c;
    Maps maps{s.dt};
    int width = 0, mrows = 0;
    switch (KIND) {
        case kFirst:
        case kDaLin:
        case kDaMlp:
            width = s.mlp ? s.h : s.o;
            maps.make(&a.a, c.xrows, s.d, c.point_rows, 0, kRowsA);
            maps.make(&a.b, c.w1, s.d, s.first(), s.K, GATED ? C::N1 / 2 : C::N1);
            if (KIND == kDaMlp) {
                maps.make(&a.a2, c.dyrows, s.o, c.point_rows, 0, kRowsA);
                maps.make(&a.b2, c.w2, s.h, s.o, s.K, kStepK);
            }
            break;
        case kSecond:
            width = s.o;
            maps.make(&a.a, c.hid, s.h, c.max_rows, 0, kRowsA);
            maps.make(&a.b, c.w2, s.h, s.o, s.K, C::N1);
            break;
        case kDx:
            width = s.d;
            maps.make(&a.a, c.da, s.first(), c.max_rows, 0, kRowsA);
            maps.make(&a.b, c.w1, s.d, s.first(), s.K, kStepK);
            break;
        case kDw1:
            width = s.d;
            mrows = s.first();
            maps.make(&a.a, c.da, s.first(), c.max_rows, 0, kStepK);
            maps.make(&a.b, c.xrows, s.d, c.point_rows, 0, kStepK);
            break;
        case kDw2:
            width = s.h;
            mrows = s.o;
            maps.make(&a.a, c.dyrows, s.o, c.point_rows, 0, kStepK);
            maps.make(&a.b, c.hid, s.h, c.max_rows, 0, kStepK);
            break;
    }
    if (!maps.ok) return cudaErrorNotSupported;
    a.ntn = (width + C::NB - 1) / C::NB;
    a.ntm = (mrows + kRowsA - 1) / kRowsA;
    const void *bias = KIND == kSecond ? c.b2 : c.b1;
    a.vec_bias = ((uintptr_t)bias & 15) == 0;
    a.vec_res = ((uintptr_t)c.res & 15) == 0;
    const int64_t most = C::kGrad ? (int64_t)s.K * a.ntm * a.ntn : (int64_t)c.rt.max_tiles * a.ntn;
    if (most > 0x7fff0000) return cudaErrorNotSupported;
    cudaError_t e = cudaFuncSetAttribute(exp_tc_kernel<T, KIND, ACT, GATED>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)C::kSmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)(most < kSms ? most : kSms);
    exp_tc_kernel<T, KIND, ACT, GATED><<<grid, kThreads, C::kSmem, st>>>(a);
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, int ACT, bool GATED>
cudaError_t run_tc(const ExpCall &c, bool backward, cudaStream_t st) {
    cudaError_t e;
    if (!backward) {
        e = launch_kind<T, kFirst, ACT, GATED>(c, st);
        if (e == cudaSuccess && c.s.mlp) e = launch_kind<T, kSecond, GMM_ACT_NONE, false>(c, st);
        return e;
    }
    if (c.s.mlp) e = launch_kind<T, kDaMlp, ACT, GATED>(c, st);
    else e = launch_kind<T, kDaLin, ACT, false>(c, st);
    if (e == cudaSuccess) e = launch_kind<T, kDx, GMM_ACT_NONE, false>(c, st);
    if (e == cudaSuccess) e = launch_kind<T, kDw1, GMM_ACT_NONE, false>(c, st);
    if (e == cudaSuccess && c.s.mlp) e = launch_kind<T, kDw2, GMM_ACT_NONE, false>(c, st);
    return e;
}

template <typename T, int ACT>
cudaError_t gate_tc(const ExpCall &c, bool backward, cudaStream_t st) {
    return c.s.gated ? run_tc<T, ACT, true>(c, backward, st)
                     : run_tc<T, ACT, false>(c, backward, st);
}

template <typename T> cudaError_t act_tc(const ExpCall &c, bool backward, cudaStream_t st) {
    switch (c.s.act) {
        case GMM_ACT_RELU: return gate_tc<T, GMM_ACT_RELU>(c, backward, st);
        case GMM_ACT_GELU: return gate_tc<T, GMM_ACT_GELU>(c, backward, st);
        case GMM_ACT_SILU: return gate_tc<T, GMM_ACT_SILU>(c, backward, st);
        default: return gate_tc<T, GMM_ACT_NONE>(c, backward, st);
    }
}

}  // namespace

cudaError_t launch_exp_tc(const ExpCall &c, bool backward, cudaStream_t s) {
    return c.s.dt == GMM_BF16 ? act_tc<__nv_bfloat16>(c, backward, s)
                              : act_tc<__half>(c, backward, s);
}

// Partial sums of dresp per row: two halves of each column tile.
int exp_tc_resp_parts(const ExpShape &s) {
    if (!s.mlp) return 2 * ((s.o + Cfg<kDaLin, false>::NB - 1) / Cfg<kDaLin, false>::NB);
    const int nb = s.gated ? Cfg<kDaMlp, true>::NB : Cfg<kDaMlp, false>::NB;
    return 2 * ((s.h + nb - 1) / nb);
}

}  // namespace gmmb
