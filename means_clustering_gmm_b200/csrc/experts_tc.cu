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
//   warps 2..17  epilogue, four warps per TMEM lane quadrant, each a quarter
//                of the tile's columns; a thread owns one row and takes 16
//                columns at a time (eight warps with 32 columns each waited
//                for their loads half of the time).
//
// Operands are used as they lie in memory: a contraction over an array's
// contiguous axis reads it K-major, one over its rows (the weights in the
// backward pass, all operands of the weight gradients) MN-major, so nothing
// is transposed.
//
// Bound, at 8192 points, 2 of 16 gated experts 2048-4096-2048 in bf16: first and
// second together 640 us (1290 TFLOP/s: a stage's 64 KB a pair from L2 take 50
// of its 64 bytes a clock), dx 420 us, dw1 460, dw2 233 (1400 TFLOP/s, the power
// cap), da 778 (1060 TFLOP/s: 128-column products for q need 96 bytes a clock).
// Contractions of one or two stages (128 columns) are bound by the epilogue.
#include "experts.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace gmmb {
namespace {

using namespace tc;

constexpr int kSms = 148;
constexpr int kEpiWarps = 16;
constexpr int kThreads = 64 + kEpiWarps * 32;
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

// Output columns per tile (NB), MMA widths of the (up to two) phases, bytes
// of a stage and the number of stages.  CG = 2: a pair of CTAs takes 256 rows,
// each CTA 128 of them and half of B's rows, which halves what a stage brings
// of B: a 128 x 256 tile moves 48 KB into and 48 KB out of shared memory for
// 512 clocks of products, a pair's half 32 KB each way, which is what 128
// bytes a clock can do.
//
// kDaMlp keeps the pre-activations and q = W2^T dY side by side: q first
// (phase 1, two buffers of 128 columns), then the pre-activations (phase 2).
// Gated, those take the other 256 columns, once: the next tile's phase 1
// covers the epilogue.  Otherwise they are double-buffered too.
//
// W: weight rows (or columns) of the other kinds' tiles.
template <int KIND, bool GATED, int CG, int W> struct Cfg {
    static constexpr bool kGrad = KIND == kDw1 || KIND == kDw2;
    static constexpr bool kTwo = KIND == kDaMlp;
    static constexpr bool kHidden = KIND == kFirst || KIND == kDaMlp;   // columns: hidden units
    static constexpr int NB = kTwo ? 128 : GATED ? W / 2 : W;
    static constexpr int N1 = kTwo ? 128 : W;
    static constexpr int N2 = kTwo ? (GATED ? 256 : 128) : 0;
    static constexpr int kB1 = N1 / CG * kStepK * 2, kB2 = N2 / CG * kStepK * 2;
    static constexpr int kBytesB = kB1 > kB2 ? kB1 : kB2;
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kStages = 192 * 1024 / kStage < 8 ? 192 * 1024 / kStage : 8;
    static constexpr int kPart = NB / 4;   // columns of an epilogue warp
    // what an epilogue warp keeps of its columns' biases (gate and up), fp32
    static constexpr bool kBias = !kGrad && KIND != kDx;
    static constexpr int kBiasBytes = kBias ? kEpiWarps * 2 * 64 * 4 : 0;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kBiasBytes + 256;
    // one CTA per tile is for short segments: only the 32-row groups of A
    // that hold rows are fetched (the products of the others are not used)
    static constexpr bool kSmallA = CG == 1 && !kGrad;
    static constexpr int kBoxA = kSmallA ? 32 : kRowsA;
    static constexpr bool kAMn = kGrad;
    static constexpr bool kBMn1 = kGrad || KIND == kDx || kTwo;
    static constexpr int kTileRows = kRowsA * CG;
    // TMEM columns of tile t's phase 1 and phase 2 accumulators
    __device__ static constexpr uint32_t col1(uint32_t t) {
        return (t & 1) * (kTwo && GATED ? 128 : 256);
    }
    __device__ static constexpr uint32_t col2(uint32_t t) {
        return GATED ? 256 : (t & 1) * 256 + 128;
    }
};

struct Args {
    ExpCall c;
    CUtensorMap a, b, a2, b2;   // phase 1 and phase 2 operands
    CUtensorMap aux;            // rows the epilogue reads (dense form)
    int prefetch_aux;
    int ntn, ntm;               // column tiles; row tiles of one expert's dW
};

struct Bars {
    uint64_t full[8], empty[8], accfull[2], accfree[2], done;
};

// One tile of this CTA: which expert, which rows and columns, how many
// contraction steps.  valid <= 0: the pair's other CTA holds the segment's
// last rows, and nothing of this half is stored.
struct Job {
    int expert, valid, col0, m0, steps1, steps2;
    int64_t row0;
};

template <int KIND, bool GATED, int CG, int W>
__device__ __forceinline__ int total_jobs(const Args &a) {
    return Cfg<KIND, GATED, CG, W>::kGrad ? a.c.s.K * a.ntm * a.ntn
                                       : a.c.rt.tiles(CG * kRowsA) * a.ntn;
}

// What a job needs from memory: loaded a job ahead, one independent load (a
// chain of them at every tile left the products waiting).
template <int KIND, bool GATED, int CG, int W>
__device__ __forceinline__ int4 job_entry(const Args &a, int idx, int total) {
    if (idx >= total) return make_int4(0, 0, 0, 0);
    const int t = idx / a.ntn;
    if constexpr (Cfg<KIND, GATED, CG, W>::kGrad) {
        const int e = t / a.ntm;
        return a.c.rt.ids ? make_int4(e, a.c.rt.seg[e], a.c.rt.cnt[e], 0)
                          : make_int4(0, 0, (int)a.c.rt.N, 0);
    } else {
        return a.c.rt.tile_entry(t, CG * kRowsA);
    }
}
template <int KIND, bool GATED, int CG, int W>
__device__ __forceinline__ Job job_of(const Args &a, int idx, int rank, const int4 &e) {
    using C = Cfg<KIND, GATED, CG, W>;
    Job j;
    const ExpShape &s = a.c.s;
    const int t = idx / a.ntn;
    j.col0 = (idx - t * a.ntn) * C::NB;
    j.expert = e.x;
    if constexpr (C::kGrad) {
        j.m0 = t % a.ntm * C::kTileRows + rank * kRowsA;
        j.row0 = e.y;
        j.valid = kRowsA;
        j.steps1 = (e.z + kStepK - 1) / kStepK;
        j.steps2 = 0;
    } else {
        j.row0 = (int64_t)e.y + rank * kRowsA;
        j.valid = e.z - rank * kRowsA < kRowsA ? e.z - rank * kRowsA : kRowsA;
        j.m0 = 0;
        const int k1 = KIND == kSecond ? s.h : KIND == kDx ? s.first() : C::kTwo ? s.o : s.d;
        const bool none = j.expert >= s.K;
        j.steps1 = none ? 0 : (k1 + kStepK - 1) / kStepK;
        j.steps2 = C::kTwo && !none ? (s.d + kStepK - 1) / kStepK : 0;
    }
    return j;
}

// Sixteen consecutive elements of a row, raw (the first eight where `both` is
// false), and as floats.  wide: 32-byte aligned, one whole sector at once;
// vec: 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load16(const T *p, bool both, bool wide, bool vec,
                                       uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                       "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h == 1 && !both) break;
        uint4 v;
        if (vec) {
            v = *reinterpret_cast<const uint4 *>(p + 8 * h);
        } else {
            __align__(16) T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = p[8 * h + i];
            v = *reinterpret_cast<const uint4 *>(e);
        }
        w[4 * h] = v.x;
        w[4 * h + 1] = v.y;
        w[4 * h + 2] = v.z;
        w[4 * h + 3] = v.w;
    }
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_of(const uint32_t (&r)[16], int i) {
    return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
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
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// Sixteen consecutive results (the first eight where `both` is false).
// wide: 32-byte aligned, one whole sector in one store.
template <typename T>
__device__ __forceinline__ void store16(T *p, const float2 (&v)[8], bool both, bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2<T>(v[i].x, v[i].y);
    if (wide) {
        store32(p, w);
        return;
    }
    uint4 *o = reinterpret_cast<uint4 *>(p);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if (both) o[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16(float *p, const float2 (&v)[8], bool both, bool) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h == 1 && !both) break;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = __float_as_uint(v[4 * h + i].x);
            w[2 * i + 1] = __float_as_uint(v[4 * h + i].y);
        }
        store32(p + 8 * h, w);
    }
}

template <typename T, int KIND, int ACT, bool GATED, int CG, int W>
__global__ void __launch_bounds__(kThreads, 1) exp_tc_kernel(const __grid_constant__ Args a) {
    using C = Cfg<KIND, GATED, CG, W>;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    float *bias_sm = reinterpret_cast<float *>(sm + (size_t)C::kStages * C::kStage);
    Bars *bars = reinterpret_cast<Bars *>(sm + (size_t)C::kStages * C::kStage + C::kBiasBytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert(sizeof(Bars) + 8 <= 256 && C::kStages <= 8, "barrier block");

    const ExpCall &c = a.c;
    const ExpShape &s = c.s;
    const ExpRoute &rt = c.rt;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CG == 2 ? (int)cluster_ctarank() : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;   // this pair's tiles
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->accfull[i], 1);
            mbar_init(&bars->accfree[i], kEpiWarps * CG);
        }
        mbar_init(&bars->done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&a.a);
        prefetch_tensormap(&a.b);
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(tmem_slot, 512);
        } else {
            tmem_alloc(tmem_slot, 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    exp_enter();
    const int total = total_jobs<KIND, GATED, CG, W>(a);

    if (warp == 0) {
        // ================================================ TMA producer
        // Each CTA fetches its own rows of A and its part of B; a pair's
        // bytes are all counted on the barrier of rank 0, whose one arrival
        // expects both CTAs' (a slot is refilled only after the products that
        // read it, so no copy of a later phase can reach an earlier one).
        // The loop is one thread's chain of instructions and was the bound
        // when it recomputed its addresses (660 clocks a stage whose products
        // take 256).
        if (lane == 0) {
            const uint32_t sm0 = smem_u32(sm);
            const uint32_t full0 = CG == 2 ? mapa_u32(&bars->full[0], 0)
                                           : smem_u32(&bars->full[0]);
            uint32_t slot = 0, parity = 1, fill = 0;
            bool ok = true;
            // the next slot, free and expecting `bytes` from this CTA
            auto open = [&](uint32_t bytes) {
                ok = mbar_wait(&bars->empty[slot], parity, c.err, abort_flag);
                if (ok && rank == 0) mbar_arrive_expect_tx(&bars->full[slot], CG * bytes);
                return ok;
            };
            auto next = [&] {
                ++fill;
                if (++slot == (uint32_t)C::kStages) {
                    slot = 0;
                    parity ^= 1;
                }
            };
            int4 entry = job_entry<KIND, GATED, CG, W>(a, first, total);
            for (int idx = first; idx < total && ok; idx += stride) {
                const Job j = job_of<KIND, GATED, CG, W>(a, idx, rank, entry);
                entry = job_entry<KIND, GATED, CG, W>(a, idx + stride, total);
                const int row = (int)j.row0;
                // what the epilogue will read beside the accumulators
                if (a.prefetch_aux)
                    for (int i = 0; i < C::NB; i += 64) tma_prefetch_2d(&a.aux, j.col0 + i, row);
                const int groups = C::kSmallA ? (j.valid + 31) / 32 : 1;
                const uint32_t bytes_a = C::kSmallA ? groups * (kBytesA / 4) : kBytesA;
                // this CTA's first column of B in a phase of N columns
                const int n1 = j.col0 + rank * (C::N1 / CG);
                for (int st = 0, k = 0; st < j.steps1; ++st, k += kStepK) {
                    if (!open(bytes_a + C::kB1)) break;
                    const uint32_t A = sm0 + slot * C::kStage, B = A + kBytesA;
                    const uint32_t bar = full0 + slot * 8;
                    if constexpr (C::kGrad) {
#pragma unroll
                        for (int i = 0; i < kRowsA / 64; ++i)
                            tma_g2s_2d<CG == 2>(A + i * kBlk, &a.a, j.m0 + i * 64, row + k, bar);
#pragma unroll
                        for (int i = 0; i < C::N1 / CG / 64; ++i)
                            tma_g2s_2d<CG == 2>(B + i * kBlk, &a.b, n1 + i * 64, row + k, bar);
                    } else {
                        for (int i = 0; i < groups; ++i)
                            tma_g2s_2d<CG == 2>(A + i * (kBytesA / 4), &a.a, k, row + i * 32, bar);
                        if constexpr (C::kBMn1) {
#pragma unroll
                            for (int i = 0; i < C::N1 / CG / 64; ++i)
                                tma_g2s_3d<CG == 2>(B + i * kBlk, &a.b, n1 + i * 64, k, j.expert,
                                                    bar);
                        } else if constexpr (KIND == kFirst && GATED) {
                            // the tile's gate rows, then its up rows: one each
                            // for a pair's CTAs
                            tma_g2s_3d<CG == 2>(B, &a.b, k, j.col0 + rank * s.h, j.expert, bar);
                            if constexpr (CG == 1)
                                tma_g2s_3d<false>(B + C::kB1 / 2, &a.b, k, j.col0 + s.h, j.expert,
                                                  bar);
                        } else {
                            tma_g2s_3d<CG == 2>(B, &a.b, k, n1, j.expert, bar);
                        }
                    }
                    next();
                }
                if constexpr (C::kTwo) {
                    const int n2 = j.col0 + (GATED ? rank * s.h : rank * (C::N2 / CG));
                    for (int st = 0, k = 0; st < j.steps2 && ok; ++st, k += kStepK) {
                        if (!open(bytes_a + C::kB2)) break;
                        const uint32_t A = sm0 + slot * C::kStage, B = A + kBytesA;
                        const uint32_t bar = full0 + slot * 8;
                        for (int i = 0; i < groups; ++i)
                            tma_g2s_2d<CG == 2>(A + i * (kBytesA / 4), &a.a2, k, row + i * 32, bar);
                        tma_g2s_3d<CG == 2>(B, &a.b2, k, n2, j.expert, bar);
                        if constexpr (GATED && CG == 1)
                            tma_g2s_3d<false>(B + C::kB2 / 2, &a.b2, k, j.col0 + s.h, j.expert,
                                              bar);
                        next();
                    }
                }
            }
            // no copy in flight at teardown: rank 0's barriers count both
            // CTAs' copies (the cluster barrier below holds the other back),
            // and the other CTA sees the last of its slots released, so that
            // no arrival reaches it after it is gone
            for (uint32_t f = fill > (uint32_t)C::kStages ? fill - C::kStages : 0; f < fill; ++f)
                mbar_wait_drain(rank == 0 ? &bars->full[f % C::kStages]
                                          : &bars->empty[f % C::kStages],
                                (f / C::kStages) & 1, c.err);
        }
    } else if (warp == 1) {
        // ================================================ MMA issuer
        if (lane == 0 && rank == 0) {
            constexpr bool kBf = !__is_same(T, __half);
            constexpr uint32_t bf = kBf ? idesc_bf16(128, 64, false, false) -
                                              idesc_f16(128, 64, false, false)
                                        : 0;
            constexpr uint32_t id1 = idesc_f16(kRowsA * CG, C::N1, C::kAMn, C::kBMn1) + bf;
            constexpr uint32_t id2 = idesc_f16(kRowsA * CG, C::N2 ? C::N2 : 64, false, false) + bf;
            const uint64_t dA = smem_desc(smem_u32(sm), C::kAMn ? kBlk : 16, 1024, kSwz128);
            const uint64_t dB1 = smem_desc(smem_u32(sm + kBytesA), C::kBMn1 ? kBlk : 16, 1024,
                                           kSwz128);
            const uint64_t dB2 = smem_desc(smem_u32(sm + kBytesA), 16, 1024, kSwz128);
            auto product = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t id, bool add) {
                if constexpr (CG == 2) mma_f16_pair(d, da, db, id, add ? 1u : 0u);
                else mma_f16(d, da, db, id, add ? 1u : 0u);
            };
            auto commit = [&](uint64_t *bar) {
                if constexpr (CG == 2) mma_commit_pair(bar);
                else mma_commit(bar);
            };
            auto free_wait = [&](int buf, uint32_t parity) {
                if constexpr (CG == 2)
                    return mbar_wait_cluster(&bars->accfree[buf], parity, c.err, abort_flag);
                else
                    return mbar_wait(&bars->accfree[buf], parity, c.err, abort_flag);
            };
            uint32_t slot = 0, parity = 0, tile = 0;
            bool ok = true;
            // one stage's products into d; `fresh`: the first overwrites
            auto stage = [&](uint32_t d, uint64_t dB, uint32_t id, uint32_t step_b, bool fresh) {
                ok = mbar_wait(&bars->full[slot], parity, c.err, abort_flag);
                if (!ok) return;
                tc_fence_after();
                const uint32_t off = slot * (C::kStage >> 4);
#pragma unroll
                for (uint32_t kk = 0; kk < kStepK / 16; ++kk)
                    product(d, dA + off + kk * ((C::kAMn ? 2048 : 32) >> 4), dB + off + kk * step_b,
                            id, !fresh || kk > 0);
                commit(&bars->empty[slot]);
                if (++slot == (uint32_t)C::kStages) {
                    slot = 0;
                    parity ^= 1;
                }
            };
            int4 entry = job_entry<KIND, GATED, CG, W>(a, first, total);
            for (int idx = first; idx < total && ok; idx += stride, ++tile) {
                const Job j = job_of<KIND, GATED, CG, W>(a, idx, 0, entry);
                entry = job_entry<KIND, GATED, CG, W>(a, idx + stride, total);
                const int buf = tile & 1;
                if (!free_wait(buf, ((tile >> 1) & 1) ^ 1)) break;
                tc_fence_after();
                const uint32_t d1 = tmem + C::col1(tile);
                for (int st = 0; st < j.steps1 && ok; ++st)
                    stage(d1, dB1, id1, (C::kBMn1 ? 2048 : 32) >> 4, st == 0);
                if constexpr (C::kTwo) {
                    // the single phase-2 accumulator: the tile before is read
                    if (GATED && ok && tile > 0 && j.steps2 > 0) {
                        ok = free_wait((tile - 1) & 1, ((tile - 1) >> 1) & 1);
                        tc_fence_after();
                    }
                    const uint32_t d2 = tmem + C::col2(tile);
                    for (int st = 0; st < j.steps2 && ok; ++st)
                        stage(d2, dB2, id2, 32 >> 4, st == 0);
                }
                if (ok) commit(&bars->accfull[buf]);
            }
            if constexpr (CG == 2) mma_commit_pair_local(&bars->done);
            else mma_commit(&bars->done);
            mbar_wait_drain(&bars->done, 0, c.err);   // no MMA in flight at teardown
        }
    } else {
        // ================================================ epilogue
        const int q = warp & 3, pt = (warp - 2) >> 2, m = q * 32 + lane;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        constexpr int kPart = C::kPart;
        float *gate_b = bias_sm + (warp - 2) * 128, *up_b = gate_b + 64;
        // columns of the result, and of the rows that are added or multiplied
        const int width = KIND == kDw2                        ? s.h
                          : KIND == kDw1 || KIND == kDx       ? s.d
                          : KIND == kSecond                   ? s.o
                          : s.mlp                             ? s.h
                                                              : s.o;
        // this kind reads a row of another array beside the accumulators
        const bool with_res = (KIND == kSecond || (KIND == kFirst && !s.mlp)) && s.direct() && c.res;
        const bool with_aux = KIND == kDaLin || with_res;
        const void *aux0 = KIND == kDaLin ? c.dy : c.res;
        const bool aux_vec = ((uintptr_t)aux0 & 15) == 0;
        const bool aux_wide = width % 16 == 0 && ((uintptr_t)aux0 & 31) == 0;
        // (workspace rows are aligned; the caller's arrays may be to 16 bytes)
        const void *dst = KIND == kDw1 ? c.dw1 : KIND == kDw2 ? c.dw2 : KIND == kDx ? c.dx : c.y;
        const bool wide = width % 16 == 0 && ((uintptr_t)dst & 31) == 0;
        uint32_t tile = 0;
        int4 entry = job_entry<KIND, GATED, CG, W>(a, first, total);
        for (int idx = first; idx < total; idx += stride, ++tile) {
            const Job j = job_of<KIND, GATED, CG, W>(a, idx, rank, entry);
            entry = job_entry<KIND, GATED, CG, W>(a, idx + stride, total);
            const int buf = tile & 1, cw = j.col0 + pt * kPart;   // this warp's first column
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
            if constexpr (C::kBias) {
                // every lane has read the biases of the tile before: its
                // columns end in branches, behind which nothing else says so
                __syncwarp();
                const T *b = (const T *)(KIND == kSecond ? c.b2 : c.b1);
                if (b && !none) b += (size_t)j.expert * (KIND == kSecond ? s.o : s.first());
#pragma unroll
                for (int i = lane; i < kPart; i += 32) {
                    const bool in = b && !none && cw + i < width;
                    gate_b[i] = in ? to_float(b[cw + i]) : 0.f;
                    if (GATED) up_b[i] = in ? to_float(b[width + cw + i]) : 0.f;
                }
            }
            // the other array's row, 16 columns ahead of their use
            const T *aux = (const T *)aux0 + tok * width;
            uint32_t next[8] = {};
            auto fetch = [&](int col) {
                if (valid && col < width)
                    load16(aux + col, col + 8 < width, aux_wide, aux_vec, next);
            };
            if (with_aux) fetch(cw);
            // and the next job's part of it (one 128-byte line a row) for L2:
            // points' rows are scattered
            int64_t next_pair = -1;
            int next_col = 0;
            if (with_aux && !s.dense && idx + stride < total) {
                const Job jn = job_of<KIND, GATED, CG, W>(a, idx + stride, rank, entry);
                next_col = jn.col0 + pt * kPart;
                if (m < jn.valid && next_col < width) next_pair = rt.pair(jn.row0 + m);
            }
            __syncwarp();
            // (a weight gradient's contraction is over its expert's points, of
            // which there may be 2^31)
            const long long limit =
                kWaitLimitCycles + (C::kGrad ? j.steps1 * kStepLimitCycles : 0);
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->accfull[buf], (tile >> 1) & 1, c.err,
                                                   abort_flag, limit)))
                break;
            tc_fence_after();
            // column 0 of the (last phase's) accumulator, and q's
            const uint32_t acc = tmem + (C::kTwo ? C::col2(tile) : C::col1(tile)) + lane_base;
            const uint32_t accq = tmem + C::col1(tile) + lane_base;
            if (next_pair >= 0)
                asm volatile("prefetch.global.L2 [%0];" ::"l"((const T *)aux0 +
                                                              rt.token(next_pair) * width +
                                                              next_col));
            const bool has = j.steps1 > 0;   // otherwise the accumulators were not written
            float part = 0.f;
            // the accumulators go back as soon as they are in registers
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        mbar_arrive_cluster_cta(mapa_u32(&bars->accfree[buf], 0));
                    else
                        mbar_arrive(&bars->accfree[buf]);
                }
            };
            const int columns = min(width - cw, kPart);   // of this warp
            if (columns <= 0) release();
#pragma unroll 1
            for (int at = 0; at < columns; at += 16) {
                const int c0 = pt * kPart + at, col = j.col0 + c0;
                const bool both = col + 8 < width;
                uint32_t r0[16], r1[16], r2[16];
                uint32_t now[8];
                __syncwarp();   // the loads below are warp-wide
                tmem_ld16(acc + c0, r0);
                if constexpr (GATED) tmem_ld16(acc + C::NB + c0, r1);
                if constexpr (C::kTwo) tmem_ld16(accq + c0, r2);
                if (with_aux) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) now[i] = next[i];
                    if (c0 + 16 < (pt + 1) * kPart) fetch(col + 16);
                }
                tmem_ld_wait();
                if (at + 16 >= columns) release();
                float2 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = pair_of(r0, i);
                // columns of this group that have a value (padded copies end
                // with hidden units that do not exist)
                const int live = !has ? 0 : C::kHidden ? c.units - col : 16;
                if (live < 16)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i >= live) {
                            if (i & 1) x[i / 2].y = 0.f;
                            else x[i / 2].x = 0.f;
                            if constexpr (GATED) r1[i] = 0u;
                            if constexpr (C::kTwo) r2[i] = 0u;
                        }
                if constexpr (C::kBias) {
                    const float4 *gb = reinterpret_cast<const float4 *>(gate_b + c0 - pt * kPart);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 b = gb[i];
                        x[2 * i] = __fadd2_rn(x[2 * i], make_float2(b.x, b.y));
                        x[2 * i + 1] = __fadd2_rn(x[2 * i + 1], make_float2(b.z, b.w));
                    }
                }
                float2 up[8];
                if constexpr (GATED) {
                    const float4 *ub = reinterpret_cast<const float4 *>(up_b + c0 - pt * kPart);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 b = ub[i];
                        up[2 * i] = __fadd2_rn(pair_of(r1, 2 * i), make_float2(b.x, b.y));
                        up[2 * i + 1] = __fadd2_rn(pair_of(r1, 2 * i + 1), make_float2(b.z, b.w));
                    }
                }
                if constexpr (C::kGrad) {
                    const int M = KIND == kDw2 ? s.o : s.first();
                    T *out = (T *)(KIND == kDw2 ? c.dw2 : c.dw1);
                    if (j.m0 + m < M)
                        store16(out + ((size_t)j.expert * M + j.m0 + m) * width + col, x, both,
                                wide);
                } else if constexpr (KIND == kDx) {
                    if (valid) {
                        if (s.direct()) store16((T *)c.dx + tok * width + col, x, both, wide);
                        else store16(c.slots + pair * width + col, x, both, true);
                    }
                } else if constexpr (KIND == kDaLin || KIND == kDaMlp) {
                    if (none || j.valid <= 0) continue;
                    T *da = (T *)c.da + row * s.first() + col;
                    const bool whole = width % 16 == 0;
                    float2 hs[8], d2[8], sum = splat(0.f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 f, df, qq;
                        act_pair<ACT>(x[i], f, df);
                        if constexpr (KIND == kDaMlp) qq = pair_of(r2, i);
                        else qq = unpack2(now[i], T{});
                        const float2 gq = __fmul2_rn(splat(g), qq);
                        float2 fu = f, du = df;
                        if constexpr (GATED) {
                            fu = __fmul2_rn(f, up[i]);
                            du = __fmul2_rn(df, up[i]);
                            d2[i] = __fmul2_rn(gq, f);
                        }
                        if (i < 4 || both) sum = __ffma2_rn(qq, fu, sum);
                        x[i] = __fmul2_rn(gq, du);
                        if constexpr (KIND == kDaMlp) hs[i] = __fmul2_rn(splat(g), fu);
                    }
                    // dresp: fp32, of accumulators that truncate, which costs 1e-9
                    // of q and of the pre-activations with each contraction index.
                    // Adding pieces of the contraction in fp32 here instead would
                    // take 96 registers a thread, all there are, and TMEM has no
                    // columns left for such sums beside a gated tile's.
                    part += sum.x + sum.y;
                    // rows past the segment are zeros: the weight gradients
                    // contract over them
                    if (!valid)
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = d2[i] = hs[i] = splat(0.f);
                    store16(da, x, both, whole);
                    if constexpr (GATED) store16(da + width, d2, both, whole);
                    if constexpr (KIND == kDaMlp)
                        store16((T *)c.hid + row * width + col, hs, both, whole);
                } else {
                    if (!valid) continue;
                    if constexpr (KIND == kFirst) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float2 f, df;
                            act_pair<ACT>(x[i], f, df);
                            x[i] = f;
                            if constexpr (GATED) x[i] = __fmul2_rn(f, up[i]);
                        }
                    }
                    if (KIND == kFirst && s.mlp) {
                        // rounded to the type: the second product's operand
                        if (!none)
                            store16((T *)c.hid + row * width + col, x, both, width % 16 == 0);
                    } else if (s.direct()) {
                        // (a point without an expert: what the sum over none gives)
                        const float gv = none ? 0.f : g;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (none) x[i] = splat(0.f);
                            x[i] = __ffma2_rn(splat(gv), x[i],
                                              with_res ? unpack2(now[i], T{}) : splat(0.f));
                        }
                        store16((T *)c.y + tok * width + col, x, both, wide);
                    } else {
                        store16(c.slots + pair * width + col, x, both, true);
                    }
                }
            }
            if constexpr (KIND == kDaLin || KIND == kDaMlp) {
                if (valid && !none && c.dresp && cw < width)
                    c.rpart[pair * c.nrpart + cw / kPart] = part;
            }
        }
    }
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        if constexpr (CG == 2) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------- host side
template <typename T, int KIND, int ACT, bool GATED, int CG, int W>
cudaError_t launch_kind(const ExpCall &c, cudaStream_t st) {
    using C = Cfg<KIND, GATED, CG, W>;
    const ExpShape &s = c.s;
    Args a;
    a.c = c;
    TensorMaps maps{s.dt};
    int width = 0, mrows = 0;
    switch (KIND) {
        case kFirst:
        case kDaLin:
            width = s.mlp ? s.h : s.o;
            maps.make(&a.a, c.xrows, s.d, c.point_rows, 0, C::kBoxA);
            maps.make(&a.b, c.w1, s.d, s.first(), s.K, GATED ? C::NB : C::N1 / CG);
            break;
        case kDaMlp:
            width = s.h;
            maps.make(&a.a, c.dyrows, s.o, c.point_rows, 0, C::kBoxA);
            maps.make(&a.b, c.w2, s.h, s.o, s.K, kStepK);
            maps.make(&a.a2, c.xrows, s.d, c.point_rows, 0, C::kBoxA);
            maps.make(&a.b2, c.w1, s.d, s.first(), s.K, GATED ? C::NB : C::N2 / CG);
            break;
        case kSecond:
            width = s.o;
            maps.make(&a.a, c.hid, s.h, c.max_rows, 0, C::kBoxA);
            maps.make(&a.b, c.w2, s.h, s.o, s.K, C::N1 / CG);
            break;
        case kDx:
            width = s.d;
            maps.make(&a.a, c.da, s.first(), c.da_rows, 0, C::kBoxA);
            maps.make(&a.b, c.w1, s.d, s.first(), s.K, kStepK);
            break;
        case kDw1:
            width = s.d;
            mrows = s.first();
            maps.make(&a.a, c.da, s.first(), c.da_rows, 0, kStepK);
            maps.make(&a.b, c.xrows, s.d, c.point_rows, 0, kStepK);
            break;
        case kDw2:
            width = s.h;
            mrows = s.o;
            maps.make(&a.a, c.dyrows, s.o, c.point_rows, 0, kStepK);
            maps.make(&a.b, c.hid, s.h, c.max_rows, 0, kStepK);
            break;
    }
    const void *aux = KIND == kDaLin ? c.dy : KIND == kSecond || KIND == kFirst ? c.res : nullptr;
    a.prefetch_aux = s.dense && aux && ((uintptr_t)aux & 15) == 0 && !(KIND == kFirst && s.mlp);
    if (a.prefetch_aux) maps.make(&a.aux, aux, width, s.N, 0, kRowsA);
    if (!maps.ok) return cudaErrorNotSupported;
    a.ntn = (width + C::NB - 1) / C::NB;
    a.ntm = (mrows + C::kTileRows - 1) / C::kTileRows;
    const int64_t most = C::kGrad ? (int64_t)s.K * a.ntm * a.ntn : (int64_t)c.rt.max_tiles * a.ntn;
    if (most > 0x7fff0000) return cudaErrorNotSupported;
    const auto kernel = exp_tc_kernel<T, KIND, ACT, GATED, CG, W>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (CG == 2) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {2, 1, 1};
        cfg.numAttrs = 2;
    }
    // one wave: as many pairs as can be resident (a GPC with an odd number of
    // SMs leaves one out)
    cfg.gridDim = dim3(kSms);
    int wave = kSms;
    if (CG == 2) {
        static DeviceConstant pairs;
        const int resident = pairs.get([&] {
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            return e != cudaSuccess ? 0 : n < 1 ? 2 : 2 * n;
        });
        if (e != cudaSuccess) return e;
        wave = resident < kSms ? resident : kSms;
    }
    const int64_t ctas = most * CG;
    cfg.gridDim = dim3((unsigned)(ctas < wave ? ctas : wave));
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return e;
    note_launches(1);
    return cudaGetLastError();
}

// Products whose rows are points run in pairs when the segments are long
// enough (kExpPairRows); a weight gradient when its own rows fill pairs too.
template <typename T, int KIND, int ACT, bool GATED, int W>
cudaError_t launch_rows_w(const ExpCall &c, cudaStream_t st) {
    return c.rt.tile_rows == 2 * kRowsA ? launch_kind<T, KIND, ACT, GATED, 2, W>(c, st)
                                        : launch_kind<T, KIND, ACT, GATED, 1, W>(c, st);
}
// Tiles are 256 weight rows wide, 128 where a result has no more columns.
// (Choosing 128 or 64 so that short segments fill the last round of SMs more
// evenly changed nothing: 333 points, 32 experts of 1000-616-520 gated 49 and
// 51 us, 128 points, 8 experts of 2048-1024-2048 gated 52 and 50.)
template <typename T, int KIND, int ACT, bool GATED>
cudaError_t launch_rows(const ExpCall &c, cudaStream_t st) {
    const int width = KIND == kDx ? c.s.d : KIND == kSecond || !c.s.mlp ? c.s.o : 256;
    if constexpr (KIND != kDaMlp && !GATED)
        if (width <= 128) return launch_rows_w<T, KIND, ACT, GATED, 128>(c, st);
    return launch_rows_w<T, KIND, ACT, GATED, 256>(c, st);
}
template <typename T, int KIND, int W>
cudaError_t launch_grad_w(const ExpCall &c, cudaStream_t st) {
    const int tiles = ((KIND == kDw2 ? c.s.o : c.s.first()) + kRowsA - 1) / kRowsA;
    return c.rt.tile_rows == 2 * kRowsA && (tiles % 2 == 0 || tiles > 8)
               ? launch_kind<T, KIND, GMM_ACT_NONE, false, 2, W>(c, st)
               : launch_kind<T, KIND, GMM_ACT_NONE, false, 1, W>(c, st);
}
template <typename T, int KIND> cudaError_t launch_grad(const ExpCall &c, cudaStream_t st) {
    return (KIND == kDw2 ? c.s.h : c.s.d) <= 128 ? launch_grad_w<T, KIND, 128>(c, st)
                                                 : launch_grad_w<T, KIND, 256>(c, st);
}

template <typename T, int ACT, bool GATED>
cudaError_t run_tc(const ExpCall &c, bool backward, cudaStream_t st) {
    cudaError_t e;
    if (!backward) {
        e = launch_rows<T, kFirst, ACT, GATED>(c, st);
        if (e == cudaSuccess && c.s.mlp) e = launch_rows<T, kSecond, GMM_ACT_NONE, false>(c, st);
        return e;
    }
    if (c.s.mlp) e = launch_rows<T, kDaMlp, ACT, GATED>(c, st);
    else e = c.plain_da() ? cudaSuccess : launch_rows<T, kDaLin, ACT, false>(c, st);
    if (e == cudaSuccess) e = launch_rows<T, kDx, GMM_ACT_NONE, false>(c, st);
    if (e == cudaSuccess) e = launch_grad<T, kDw1>(c, st);
    if (e == cudaSuccess && c.s.mlp) e = launch_grad<T, kDw2>(c, st);
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

// Partial sums of dresp per row: one from each epilogue warp of a tile.
int exp_tc_resp_parts(const ExpShape &s) {
    const int width = s.mlp ? s.h : s.o, part = s.mlp || width <= 128 ? 32 : 64;
    return (width + part - 1) / part;
}

}  // namespace gmmb
