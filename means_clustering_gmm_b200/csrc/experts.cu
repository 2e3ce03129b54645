// C ABI of the experts' products (declared in include/gmm_b200.h): argument
// checks, workspace layout and the order of the launches.
#include "experts.h"

#include <climits>

using namespace gmmb;

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool valid_shape(const gmm_expert_shape *s, bool mlp) {
    if (!s || s->N < 1 || s->d < 1 || s->d > GMM_EXPERT_MAX_DIM || s->o < 1 ||
        s->o > GMM_EXPERT_MAX_DIM || s->K < 1 || s->K > GMM_EXPERT_MAX_K || s->r < 0 ||
        s->r > kTopMax)
        return false;
    if (mlp ? (s->h < 1 || s->h > GMM_EXPERT_MAX_DIM) : s->h != 0) return false;
    if (s->dtype != GMM_F32 && s->dtype != GMM_BF16 && s->dtype != GMM_F16) return false;
    if (s->activation < GMM_ACT_NONE || s->activation > GMM_ACT_SILU) return false;
    if (s->gated != 0 && (s->gated != 1 || !mlp)) return false;
    if (s->r == 0 && s->K != 1) return false;
    // rows are counted in 32 bits, segments rounded up to whole tiles
    const int64_t rows = ((int64_t)1 << 31) - (int64_t)(GMM_EXPERT_MAX_K + 2) * kExpTile;
    return s->N <= rows / (s->r ? s->r : 1);
}

ExpShape make_shape(const gmm_expert_shape *s) {
    ExpShape p;
    p.N = s->N;
    p.P = s->N * (s->r ? s->r : 1);
    p.d = s->d;
    p.h = s->h;
    p.o = s->o;
    p.K = s->K;
    p.r = s->r;
    p.gated = s->gated == 1;
    p.gh = p.gated ? 2 * p.h : p.h;
    p.dt = (gmm_dtype)s->dtype;
    p.act = s->activation;
    p.mlp = s->h > 0;
    p.dense = s->r == 0;
    return p;
}

// Tensor maps want rows of whole 16-byte units: other widths run on copies.
int up8(int w) { return (w + 7) / 8 * 8; }
bool padded(const ExpShape &p, int path) {
    return path == 2 && (p.d % 8 || p.h % 8 || p.o % 8);
}
ExpShape pad_shape(ExpShape p) {
    p.d = up8(p.d);
    p.h = up8(p.h);
    p.o = up8(p.o);
    p.gh = p.gated ? 2 * p.h : p.h;
    return p;
}

int path_of(const ExpShape &p, bool backward, uint32_t flags) {
    if ((flags & GMM_FLAG_FORCE_SIMT) || p.dt == GMM_F32) return 0;
    if (!padded(p, 2) && !backward && p.N <= kExpFewPoints && p.P <= GMM_EXPERT_FEW_PAIRS)
        return 1;
    return 2;
}

struct Layout {
    size_t cnt, seg, tile_at, pair_at, ntiles, row_pair, hist, hid, da, xrows, dyrows, slots,
        rpart, colpart, total;
    int64_t max_rows;
    int max_tiles, nrpart;
    size_t esize;
};

// `p`: the padded shape where the call runs on copies.
Layout layout_of(const ExpShape &p, bool backward, int path) {
    Layout L;
    const int64_t segs = p.dense ? 1 : (p.K + 1 < p.P ? p.K + 1 : p.P);
    L.max_tiles = (int)((p.P + segs * (kExpTile - 1)) / kExpTile);
    if (L.max_tiles < 1) L.max_tiles = 1;
    L.max_rows = (int64_t)L.max_tiles * kExpTile;
    L.esize = path == 0 ? 4 : 2;
    const int width = p.mlp ? p.h : p.o;
    L.nrpart = path == 0 ? (width + 63) / 64 : exp_tc_resp_parts(p);
    size_t o = kAlign;   // error word
    auto take = [&](size_t &off, size_t bytes) {
        off = o;
        o = align_up(o + bytes);
    };
    const size_t KK = (size_t)p.K + 1;
    const size_t chunks = p.dense ? 0 : (size_t)((p.P + exp_chunk(p.K) - 1) / exp_chunk(p.K));
    take(L.cnt, p.dense ? 0 : KK * 4);
    take(L.seg, p.dense ? 0 : (KK + 1) * 4);
    take(L.tile_at, p.dense ? 0 : (size_t)L.max_tiles * 16);
    take(L.pair_at, p.dense ? 0 : (size_t)L.max_tiles * 16);
    take(L.ntiles, 8);
    take(L.row_pair, p.dense ? 0 : (size_t)L.max_rows * 4);
    take(L.hist, chunks * KK * 4);
    take(L.hid, p.mlp ? (size_t)L.max_rows * p.h * L.esize : 0);
    take(L.da, backward ? (size_t)L.max_rows * p.first() * L.esize : 0);
    const bool sorted = path == 2 && !p.dense;
    take(L.xrows, sorted ? (size_t)L.max_rows * p.d * 2 : 0);
    take(L.dyrows, sorted && backward && p.mlp ? (size_t)L.max_rows * p.o * 2 : 0);
    const int wide = backward ? p.d : p.o;
    take(L.slots, p.direct() ? 0 : (size_t)p.P * wide * 4);
    take(L.rpart, backward ? (size_t)p.P * L.nrpart * 4 : 0);
    // partial bias gradients
    const size_t cols =
        backward ? (size_t)exp_colsum_slices(p) * (p.first() + (p.mlp ? p.o : 0)) : 0;
    take(L.colpart, cols * p.K * 4);
    L.total = o;
    return L;
}

ExpCall make_call(const ExpShape &p, const Layout &L, void *ws, const int32_t *ids) {
    ExpCall c = {};
    char *b = (char *)ws;
    c.s = p;
    c.err = (int *)b;
    c.rt.cnt = (int *)(b + L.cnt);
    c.rt.seg = (int *)(b + L.seg);
    c.rt.tile_at = (int4 *)(b + L.tile_at);
    c.rt.pair_at = (int4 *)(b + L.pair_at);
    c.rt.ntiles = (int *)(b + L.ntiles);
    c.rt.row_pair = (int *)(b + L.row_pair);
    c.rt.hist = (int *)(b + L.hist);
    c.rt.chunk = exp_chunk(p.K);
    c.rt.ids = ids;
    c.rt.N = p.N;
    c.rt.P = p.P;
    c.rt.K = p.K;
    c.rt.r = p.r ? p.r : 1;
    c.rt.max_tiles = L.max_tiles;
    c.rt.tile_rows = p.P >= kExpPairRows * p.K ? 2 * kExpTile : kExpTile;
    c.hid = b + L.hid;
    c.da = b + L.da;
    c.xrows = b + L.xrows;
    c.dyrows = b + L.dyrows;
    c.point_rows = p.dense ? p.N : L.max_rows;
    c.slots = (float *)(b + L.slots);
    c.rpart = (float *)(b + L.rpart);
    c.colpart = (float *)(b + L.colpart);
    c.max_rows = c.da_rows = L.max_rows;
    c.nrpart = L.nrpart;
    c.esize = L.esize;
    return c;
}

bool known_flags(uint32_t flags) { return (flags & ~(uint32_t)GMM_FLAG_FORCE_SIMT) == 0; }

// The checks the four entry points share.  `big` arrays are 16-byte aligned
// where their rows are whole 16-byte units; others are read and written element by
// element (the copies of 16-bit types, the CUDA cores' scalar form) and aligned
// to that, as `small` ones are.
struct Checks {
    bool ok = true;
    size_t elem;
    void big(const void *p, int width) {
        ok = ok && p && aligned(p, width * elem % 16 == 0 ? 16 : elem);
    }
    void small(const void *p, size_t a) { ok = ok && (!p || aligned(p, a)); }
    void routing(const gmm_expert_shape *s, const int32_t *ids, const float *resp) {
        ok = ok && (ids != nullptr) == (s->r > 0) && (s->r > 0 || !resp);
        small(ids, 4);
        small(resp, 4);
    }
    void pair(const void *a, const void *grad) {   // an optional input and its gradient
        ok = ok && (a == nullptr) == (grad == nullptr);
    }
    void workspace(const void *ws, size_t have, size_t need) {
        ok = ok && ws && aligned(ws, kAlign) && have >= need;
    }
};

// The padded copies of a call's arrays, at the end of its workspace.  take()
// gives an input its copy, give() an output its padded form; both leave arrays
// alone whose own widths need nothing.
struct Pads {
    bool on;
    size_t o;       // offset past what is taken
    char *ws;       // NULL: only sizes are wanted
    PadJobs in, out;
    Pads(bool on_, size_t base, void *w) : on(on_), o(base), ws((char *)w), in(), out() {}
    void *job(PadJobs &list, const void *a, int planes, int rows, int cols, int rows_to,
              int cols_to, int per_expert) {
        if (!on || (rows == rows_to && cols == cols_to)) return const_cast<void *>(a);
        void *wide = ws + o;
        o = align_up(o + (size_t)planes * rows_to * cols_to * 2);
        if (!ws || !a) return nullptr;
        list.j[list.n++] = PadJob{const_cast<void *>(a), wide, planes, rows, cols, rows_to,
                                  cols_to, per_expert};
        return wide;
    }
    // every array of a call, in `c` on entry as the caller gave it
    void arrays(ExpCall &c, const ExpShape &p, bool backward) {
        const int n = (int)p.N, dp = up8(p.d), hp = up8(p.h), op = up8(p.o);
        const int half = p.gated ? 2 : 1;   // W1's blocks of rows per expert
        const int r1 = p.mlp ? p.h : p.o, r1p = p.mlp ? hp : op;
        c.x = job(in, c.x, 1, n, p.d, n, dp, 0);
        c.w1 = job(in, c.w1, p.K * half, r1, p.d, r1p, dp, half);
        c.b1 = job(in, c.b1, p.K * half, 1, r1, 1, r1p, half);
        if (p.mlp) {
            c.w2 = job(in, c.w2, p.K, p.o, p.h, op, hp, 1);
            c.b2 = job(in, c.b2, p.K, 1, p.o, 1, op, 1);
        }
        if (!backward) {
            c.res = job(in, c.res, 1, n, p.o, n, op, 0);
            c.y = job(out, c.y, 1, n, p.o, n, op, 0);
            return;
        }
        c.dy = job(in, c.dy, 1, n, p.o, n, op, 0);
        c.dx = job(out, c.dx, 1, n, p.d, n, dp, 0);
        c.dw1 = job(out, c.dw1, p.K * half, r1, p.d, r1p, dp, half);
        c.db1 = job(out, c.db1, p.K * half, 1, r1, 1, r1p, half);
        if (p.mlp) {
            c.dw2 = job(out, c.dw2, p.K, p.o, p.h, op, hp, 1);
            c.db2 = job(out, c.db2, p.K, 1, p.o, 1, op, 1);
        }
    }
};

size_t total_bytes(const ExpShape &p, bool backward, uint32_t flags) {
    const int path = path_of(p, backward, flags);
    const bool on = padded(p, path);
    Pads pads(on, layout_of(on ? pad_shape(p) : p, backward, path).total, nullptr);
    ExpCall c = {};
    pads.arrays(c, p, backward);
    return pads.o;
}

// One checked call: routing, copies, products, the sums after them.
gmm_status run(ExpCall &c, const ExpShape &p, const Layout &L, int path, bool backward, void *ws,
               cudaStream_t s) {
    if (path == 1) return launch_exp_few(c, s) == cudaSuccess ? GMM_OK : GMM_ERR_CUDA;
    Pads pads(padded(p, path), L.total, ws);
    pads.arrays(c, p, backward);
    pads.in.cnt = p.dense ? nullptr : c.rt.cnt;
    cudaError_t e = launch_exp_route(c, s);
    if (e == cudaSuccess) e = launch_exp_pad(pads.in, false, s);
    if (path == 0) {
        if (e == cudaSuccess) e = launch_exp_simt(c, backward, s);
    } else {
        const bool plain = backward && c.plain_da();
        if (plain && !c.s.dense) c.dyrows = c.da;
        if (c.s.dense) {
            c.xrows = const_cast<void *>(c.x);
            c.dyrows = const_cast<void *>(c.dy);
            if (plain) {
                c.da = c.dyrows;
                c.da_rows = p.N;
            }
        } else if (e == cudaSuccess) {
            e = launch_exp_gather(c, backward, s);
        }
        if (e == cudaSuccess) e = launch_exp_tc(c, backward, s);
    }
    if (e == cudaSuccess) e = launch_exp_combine(c, backward, s);
    if (e == cudaSuccess && backward) e = launch_exp_bias_grads(c, s);
    if (e == cudaSuccess) e = launch_exp_pad(pads.out, true, s);
    return e == cudaSuccess ? GMM_OK : GMM_ERR_CUDA;
}

gmm_status forward(const gmm_expert_shape *shape, bool mlp, const void *X, const int32_t *ids,
                   const float *resp, const void *W1, const void *b1, const void *W2,
                   const void *b2, const void *residual, void *Y, void *ws, size_t ws_bytes,
                   uint32_t flags, cudaStream_t s) {
    if (!valid_shape(shape, mlp) || !known_flags(flags)) return GMM_ERR_INVALID_ARG;
    const ExpShape p = make_shape(shape);
    const int path = path_of(p, false, flags);
    const ExpShape q = padded(p, path) ? pad_shape(p) : p;
    const Layout L = layout_of(q, false, path);
    Checks k;
    k.elem = p.dt == GMM_F32 ? 4 : 2;
    k.big(X, p.d);
    k.big(W1, p.d);
    if (mlp) k.big(W2, p.h);
    k.big(Y, p.o);
    k.small(b1, k.elem);
    k.small(b2, k.elem);
    k.small(residual, k.elem);
    k.routing(shape, ids, resp);
    k.ok = k.ok && Y != X;
    k.workspace(ws, ws_bytes, total_bytes(p, false, flags));
    if (!k.ok) return GMM_ERR_INVALID_ARG;
    ExpCall c = make_call(q, L, ws, ids);
    c.units = mlp ? p.h : INT_MAX;
    c.x = X;
    c.w1 = W1;
    c.b1 = b1;
    c.w2 = W2;
    c.b2 = b2;
    c.res = residual;
    c.resp = resp;
    c.y = Y;
    return run(c, p, L, path, false, ws, s);
}

gmm_status backward(const gmm_expert_shape *shape, bool mlp, const void *dY, const void *X,
                    const int32_t *ids, const float *resp, const void *W1, const void *b1,
                    const void *W2, const void *b2, void *dX, void *dW1, void *db1, void *dW2,
                    void *db2, float *dresp, void *ws, size_t ws_bytes, uint32_t flags,
                    cudaStream_t s) {
    if (!valid_shape(shape, mlp) || !known_flags(flags)) return GMM_ERR_INVALID_ARG;
    const ExpShape p = make_shape(shape);
    const int path = path_of(p, true, flags);
    const ExpShape q = padded(p, path) ? pad_shape(p) : p;
    const Layout L = layout_of(q, true, path);
    Checks k;
    k.elem = p.dt == GMM_F32 ? 4 : 2;
    k.big(dY, p.o);
    k.big(X, p.d);
    k.big(W1, p.d);
    k.big(dX, p.d);
    k.big(dW1, p.d);
    if (mlp) {
        k.big(W2, p.h);
        k.big(dW2, p.h);
    }
    k.small(b1, k.elem);
    k.small(b2, k.elem);
    k.small(db1, k.elem);
    k.small(db2, k.elem);
    k.small(dresp, 4);
    k.pair(b1, db1);
    k.pair(b2, db2);
    k.pair(resp, dresp);
    k.routing(shape, ids, resp);
    k.ok = k.ok && dX != X && dX != dY;
    k.workspace(ws, ws_bytes, total_bytes(p, true, flags));
    if (!k.ok) return GMM_ERR_INVALID_ARG;
    ExpCall c = make_call(q, L, ws, ids);
    c.units = mlp ? p.h : INT_MAX;
    c.dy = dY;
    c.x = X;
    c.w1 = W1;
    c.b1 = b1;
    c.w2 = W2;
    c.b2 = b2;
    c.resp = resp;
    c.dx = dX;
    c.dw1 = dW1;
    c.db1 = db1;
    c.dw2 = dW2;
    c.db2 = db2;
    c.dresp = dresp;
    return run(c, p, L, path, true, ws, s);
}

}  // namespace

extern "C" {

int gmm_expert_path(const gmm_expert_shape *shape, int backward_call, uint32_t flags) {
    if (!shape || !valid_shape(shape, shape->h > 0) || !known_flags(flags)) return -1;
    return path_of(make_shape(shape), backward_call != 0, flags);
}

size_t gmm_expert_workspace_size(const gmm_expert_shape *shape, int backward_call,
                                 uint32_t flags) {
    if (!shape || !valid_shape(shape, shape->h > 0) || !known_flags(flags)) return 0;
    const ExpShape p = make_shape(shape);
    const size_t fwd = total_bytes(p, false, flags);
    if (!backward_call) return fwd;
    const size_t bwd = total_bytes(p, true, flags);
    return bwd > fwd ? bwd : fwd;
}

gmm_status gmm_expert_linear(const gmm_expert_shape *shape, const void *X, const int32_t *ids,
                             const float *resp, const void *W, const void *b,
                             const void *residual, void *Y, void *ws, size_t ws_bytes,
                             uint32_t flags, void *stream) {
    return forward(shape, false, X, ids, resp, W, b, nullptr, nullptr, residual, Y, ws, ws_bytes,
                   flags, (cudaStream_t)stream);
}

gmm_status gmm_expert_linear_backward(const gmm_expert_shape *shape, const void *dY,
                                      const void *X, const int32_t *ids, const float *resp,
                                      const void *W, const void *b, void *dX, void *dW, void *db,
                                      float *dresp, void *ws, size_t ws_bytes, uint32_t flags,
                                      void *stream) {
    return backward(shape, false, dY, X, ids, resp, W, b, nullptr, nullptr, dX, dW, db, nullptr,
                    nullptr, dresp, ws, ws_bytes, flags, (cudaStream_t)stream);
}

gmm_status gmm_expert_mlp(const gmm_expert_shape *shape, const void *X, const int32_t *ids,
                          const float *resp, const void *W1, const void *b1, const void *W2,
                          const void *b2, const void *residual, void *Y, void *ws,
                          size_t ws_bytes, uint32_t flags, void *stream) {
    return forward(shape, true, X, ids, resp, W1, b1, W2, b2, residual, Y, ws, ws_bytes, flags,
                   (cudaStream_t)stream);
}

gmm_status gmm_expert_mlp_backward(const gmm_expert_shape *shape, const void *dY, const void *X,
                                   const int32_t *ids, const float *resp, const void *W1,
                                   const void *b1, const void *W2, const void *b2, void *dX,
                                   void *dW1, void *db1, void *dW2, void *db2, float *dresp,
                                   void *ws, size_t ws_bytes, uint32_t flags, void *stream) {
    return backward(shape, true, dY, X, ids, resp, W1, b1, W2, b2, dX, dW1, db1, dW2, db2, dresp,
                    ws, ws_bytes, flags, (cudaStream_t)stream);
}

}  // extern "C"
