"""The operators that follow soft assignment: the experts' products.

``soft_assign`` (or k-means) gives each of N points up to r components, ``ids``
[N, r] (-1: none), and their weights ``resp`` [N, r].  The operators here send
each point through the maps of its components and add the results up by
weight:

- ``linear``:  y_n = sum_i resp_ni f(W_e x_n + b_e) + residual_n, e = ids_ni
  (``r`` = 0 in a case: no ids, one dense map for all points);
- ``mlp``:     y_n = sum_i resp_ni (W2_e h + b2_e) + residual_n with
  h = f(W1_e x_n + b1_e), or gated h = f(a) * u for [a, u] = W1_e x_n + b1_e;
- ``linear_bwd``, ``mlp_bwd``: the gradients of every input, given dy.

``run`` computes them with elementary torch operations in 32 bits (``own``
false) or by the calls of this package (``own`` true).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(name, op, n, d, o, k, r, dtype, act, h=0, gated=False, bias=True, res=False, cut=0.0):
    c = dict(op=op, n=n, d=d, h=h, o=o, k=k, r=r, dtype=dtype, act=act, gated=gated, bias=bias,
             res=res, cut=cut)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one point through one dense map: a projection while serving, where latency counts
        _case("linear 1 dense", "linear", 1, 1024, 4096, 1, 0, "bf16", "gelu", res=True),
        # a batch through one dense map, with the whole epilogue: a training or prefill step
        _case("linear 4096 dense", "linear", 4096, 1024, 4096, 1, 0, "bf16", "gelu", res=True),
        # local linear models of a small fitted mixture: fp32, odd sizes, points below the cut
        _case("linear 1000 routed f32", "linear", 1000, 100, 75, 8, 2, "f32", "none", res=True,
              cut=0.2),
        # training the local maps of a mixture (d = 128 is this package's usual width)
        _case("linear bwd 16384 routed", "linear_bwd", 16384, 128, 512, 16, 2, "f16", "silu",
              cut=0.1),
        # training a dense map
        _case("linear bwd 8192 dense", "linear_bwd", 8192, 1024, 4096, 1, 0, "bf16", "gelu"),
        # one token through a mixture of experts: a serving step
        _case("mlp 1 token", "mlp", 1, 2048, 2048, 64, 8, "bf16", "silu", h=1024, gated=True,
              bias=False, res=True),
        # a small batch of serving steps, experts shared by some of the tokens
        _case("mlp 16 tokens", "mlp", 16, 1024, 1024, 64, 4, "f16", "gelu", h=2048, res=True),
        # a short ragged prompt: sizes off every tile, experts that get nothing, points cut
        _case("mlp 333 tokens ragged", "mlp", 333, 1000, 520, 32, 2, "bf16", "silu", h=616,
              gated=True, cut=0.3),
        # experts behind k-means clusters (one component a point), fp32
        _case("mlp 2048 clusters f32", "mlp", 2048, 128, 128, 8, 1, "f32", "relu", h=256),
        # a prefill or forward training step
        _case("mlp 8192 tokens", "mlp", 8192, 2048, 2048, 16, 2, "bf16", "silu", h=4096,
              gated=True, bias=False, res=True),
        # training steps of the layer: a small one with many experts, and a large one
        _case("mlp bwd 512 tokens", "mlp_bwd", 512, 512, 512, 64, 2, "f16", "gelu", h=1024,
              cut=0.2),
        _case("mlp bwd 8192 tokens", "mlp_bwd", 8192, 2048, 2048, 16, 2, "bf16", "silu", h=4096,
              gated=True, bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: from one point to 16384, widths from 64 to 4096 (most of
    them multiples of 8, some odd), 1 to 256 experts, every type and form."""
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["linear", "linear", "linear_bwd", "mlp", "mlp", "mlp", "mlp_bwd", "mlp_bwd"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f16", "f32"])
        n = _log(rng, 1, 16384 if dtype != "f32" else 4096)
        top = 4096 if dtype != "f32" else 512
        odd = rng.random() < 0.15
        d, h, o = (_log(rng, 64, top) if odd else 8 * _log(rng, 8, top // 8) for _ in range(3))
        r = rng.choice([0, 1, 2, 2, 4, 8])
        k = 1 if r == 0 else max(r, _log(rng, 2, 256))
        # relu's derivative jumps at 0, where rounding alone picks the side: forward cases only
        acts = ["none", "gelu", "silu"] + ([] if op.endswith("bwd") else ["relu"])
        c = _case(None, op, n, d, o, k, r, dtype, rng.choice(acts),
                  bias=rng.random() < 0.5, res=op in ("linear", "mlp") and rng.random() < 0.5,
                  cut=rng.choice([0.0, 0.0, 0.2]))
        if op.startswith("mlp"):
            c["h"], c["gated"] = h, rng.random() < 0.5
        w = work(c)
        # odd widths run on CUDA cores, as fp32 does: keep them to sizes such a user has
        if w["flops"] > (most if dtype != "f32" and not odd else most / 64) or w["bytes"] > 2e9:
            continue
        return c


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt, n, d, h, o, k, r = (_DT[c["dtype"]], c["n"], c["d"], c["h"], c["o"], c["k"], c["r"])

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

    s = {"case": c, "x": normal(n, d), "ids": None, "resp": None, "res": None}
    if r:
        # components of unequal weight, each point's own in order of responsibility
        w = torch.rand(k, generator=g, device=dev).square() + 0.05
        u = torch.rand(n, k, generator=g, device=dev).clamp_min(1e-9)
        s["ids"] = (u.log() / w).topk(r, dim=1).indices.to(torch.int32)
        p = torch.rand(n, r, generator=g, device=dev).add(0.05).sort(dim=1, descending=True).values
        s["resp"] = p / p.sum(1, keepdim=True)
        if c["cut"]:
            out = torch.rand(n, r, generator=g, device=dev) < c["cut"]
            s["ids"] = s["ids"].masked_fill(out, -1)
            s["resp"] = s["resp"].masked_fill(out, 0.0)
    if c["op"].startswith("linear"):
        s["w"] = normal(k, o, d, scale=d ** -0.5)
        s["b"] = normal(k, o, scale=0.5) if c["bias"] else None
    else:
        gh = 2 * h if c["gated"] else h
        s["w1"] = normal(k, gh, d, scale=d ** -0.5)
        s["b1"] = normal(k, gh, scale=0.5) if c["bias"] else None
        s["w2"] = normal(k, o, h, scale=h ** -0.5)
        s["b2"] = normal(k, o, scale=0.5) if c["bias"] else None
    if c["op"].endswith("bwd"):
        s["dy"] = normal(n, o)
    elif c["res"]:
        s["res"] = normal(n, o)
    if own:   # the workspace that a program keeps for calls of these sizes
        import means_clustering_gmm_b200 as gmm
        bwd = c["op"].endswith("bwd")
        if c["op"].startswith("linear"):
            s["ws"] = gmm.Workspace.for_expert_linear(n, d, o, k, r, dt, backward=bwd)
        else:
            s["ws"] = gmm.Workspace.for_expert_mlp(n, d, h, o, k, r, dt, gated=c["gated"],
                                                   backward=bwd)
    return s


# ------------------------------------------------------------ plain form
def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (
            2 * math.pi) ** -0.5
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


class _Groups:
    """The (point, slot) pairs sorted by component, each component's pairs in
    the rows of one [used, most, width] block."""

    def __init__(self, s):
        c, x = s["case"], s["x"]
        self.n, self.k, self.r = c["n"], c["k"], max(1, c["r"])
        ids = s["ids"]
        if ids is None:
            ids = torch.zeros(self.n, 1, dtype=torch.int32, device=x.device)
        flat = ids.reshape(-1).long()
        pair = (flat >= 0).nonzero().reshape(-1)
        e, order = flat[pair].sort(stable=True)
        self.pair = pair[order]
        self.tok = self.pair // self.r
        count = torch.bincount(e, minlength=self.k)
        self.used = (count > 0).nonzero().reshape(-1)
        place = torch.cumsum(count > 0, 0) - 1
        self.u = place[e]
        self.pos = torch.arange(e.numel(), device=x.device) - (torch.cumsum(count, 0) - count)[e]
        self.most = int(count.max())
        g = s["resp"]
        self.g = (torch.ones(self.n * self.r, device=x.device) if g is None else g.reshape(-1))[
            self.pair, None]

    def block(self, rows):
        """[used, most, width] from one row for each pair, zeros past them."""
        b = torch.zeros(self.used.numel(), self.most, rows.shape[1], device=rows.device)
        b[self.u, self.pos] = rows
        return b

    def rows(self, block):
        return block[self.u, self.pos]

    def per_point(self, rows):
        """Each point's sum over its pairs."""
        s = torch.zeros(self.n * self.r, rows.shape[1], device=rows.device)
        s[self.pair] = rows
        return s.view(self.n, self.r, -1).sum(1)

    def per_pair(self, values):
        s = torch.zeros(self.n * self.r, device=values.device)
        s[self.pair] = values
        return s.view(self.n, self.r)

    def all_experts(self, t, like):
        full = torch.zeros(like.shape, device=t.device)
        full[self.used] = t
        return full.to(like.dtype)

    def map(self, block, w, b):
        y = torch.bmm(block, w[self.used].float().transpose(1, 2))
        return y if b is None else y + b[self.used].float()[:, None]


def _plain_linear(s, G):
    c = s["case"]
    z = G.map(G.block(s["x"].float()[G.tok]), s["w"], s["b"])
    y = G.per_point(G.rows(_act(z, c["act"])) * G.g)
    return (y if s["res"] is None else y + s["res"].float()).to(s["x"].dtype)


def _plain_linear_bwd(s, G):
    c = s["case"]
    x = G.block(s["x"].float()[G.tok])
    dy = G.block(s["dy"].float()[G.tok])
    z = G.map(x, s["w"], s["b"])
    dz = dy * G.block(G.g) * _dact(z, c["act"])
    out = {"dx": G.per_point(G.rows(torch.bmm(dz, s["w"][G.used].float()))).to(s["x"].dtype),
           "dw": G.all_experts(torch.bmm(dz.transpose(1, 2), x), s["w"])}
    if s["b"] is not None:
        out["db"] = G.all_experts(dz.sum(1), s["b"])
    if s["resp"] is not None:
        out["dresp"] = G.per_pair(G.rows(dy * _act(z, c["act"])).sum(1))
    return out


def _hidden(s, G, x):
    c = s["case"]
    z = G.map(x, s["w1"], s["b1"])
    if not c["gated"]:
        return z, None, _act(z, c["act"])
    a, u = z.chunk(2, dim=2)
    return a, u, _act(a, c["act"]) * u


def _plain_mlp(s, G):
    _, _, h = _hidden(s, G, G.block(s["x"].float()[G.tok]))
    y = G.per_point(G.rows(G.map(h, s["w2"], s["b2"])) * G.g)
    return (y if s["res"] is None else y + s["res"].float()).to(s["x"].dtype)


def _plain_mlp_bwd(s, G):
    c = s["case"]
    x = G.block(s["x"].float()[G.tok])
    dy = G.block(s["dy"].float()[G.tok])
    g = G.block(G.g)
    a, u, h = _hidden(s, G, x)
    q = torch.bmm(dy, s["w2"][G.used].float())
    dresp = (q * h).sum(2)
    if s["b2"] is not None:
        dresp = dresp + (dy * s["b2"][G.used].float()[:, None]).sum(2)
    dh = q * g
    if c["gated"]:
        da = torch.cat([dh * u * _dact(a, c["act"]), dh * _act(a, c["act"])], 2)
    else:
        da = dh * _dact(a, c["act"])
    out = {"dx": G.per_point(G.rows(torch.bmm(da, s["w1"][G.used].float()))).to(s["x"].dtype),
           "dw1": G.all_experts(torch.bmm(da.transpose(1, 2), x), s["w1"]),
           "dw2": G.all_experts(torch.bmm((dy * g).transpose(1, 2), h), s["w2"])}
    if s["b1"] is not None:
        out["db1"] = G.all_experts(da.sum(1), s["b1"])
        out["db2"] = G.all_experts((dy * g).sum(1), s["b2"])
    if s["resp"] is not None:
        out["dresp"] = G.per_pair(G.rows(dresp[..., None])[:, 0])
    return out


_PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "mlp": _plain_mlp,
          "mlp_bwd": _plain_mlp_bwd}


def run(state):
    s, c = state, state["case"]
    if not own:
        return _PLAIN[c["op"]](s, _Groups(s))
    import means_clustering_gmm_b200 as gmm
    if c["op"] == "linear":
        return gmm.expert_linear(s["x"], s["ids"], s["resp"], s["w"], s["b"], s["ws"],
                                 activation=c["act"], residual=s["res"])
    if c["op"] == "mlp":
        return gmm.expert_mlp(s["x"], s["ids"], s["resp"], s["w1"], s["b1"], s["w2"], s["b2"],
                              s["ws"], activation=c["act"], gated=c["gated"], residual=s["res"])
    if c["op"] == "linear_bwd":
        names = ("dx", "dw", "db", "dresp")
        got = gmm.expert_linear_backward(s["dy"], s["x"], s["ids"], s["resp"], s["w"], s["b"],
                                         s["ws"], activation=c["act"])
    else:
        names = ("dx", "dw1", "db1", "dw2", "db2", "dresp")
        got = gmm.expert_mlp_backward(s["dy"], s["x"], s["ids"], s["resp"], s["w1"], s["b1"],
                                      s["w2"], s["b2"], s["ws"], activation=c["act"],
                                      gated=c["gated"])
    return {k: v for k, v in zip(names, got) if v is not None}


def work(case):
    """Every input read once (the weights of the experts in use), every output
    written once; the products that each direction cannot do without."""
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    n, d, h, o, k, r = c["n"], c["d"], c["h"], c["o"], c["k"], max(1, c["r"])
    pairs = max(1.0, n * r * (1 - c["cut"]))
    e = k * (1 - (1 - min(1.0, r / k)) ** (pairs / r))
    bwd = c["op"].endswith("bwd")
    if c["op"].startswith("linear"):
        per, recompute = o * d, o * d if c["act"] != "none" or c["r"] else 0
    else:
        gd = (2 if c["gated"] else 1) * d
        per, recompute = h * (gd + o), h * gd
    flops = 2 * pairs * (2 * per + recompute if bwd else per)
    rows = n * (2 * d + o) if bwd else n * (d + o * (2 if c["res"] else 1))
    weights = e * per + (k * per if bwd else 0)
    return {"bytes": float(size * (rows + weights) + 8 * n * c["r"]), "flops": float(flops)}


# -------------------------------------------------------- the definition
def exact(case, seed):
    """The definition in 64 bits, one component after the other."""
    c, s = case, prepare(case, seed)
    x = s["x"].double()
    n, r, k, dev = c["n"], max(1, c["r"]), c["k"], x.device
    ids = torch.zeros(n, 1, dtype=torch.long, device=dev) if s["ids"] is None else s["ids"].long()
    wt = torch.ones(n, r, dtype=torch.float64, device=dev) if s["resp"] is None else s[
        "resp"].double()
    bwd, mlp = c["op"].endswith("bwd"), c["op"].startswith("mlp")
    dy = s["dy"].double() if bwd else None
    sig, root = torch.sigmoid, math.sqrt(2.0)

    def f(z):
        return {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0 * z),
                "gelu": lambda: z * 0.5 * torch.erfc(-z / root), "silu": lambda: z * sig(z)}[
                    c["act"]]()

    def df(z):
        if c["act"] == "gelu":
            return 0.5 * torch.erfc(-z / root) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if c["act"] == "silu":
            return sig(z) + z * sig(z) * sig(-z)
        return torch.ones_like(z) if c["act"] == "none" else torch.where(z > 0, 1.0, 0.0).to(z)

    names = [m for m in ("w", "b", "w1", "b1", "w2", "b2") if s.get(m) is not None]
    grads = {m: torch.zeros(s[m].shape, dtype=torch.float64, device=dev) for m in names} if bwd else {}
    out = torch.zeros(n, c["d"] if bwd else c["o"], dtype=torch.float64, device=dev)
    dresp = torch.zeros(n, r, dtype=torch.float64, device=dev)
    for e in range(k):
        at, slot = torch.where(ids == e)
        if at.numel() == 0:
            continue
        xe, we = x[at], wt[at, slot][:, None]
        p = {m: s[m][e].double() for m in names}
        z = xe @ p["w1" if mlp else "w"].T
        first = "b1" if mlp else "b"
        if first in p:
            z = z + p[first]
        if mlp:
            a, u = (z[:, :c["h"]], z[:, c["h"]:]) if c["gated"] else (z, torch.ones_like(z))
            hid = f(a) * u
            y = hid @ p["w2"].T + (p["b2"] if "b2" in p else 0)
        else:
            y = f(z)
        if not bwd:
            out.index_add_(0, at, we * y)
            continue
        de = dy[at]
        dresp[at, slot] = (de * y).sum(1)
        if mlp:
            grads["w2"][e] = (we * de).T @ hid
            if "b2" in p:
                grads["b2"][e] = (we * de).sum(0)
            back = (we * de) @ p["w2"]
            dz = back * u * df(a)
            if c["gated"]:
                dz = torch.cat([dz, back * f(a)], 1)
            grads["w1"][e] = dz.T @ xe
            if "b1" in p:
                grads["b1"][e] = dz.sum(0)
            out.index_add_(0, at, dz @ p["w1"])
        else:
            dz = we * de * df(z)
            grads["w"][e] = dz.T @ xe
            if "b" in p:
                grads["b"][e] = dz.sum(0)
            out.index_add_(0, at, dz @ p["w"])
    if not bwd:
        return out if s["res"] is None else out + s["res"].double()
    got = {"dx": out, **{"d" + m: v for m, v in grads.items()}}
    if s["resp"] is not None:
        got["dresp"] = dresp
    return got
