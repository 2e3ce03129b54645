"""The experts' products (expert_linear, expert_mlp and their gradients)
against the formulas in float64, element by element.

Every tolerance is a bound carried along with the reference: sums of n fp32
products are off by at most gamma(n) = 2 (n + 8) 2^-24 of the sum of absolute
values (the factor 2 covers accumulators that truncate), a rounding to the
16-bit type by its half step, the activations by 2^-19 of their arguments'
scale, and each error passes on through the absolute values of what it is
multiplied by (|f'| <= 1.13, |f''| <= 0.8 for all four activations).
"""
import math

import pytest
import torch

import means_clustering_gmm_b200 as gmm

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIMT = gmm.GMM_FLAG_FORCE_SIMT


def gamma(n):
    return 2.0 * (n + 8) * 2.0 ** -24


def half_step(dt):
    return torch.finfo(dt).eps / 2


def act(z, name):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * torch.erfc(-z / math.sqrt(2))}[name]()


def dact(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    return torch.ones_like(z)


def inputs(seed, N, d, h, o, K, r, dtype, gated=False, bias=True, res=False, cut=0.0, resp=True,
           use=None):
    """Seeded arrays on the CPU; `use`: the experts that ids name."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    n = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dt)  # noqa: E731
    first = (2 * h if gated else h) if h else o
    s = {"x": n(N, d), "w1": n(K, first, d, scale=d ** -0.5), "w2": None, "b2": None,
         "b1": n(K, first, scale=0.5) if bias else None, "dy": n(N, o),
         "res": n(N, o) if res else None, "ids": None, "resp": None}
    if h:
        s["w2"] = n(K, o, h, scale=h ** -0.5)
        s["b2"] = n(K, o, scale=0.5) if bias else None
    if r:
        pool = torch.tensor(use if use is not None else range(K))
        s["ids"] = pool[torch.randint(len(pool), (N, r), generator=g)].to(torch.int32)
        s["ids"][torch.rand(N, r, generator=g) < cut] = -1
        if resp:
            s["resp"] = torch.rand(N, r, generator=g) + 0.05
    return s


def reference(s, activation, gated, dt):
    """Results in float64 and, under the same names, bounds of their error."""
    x, dy = s["x"].double(), s["dy"].double()
    N, d = x.shape
    K, first = s["w1"].shape[:2]
    mlp = s["w2"] is not None
    o = s["w2"].shape[1] if mlp else first
    h = first // 2 if gated else first
    r = s["ids"].shape[1] if s["ids"] is not None else 1
    ids = s["ids"] if s["ids"] is not None else torch.zeros(N, 1, dtype=torch.int32)
    wt = s["resp"].double() if s["resp"] is not None else torch.ones(N, r, dtype=torch.float64)
    u16 = half_step(dt) if dt != torch.float32 else 0.0
    z64 = lambda *sh: torch.zeros(*sh, dtype=torch.float64)  # noqa: E731
    v = {"y": z64(N, o), "dx": z64(N, d), "dw1": z64(*s["w1"].shape), "dresp": z64(N, r)}
    if s["b1"] is not None:
        v["db1"] = z64(K, first)
    if mlp:
        v["dw2"] = z64(*s["w2"].shape)
        if s["b2"] is not None:
            v["db2"] = z64(K, o)
    b = {k: torch.zeros_like(t) for k, t in v.items()}
    F = 2.0 ** -19
    for e in range(K):
        n, i = torch.where(ids == e)
        if n.numel() == 0:
            continue
        T = n.numel()
        xe, de, g = x[n], dy[n], wt[n, i][:, None]
        w1 = s["w1"][e].double()
        b1 = s["b1"][e].double() if s["b1"] is not None else z64(first)
        z = xe @ w1.T + b1
        ez = gamma(d) * (xe.abs() @ w1.abs().T + b1.abs())
        a, u = (z[:, :h], z[:, h:]) if gated else (z, torch.ones_like(z))
        ea, eu = (ez[:, :h], ez[:, h:]) if gated else (ez, torch.zeros_like(ez))
        f, df = act(a, activation), dact(a, activation)
        ef = 1.13 * ea + F * (a.abs() + f.abs())
        edf = 0.8 * ea + F * (1 + a.abs())
        if activation in ("none", "relu"):
            edf = torch.zeros_like(ea)   # relu: the inputs keep z away from 0
        hid = f * u
        eh = ef * u.abs() + f.abs() * eu + ef * eu
        if mlp:
            w2 = s["w2"][e].double()
            b2 = s["b2"][e].double() if s["b2"] is not None else z64(o)
            out = hid @ w2.T + b2
            eo = (eh + u16 * (hid.abs() + eh)) @ w2.abs().T + gamma(h) * (
                hid.abs() @ w2.abs().T + b2.abs())
            q = de @ w2
            eq = gamma(o) * (de.abs() @ w2.abs())
        else:
            out, eo, q, eq = f, ef, de, torch.zeros_like(de)
        v["y"].index_add_(0, n, g * out)
        b["y"].index_add_(0, n, g * eo + gamma(r) * g * out.abs())
        v["dresp"][n, i] = (de * out).sum(1)
        b["dresp"][n, i] = (
            (q.abs() * eh + eq * (hid.abs() + eh)).sum(1) + gamma(h + o) * (
                (q.abs() * hid.abs()).sum(1) + (de.abs() * (b2.abs() if mlp else 0)).sum(1)))
        # the pre-activations' gradient, rounded to the type
        def grad(*factors):
            val = g * math.prod(t for t, _ in factors)
            up = g * math.prod(t.abs() + et for t, et in factors)
            err = up - val.abs() + gamma(4) * up
            return val, err + u16 * (val.abs() + err) + tiny(dt)
        if gated:
            ga, ega = grad((q, eq), (u, eu), (df, edf))
            gu, egu = grad((q, eq), (f, ef))
            da, eda = torch.cat([ga, gu], 1), torch.cat([ega, egu], 1)
        else:
            da, eda = grad((q, eq), (df, edf))
        if s["b1"] is not None:
            v["db1"][e] = da.sum(0)
            b["db1"][e] = eda.sum(0) + gamma(T) * da.abs().sum(0)
        v["dw1"][e] = da.T @ xe
        b["dw1"][e] = eda.T @ xe.abs() + gamma(T) * (da.abs().T @ xe.abs())
        v["dx"].index_add_(0, n, da @ w1)
        b["dx"].index_add_(0, n, eda @ w1.abs() + gamma(first + r) * (da.abs() @ w1.abs()))
        if mlp:
            hs, ehs = grad((hid, eh))
            v["dw2"][e] = de.T @ hs
            b["dw2"][e] = de.abs().T @ ehs + gamma(T) * (de.abs().T @ hs.abs())
            if s["b2"] is not None:
                v["db2"][e] = (g * de).sum(0)
                b["db2"][e] = gamma(T) * (g * de).abs().sum(0)
    if s["res"] is not None:
        v["y"] += s["res"].double()
        b["y"] += gamma(2) * (v["y"].abs() + s["res"].double().abs())
    for k in v:   # the rounding of the result
        u = half_step(torch.float32 if k == "dresp" else dt)
        b[k] += u * (v[k].abs() + b[k]) + tiny(torch.float32 if k == "dresp" else dt)
    return v, b


def tiny(dt):
    """Half the step of the type's subnormals."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def cuda(s):
    return {k: t.cuda() if isinstance(t, torch.Tensor) else t for k, t in s.items()}


def workspace(s, gated, backward, flags=0):
    N, d = s["x"].shape
    K, first = s["w1"].shape[:2]
    r = 0 if s["ids"] is None else s["ids"].shape[1]
    if s["w2"] is None:
        return gmm.Workspace.for_expert_linear(N, d, first, K, r, s["x"].dtype, backward=backward,
                                               flags=flags)
    return gmm.Workspace.for_expert_mlp(N, d, first // 2 if gated else first, s["w2"].shape[1], K,
                                        r, s["x"].dtype, gated=gated, backward=backward,
                                        flags=flags)


def forward(c, activation, gated=False, flags=0, ws=None, **kw):
    ws = ws or workspace(c, gated, False, flags)
    if c["w2"] is None:
        y = gmm.expert_linear(c["x"], c["ids"], c["resp"], c["w1"], c["b1"], ws,
                              activation=activation, residual=c["res"], flags=flags, **kw)
    else:
        y = gmm.expert_mlp(c["x"], c["ids"], c["resp"], c["w1"], c["b1"], c["w2"], c["b2"], ws,
                           activation=activation, gated=gated, residual=c["res"], flags=flags,
                           **kw)
    return y, ws


def backward(c, activation, gated=False, flags=0, ws=None, **kw):
    ws = ws or workspace(c, gated, True, flags)
    if c["w2"] is None:
        got = gmm.expert_linear_backward(c["dy"], c["x"], c["ids"], c["resp"], c["w1"], c["b1"],
                                         ws, activation=activation, flags=flags, **kw)
        names = ("dx", "dw1", "db1", "dresp")
    else:
        got = gmm.expert_mlp_backward(c["dy"], c["x"], c["ids"], c["resp"], c["w1"], c["b1"],
                                      c["w2"], c["b2"], ws, activation=activation, gated=gated,
                                      flags=flags, **kw)
        names = ("dx", "dw1", "db1", "dw2", "db2", "dresp")
    return {k: t for k, t in zip(names, got) if t is not None}, ws


def within(got, v, b, label):
    for k, t in got.items():
        err = (t.double().cpu() - v[k]).abs()
        bad = ~(err <= b[k])
        worst = (err / b[k].clamp_min(1e-300)).max()
        assert not bad.any(), (label, k, int(bad.sum()), float(worst),
                               [int(x) for x in bad.nonzero()[0]])


def check(s, activation, gated=False, flags=0, back=True):
    dt = s["x"].dtype
    v, b = reference(s, activation, gated, dt)
    c = cuda(s)
    y, ws = forward(c, activation, gated, flags)
    assert gmm.gmm_last_error(ws) == 0
    within({"y": y}, v, b, "forward")
    if back:
        got, ws = backward(c, activation, gated, flags)
        assert gmm.gmm_last_error(ws) == 0
        if s["resp"] is None:
            assert "dresp" not in got
        within(got, v, b, "backward")


LINEAR = [
    # N, d, o, K, r, dtype, activation, options
    (1, 1, 1, 1, 0, "f32", "none", {}),
    (1, 64, 8, 1, 0, "bf16", "gelu", {"res": True}),
    (3, 17, 5, 2, 1, "f32", "silu", {"resp": False}),
    (130, 40, 72, 5, 3, "bf16", "silu", {"cut": 0.3, "res": True}),
    (257, 128, 264, 4, 2, "f16", "gelu", {"cut": 0.2}),
    (300, 64, 64, 7, 1, "bf16", "none", {"cut": 0.4, "res": True}),       # points without any
    (300, 64, 64, 7, 1, "f16", "none", {"resp": False, "bias": False}),
    (200, 33, 65, 6, 2, "bf16", "gelu", {"cut": 0.2}),                    # odd widths
    (129, 72, 136, 1, 0, "f16", "silu", {"res": True}),
    (520, 256, 512, 1, 0, "bf16", "none", {"bias": False}),
    (300, 128, 128, 64, 8, "bf16", "gelu", {}),                           # short segments
    (700, 64, 40, 300, 2, "f16", "silu", {"use": [0, 299, 17]}),          # unused experts
    (1000, 72, 264, 2, 2, "bf16", "silu", {"cut": 0.1, "res": True}),     # pairs of row tiles
    (900, 136, 600, 2, 1, "f16", "none", {"cut": 0.3}),
    (385, 64, 64, 1, 0, "bf16", "gelu", {"res": True}),
    (5000, 16, 8, 3, 8, "bf16", "none", {"cut": 0.5}),                    # 40000 pairs
    (600, 16, 8, 2000, 2, "f16", "none", {"cut": 0.1}),                   # many experts
    (9000, 16, 8, 400, 1, "bf16", "silu", {"cut": 0.1}),
    (9000, 8, 8, 1, 4, "bf16", "silu", {"cut": 0.1}),                     # one, many times
    (700, 72, 136, 3, 2, "bf16", "none", {"cut": 0.2, "resp": False}),    # dz is dY itself
    (300, 72, 136, 1, 0, "f16", "none", {}),
    (300, 71, 135, 1, 0, "f16", "none", {}),
    (64, 136, 72, 1, 0, "bf16", "gelu", {"res": True}),
    (2, 1032, 4000, 1, 0, "f16", "silu", {"res": True}),
    (64, 200, 40, 3, 4, "bf16", "silu", {"cut": 0.3, "res": True}),
    (50, 64, 40, 3, 1, "bf16", "gelu", {"cut": 0.4, "res": True}),
]


@pytest.mark.parametrize("N,d,o,K,r,dtype,activation,opt", LINEAR)
@pytest.mark.parametrize("flags", [0, SIMT])
def test_linear(N, d, o, K, r, dtype, activation, opt, flags):
    check(inputs(N + d + o, N, d, 0, o, K, r, dtype, **opt), activation, flags=flags)


MLP = [
    # N, d, h, o, K, r, dtype, activation, gated, options
    (1, 1, 1, 1, 1, 0, "f32", "silu", False, {}),
    (1, 64, 64, 64, 8, 2, "bf16", "silu", True, {"res": True}),
    (5, 72, 40, 24, 3, 2, "f16", "gelu", False, {"cut": 0.3}),
    (1, 4096, 2048, 136, 9, 8, "bf16", "silu", True, {}),
    (16, 128, 64, 136, 64, 4, "bf16", "silu", True, {"bias": False, "res": True}),
    (31, 264, 104, 128, 5, 8, "f16", "none", True, {}),
    (33, 31, 29, 27, 3, 2, "bf16", "silu", True, {"cut": 0.2}),           # odd widths
    (130, 64, 200, 72, 4, 2, "bf16", "gelu", False, {"cut": 0.3, "res": True}),
    (300, 136, 72, 264, 5, 1, "f16", "silu", True, {"cut": 0.3, "res": True}),
    (257, 64, 128, 64, 1, 0, "bf16", "silu", True, {"res": True}),
    (400, 128, 320, 128, 16, 2, "bf16", "silu", True, {}),
    (300, 64, 64, 64, 64, 8, "f16", "gelu", False, {"bias": False}),
    (150, 50, 60, 70, 6, 3, "f32", "gelu", True, {"cut": 0.2}),
    (150, 50, 60, 70, 6, 3, "bf16", "gelu", True, {"cut": 0.2, "res": True}),   # padded copies:
    (700, 64, 61, 64, 2, 2, "f16", "silu", True, {}),                           # h alone
    (90, 63, 64, 64, 40, 1, "bf16", "silu", False, {"resp": False}),            # d alone
    (200, 8, 16, 9, 1, 0, "f16", "gelu", False, {"res": True}),                 # o alone, dense
    (1, 7, 5, 3, 4, 2, "bf16", "silu", True, {"bias": False}),
    (600, 64, 72, 64, 200, 2, "bf16", "none", False, {"use": [3, 198, 199], "resp": False}),
    (1000, 72, 136, 200, 2, 2, "bf16", "silu", True, {"cut": 0.1, "res": True}),   # pairs of tiles
    (700, 200, 264, 72, 2, 2, "f16", "gelu", False, {}),
    (641, 64, 320, 64, 1, 0, "bf16", "silu", True, {"bias": False}),
    (32, 520, 136, 40, 40, 8, "bf16", "silu", True, {"cut": 0.2, "res": True}),     # 256 pairs
    (64, 64, 1032, 24, 2, 4, "f16", "gelu", False, {"res": True}),                  # 128 a expert
    (64, 72, 40, 1000, 300, 4, "bf16", "silu", False, {"resp": False}),
    (64, 64, 64, 64, 1, 0, "f16", "silu", True, {"res": True}),
]


@pytest.mark.parametrize("N,d,h,o,K,r,dtype,activation,gated,opt", MLP)
@pytest.mark.parametrize("flags", [0, SIMT])
def test_mlp(N, d, h, o, K, r, dtype, activation, gated, opt, flags):
    check(inputs(N + d + h, N, d, h, o, K, r, dtype, gated=gated, **opt), activation, gated, flags)


@pytest.mark.parametrize("N,d,h,o,K,r,gated,opt", [
    (1700, 64, 0, 1160, 1, 0, False, {"res": True}),          # 8 rows a thread, 14 x 19 tiles
    (1650, 36, 40, 560, 3, 2, True, {"cut": 0.1}),            # 26 x 9, segments of unequal length
    (1650, 560, 0, 24, 4, 2, False, {"cut": 0.4, "res": True}),   # the points' gradient
    (1700, 563, 0, 21, 1, 0, False, {}),                      # odd widths
    (90, 40, 72, 24, 7, 2, True, {"cut": 0.3, "res": True}),  # 2 rows a thread
])
def test_fp32_rows_a_thread(N, d, h, o, K, r, gated, opt):
    use = [0, 0, 0, 1, 2, 2, K - 1] if K > 2 else None        # lengths differ
    check(inputs(21, N, d, h, o, K, r, "f32", gated, use=use, **opt), "silu", gated)


@pytest.mark.parametrize("N,d,h,o,K,r,gated,opt", [
    (1, 1024, 0, 520, 1, 0, False, {"res": True}),
    (8, 36, 20, 12, 1, 0, True, {}),                          # two groups of four rows
    (1, 64, 136, 72, 12, 8, True, {"res": True}),
    (40, 64, 40, 24, 11, 2, False, {"cut": 0.5, "res": True}),    # points without any
    (30, 64, 0, 24, 5, 1, False, {"cut": 0.5, "resp": False}),
    (29, 33, 21, 65, 9, 2, True, {"cut": 0.2}),               # odd widths
    (150, 40, 24, 16, 40, 2, False, {"use": [0, 0, 0, 39]}),  # one expert has most of the rows
])
def test_fp32_few_rows(N, d, h, o, K, r, gated, opt):
    check(inputs(22, N, d, h, o, K, r, "f32", gated, **opt), "gelu", gated)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gated", [False, True])
def test_relu_with_whole_numbers(dtype, gated):
    """Small whole numbers with biases of a half: no pre-activation is near 0,
    and every product up to the hidden layer is exact."""
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randint(-2, 3, s, generator=g).to(DT[dtype])  # noqa: E731
    N, d, h, o, K, r = 140, 24, 40, 16, 3, 2
    first = 2 * h if gated else h
    s = {"x": n(N, d), "w1": n(K, first, d), "b1": n(K, first) + 0.5, "w2": n(K, o, h),
         "b2": n(K, o), "dy": n(N, o), "res": None,
         "ids": torch.randint(K, (N, r), generator=g).to(torch.int32),
         "resp": torch.rand(N, r, generator=g)}
    for flags in (0, SIMT):
        check(s, "relu", gated, flags)


@pytest.mark.parametrize("mlp", [False, True])
@pytest.mark.parametrize("r", [1, 2])
def test_no_point_has_an_expert(mlp, r):
    s = inputs(1, 40, 64, 64 if mlp else 0, 64, 3, r, "bf16", res=True, cut=2.0)
    assert bool((s["ids"] < 0).all())
    c = cuda(s)
    y, ws = forward(c, "silu")
    assert gmm.gmm_last_error(ws) == 0 and torch.equal(y, c["res"])
    y, ws = forward(dict(c, res=None), "silu")
    assert not y.any()
    got, ws = backward(c, "silu")
    assert gmm.gmm_last_error(ws) == 0
    for k, t in got.items():
        assert not t.any(), k


@pytest.mark.parametrize("flags", [0, SIMT])
@pytest.mark.parametrize("N", [9, 300])
def test_bad_ids_are_skipped_and_reported(flags, N):
    """An id at or above K is skipped like -1 and recorded."""
    s = inputs(3, N, 64, 64, 64, 4, 2, "bf16")
    bad = dict(s, ids=s["ids"].clone())
    bad["ids"][5, 1] = 4
    bad["ids"][8, 0] = 2 ** 31 - 1
    skip = dict(s, ids=torch.where(bad["ids"] >= 4, -1, bad["ids"]))
    for call in (lambda c: forward(c, "gelu", flags=flags),
                 lambda c: backward(c, "gelu", flags=flags)):
        got, ws = call(cuda(bad))
        assert gmm.gmm_last_error(ws) == 6 and gmm.gmm_last_error(ws) == 0
        want, ws = call(cuda(skip))
        assert gmm.gmm_last_error(ws) == 0
        for a, b in zip(*((t.values() if isinstance(t, dict) else [t]) for t in (got, want))):
            assert torch.equal(a, b)


@pytest.mark.parametrize("flags", [0, SIMT])
@pytest.mark.parametrize("N", [12, 260])
def test_nan_stays_with_its_point(flags, N):
    """A point of NaNs spoils its own results and its experts' gradients only;
    one without an expert spoils nothing, and weights that no point uses are
    not read into any result."""
    s = inputs(4, N, 64, 64, 64, 6, 2, "bf16", use=[0, 1, 2, 3])
    s["w1"][5] = float("nan")
    s["w2"][5] = float("inf")
    clean = forward(cuda(s), "silu", flags=flags)[0]
    clean_g = backward(cuda(s), "silu", flags=flags)[0]
    assert clean.isfinite().all() and all(t.isfinite().all() for t in clean_g.values())
    s["ids"][3] = -1
    s["resp"][3] = float("nan")
    for k in ("x", "dy"):
        s[k][3] = float("nan")
    s["x"][7] = float("nan")
    s["ids"][7] = torch.tensor([2, -1])
    y = forward(cuda(s), "silu", flags=flags)[0]
    g = backward(cuda(s), "silu", flags=flags)[0]
    keep = [n for n in range(N) if n not in (3, 7)]
    assert torch.equal(y[keep], clean[keep]) and y[7].isnan().all() and not y[3].any()
    assert torch.equal(g["dx"][keep], clean_g["dx"][keep]) and not g["dx"][3].any()
    for k in ("dw1", "dw2", "db1", "db2"):
        assert g[k][[0, 1, 3, 4, 5]].isfinite().all(), k
    assert g["dw1"][2].isnan().any()


@pytest.mark.parametrize("N", [3, 40, 700])
@pytest.mark.parametrize("h", [0, 72])
def test_element_aligned_biases_and_residual(N, h):
    """Biases and the residual may start at any element; everything else at
    any 16 bytes (not more)."""
    s = inputs(31, N, 64, h, 72, 2, 2 if h else 1, "bf16", res=True)
    want = forward(cuda(s), "gelu")[0], backward(cuda(s), "gelu")[0]
    c = {}
    for k, t in s.items():
        off = {"b1": 1, "b2": 3, "res": 5}.get(k, 8)
        if t is None or k in ("ids", "resp"):
            c[k] = None if t is None else t.cuda()
            continue
        room = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
        c[k] = room[off:].view(t.shape).copy_(t)
    assert torch.equal(forward(c, "gelu")[0], want[0])
    got = backward(c, "gelu")[0]
    assert all(torch.equal(got[k], want[1][k]) for k in got)
    out = torch.empty(N * 72 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(N, 72)
    assert torch.equal(forward(c, "gelu", out=out)[0], want[0])


@pytest.mark.parametrize("K,r,N", [(40, 2, 1), (40, 2, 300)])
def test_weights_past_32_bits(K, r, N):
    """The last expert's weights lie past 2^32 elements."""
    d, o = 4096, 32768
    s = inputs(32, N, d, 0, 8, 1, r, "bf16", bias=False)
    w = torch.zeros(K, o, d, dtype=torch.bfloat16, device="cuda")
    cols = 264
    rows = (torch.randn(cols, d, generator=torch.Generator().manual_seed(3)) / 64).bfloat16()
    w[K - 1, o - cols:] = rows.cuda()
    assert w.numel() > 2 ** 32
    s["ids"] = torch.full((N, r), K - 1, dtype=torch.int32)
    s["ids"][:, 1] = -1
    c = cuda(s)
    ws = gmm.Workspace.for_expert_linear(N, d, o, K, r, torch.bfloat16)
    y = gmm.expert_linear(c["x"], c["ids"], c["resp"], w, None, ws)
    assert gmm.gmm_last_error(ws) == 0
    assert not y[:, :o - cols].any()
    x = s["x"].double()
    g = s["resp"][:, :1].double()
    v = g * (x @ rows.double().T)
    b = gamma(d) * g * (x.abs() @ rows.double().abs().T)
    b += half_step(torch.bfloat16) * (v.abs() + b)
    assert ((y[:, o - cols:].cpu().double() - v).abs() <= b).all()


def test_points_past_32_bits():
    """Rows of X and Y past 2^32 elements, dense and routed."""
    N, d, o = (1 << 25) + 300, 128, 8
    x = torch.zeros(N, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(512, d, generator=torch.Generator().manual_seed(4)).bfloat16()
    x[N - 512:] = tail.cuda()
    w = torch.randn(2, o, d, generator=torch.Generator().manual_seed(5)).bfloat16()
    for r in (0, 1):
        k = 2 if r else 1
        ids = None
        if r:
            ids = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
            ids[N - 512::2] = 1
        ws = gmm.Workspace.for_expert_linear(N, d, o, k, r, torch.bfloat16)
        y = gmm.expert_linear(x, ids, None, w[:k].contiguous().cuda(), None, ws)
        assert gmm.gmm_last_error(ws) == 0 and not y[:N - 512].any()
        e = torch.zeros(512, dtype=torch.long)
        if r:
            e[::2] = 1
        t = tail.double()
        v = torch.einsum("nd,nod->no", t, w.double()[e])
        b = gamma(d) * torch.einsum("nd,nod->no", t.abs(), w.double()[e].abs())
        b += half_step(torch.bfloat16) * (v.abs() + b)
        assert ((y[N - 512:].cpu().double() - v).abs() <= b).all()
        del ws, y


def test_capture_of_a_first_call():
    """Sizes whose kernels may not have run yet, captured at once."""
    c = cuda(inputs(33, 70, 72, 88, 40, 3, 2, "f16", gated=True, bias=False))
    ws = workspace(c, True, True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = forward(c, "none", True, ws=ws)
        g, _ = backward(c, "none", True, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, forward(c, "none", True)[0])
    want = backward(c, "none", True)[0]
    assert all(torch.equal(g[k], want[k]) for k in want)


@pytest.mark.parametrize("N", [1, 50, 200])
def test_same_expert_twice(N):
    """Two entries that name one expert add up."""
    s = inputs(8, N, 64, 72, 64, 3, 4, "bf16", res=True)
    s["ids"][:, 1] = s["ids"][:, 0]
    s["ids"][::2, 3] = s["ids"][::2, 0]
    check(s, "silu")


@pytest.mark.parametrize("h", [0, 72])
def test_result_may_replace_the_residual(h):
    for r, N, o in ((2, 300, 64), (0, 300, 64), (1, 300, 64), (2, 4, 64), (0, 1, 64),
                    (0, 3000, 520), (1, 9000, 328)):
        s = inputs(9, N, 64, h, o, 3 if r else 1, r, "bf16", res=True)
        c = cuda(s)
        want = forward(c, "silu")[0]
        got = forward(c, "silu", out=c["res"])[0]
        assert got.data_ptr() == c["res"].data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("r,activation", [(0, "gelu"), (1, "silu")])
def test_many_tiles_a_block(r, activation):
    """More tiles than blocks, the last column tile narrower than the others:
    rows and residuals that are loaded a tile ahead meet their own tile."""
    s = inputs(21, 12000, 64, 0, 600, 4 if r else 1, r, "f16", res=True, cut=0.2 if r else 0.0)
    check(s, activation)


@pytest.mark.parametrize("N", [5, 400])
def test_repeats_are_bitwise_equal(N):
    """On one workspace, after other sizes ran on it, and on another one."""
    s = cuda(inputs(10, N, 128, 136, 128, 5, 2, "bf16", cut=0.2))
    other = cuda(inputs(11, max(1, N // 3), 64, 64, 64, 2, 1, "bf16"))
    y0, ws = forward(s, "gelu", ws=workspace(s, False, True))
    g0, _ = backward(s, "gelu", ws=ws)
    forward(other, "gelu", ws=ws)
    backward(other, "gelu", ws=ws)
    for _ in range(3):
        y1, _ = forward(s, "gelu", ws=ws)
        g1, _ = backward(s, "gelu", ws=ws)
        assert torch.equal(y0, y1) and all(torch.equal(g0[k], g1[k]) for k in g0)
    y2, _ = forward(s, "gelu")
    assert torch.equal(y0, y2)


@pytest.mark.parametrize("N,d,h,o,K,r,dtype,gated", [
    (300, 64, 72, 136, 6, 2, "bf16", True),       # segments end inside tiles
    (900, 64, 0, 264, 2, 1, "f16", False),        # pairs of row tiles
    (130, 33, 21, 65, 5, 3, "bf16", False),       # padded copies
    (300, 64, 72, 136, 1, 0, "f16", True),
    (4, 64, 72, 136, 6, 2, "bf16", True),         # few points forward
    (300, 40, 72, 136, 6, 2, "f32", True),
    (5000, 40, 24, 16, 60, 1, "f32", False),      # counting sort in steps
])
def test_contents_of_the_workspace_do_not_matter(N, d, h, o, K, r, dtype, gated):
    """Only its error word has to be clear: the rest may hold NaNs."""
    use = list(range(K - 1)) or None              # an expert that nobody uses
    s = cuda(inputs(13, N, d, h, o, K, r, dtype, gated, cut=0.2 if r else 0.0, use=use))
    ws = workspace(s, gated, True)
    ws.view.zero_()
    y0, _ = forward(s, "silu", gated, ws=ws)
    ws.view.zero_()
    g0, _ = backward(s, "silu", gated, ws=ws)
    for run in (lambda: ({"y": forward(s, "silu", gated, ws=ws)[0]}, {"y": y0}),
                lambda: (backward(s, "silu", gated, ws=ws)[0], g0)):
        ws.view[256:] = 255
        got, want = run()
        assert gmm.gmm_last_error(ws) == 0
        for k in want:
            assert torch.equal(got[k], want[k]) and got[k].isfinite().all(), k


@pytest.mark.parametrize("N", [3, 200])
def test_captured_calls(N):
    """Two captured graphs with a workspace each, replayed in turn on new
    inputs, give what eager calls give."""
    sets = [cuda(inputs(20 + i, N, 64, 72, 64, 4, 2, "bf16")) for i in range(2)]
    graphs = []
    for c in sets:
        ws = workspace(c, False, True)
        forward(c, "silu", ws=ws)
        backward(c, "silu", ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, _ = forward(c, "silu", ws=ws)
            g, _ = backward(c, "silu", ws=ws)
        graphs.append((graph, c, y, g))
    for turn in range(2):
        for graph, c, y, g in graphs:
            c["x"].copy_(torch.randn(c["x"].shape, device="cuda"))
            c["ids"].copy_(torch.randint(-1, 4, c["ids"].shape, device="cuda"))
            graph.replay()
        for graph, c, y, g in graphs:
            torch.cuda.synchronize()
            assert torch.equal(y, forward(c, "silu")[0])
            want = backward(c, "silu")[0]
            assert all(torch.equal(g[k], want[k]) for k in want)


def test_another_stream():
    """The stream argument: outputs are allocated on it, and two calls on two
    streams with a workspace each run at once."""
    s = cuda(inputs(12, 300, 128, 136, 128, 5, 2, "bf16"))
    want = forward(s, "gelu")[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [workspace(s, False, False) for _ in range(2)]
    torch.cuda.synchronize()
    got = [forward(s, "gelu", ws=w, stream=st)[0] for _ in range(4) for w, st in zip(spaces, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


@pytest.mark.parametrize("gated", [False, True])
def test_gradients_against_differences(gated):
    """fp32 gradients against central differences of the float64 formula: the
    truncation of a difference of step t is t^2/6 of the third derivative; at
    t = 1e-4 it is far below the bounds of the fp32 results."""
    s = inputs(13, 12, 10, 9, 8, 3, 2, "f32", gated=gated)
    got, _ = backward(cuda(s), "gelu", gated)
    _, b = reference(s, "gelu", gated, torch.float32)

    def loss(t):
        y = reference_y(t, "gelu", gated)
        return float((y * s["dy"].double()).sum())

    g = torch.Generator().manual_seed(1)
    for name, key in (("x", "dx"), ("w1", "dw1"), ("b1", "db1"), ("w2", "dw2"), ("b2", "db2"),
                      ("resp", "dresp")):
        flat = s[name].double().reshape(-1)
        for at in torch.randperm(flat.numel(), generator=g)[:6].tolist():
            vals = []
            for sign in (1, -1):
                t = flat.clone()
                t[at] += sign * 1e-4
                vals.append(loss(dict(s, **{name: t.reshape(s[name].shape)})))
            diff = (vals[0] - vals[1]) / 2e-4
            have = float(got[key].reshape(-1)[at])
            assert abs(have - diff) <= float(b[key].reshape(-1)[at]) + 1e-6 * (1 + abs(diff)), (
                name, at, have, diff)


def reference_y(s, activation, gated):
    y = torch.zeros(s["dy"].shape, dtype=torch.float64)
    for e in range(s["w1"].shape[0]):
        n, i = torch.where(s["ids"] == e)
        z = s["x"].double()[n] @ s["w1"][e].double().T + s["b1"][e].double()
        if gated:
            a, u = z.chunk(2, 1)
            hid = act(a, activation) * u
        else:
            hid = act(z, activation)
        y.index_add_(0, n, s["resp"].double()[n, i][:, None] *
                     (hid @ s["w2"][e].double().T + s["b2"][e].double()))
    return y


def test_soft_assignment_to_trained_experts():
    """The whole path: a fitted mixture routes its points, the experts' layer
    runs forward and backward on the routing as it is, for a batch and for
    single points."""
    g = torch.Generator().manual_seed(14)
    K, d, N, r, h, o = 6, 64, 900, 3, 96, 32
    centres = torch.randn(K, d, generator=g) * 1.2
    X = (centres[torch.randint(K, (N,), generator=g)] + torch.randn(N, d, generator=g)).to(
        torch.bfloat16).cuda()
    m, v, lw = gmm.init_kmeans(X, X[:K].float().contiguous(), iters=3)
    m, v, lw, _, _ = gmm.fit(X, m, v, lw, max_iters=5)
    ws = gmm.Workspace.for_gmm(N, d, K, X.dtype)
    ids, resp, _ = gmm.soft_assign(X, m, v, lw, r, 0.02, ws)
    s = inputs(15, N, d, h, o, K, r, "bf16", gated=True, res=True)
    s.update(x=X.cpu(), ids=ids.cpu(), resp=resp.cpu())
    check(s, "silu", True)
    one = dict(s, **{k: s[k][:1].contiguous() for k in ("x", "ids", "resp", "dy", "res")})
    check(one, "silu", True)
    # the hard partition of k-means, one component a point
    _, _, _, hard = gmm.init_kmeans(X, m, iters=1, want_ids=True)
    check(dict(s, ids=hard[:, None].cpu().contiguous(), resp=None), "silu", True)
