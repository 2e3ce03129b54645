"""Mixtures of experts on the components of an assignment (gmm_expert_*).

``soft_assign`` lists up to r components of every point with their
responsibilities; the calls here send the point through the maps of those
components and add the results up by responsibility.  k-means ids serve as
``ids`` [N, 1] with ``resp=None``; ``ids=None`` is a dense layer (one expert).

    ids, resp, _ = gmm.soft_assign(X, means, variances, logw, r, tau, ws)
    ews = gmm.Workspace.for_expert_mlp(N, d, h, o, K, r, X.dtype, gated=True, backward=True)
    Y = gmm.expert_mlp(X, ids, resp, W1, b1, W2, b2, ews, activation="silu", gated=True)
    dX, dW1, db1, dW2, db2, dresp = gmm.expert_mlp_backward(
        dY, X, ids, resp, W1, b1, W2, b2, ews, activation="silu", gated=True)

Argument marshalling only, as in ``api``; include/gmm_b200.h states each
operation.  Calls that share a workspace must not overlap in time on the
device (two captured graphs that may run at once need one each).  ``stream``
(default: the current one of X's device) is where a call runs and its outputs
belong; its inputs have to be ready there.  Arrays given to a call with
``stream`` may be dropped at once: their memory is kept until it is done.
Bases of X, dY, the weights and ``out`` must be 16-byte aligned where their rows
are whole 16-byte units (whole tensors are).  An id at or above K is skipped and recorded: ``gmm_last_error(ws)``
reports GMM_ERR_RANGE.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import GMM_FLAG_NONE, ExpertShape, check
from .api import _DT, Workspace, keep_for

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}

__all__ = ["expert_linear", "expert_linear_backward", "expert_mlp", "expert_mlp_backward",
           "expert_path", "expert_workspace_size"]


_shapes = {}   # ExpertShape (and its pointer) by the values it holds


def _shape(N, d, h, o, K, r, dtype, activation="none", gated=False):
    key = (N, d, h, o, K, r, dtype, activation, gated)
    p = _shapes.get(key)
    if p is None:
        if activation not in ACTIVATIONS:
            raise ValueError(
                f"activation: expected one of {sorted(ACTIVATIONS)}, got {activation!r}")
        if dtype not in _DT:
            raise ValueError("dtype must be float32, bfloat16 or float16")
        if len(_shapes) >= 4096:
            _shapes.clear()
        # (ctypes would cut larger numbers down to valid ones)
        N, d, h, o, K, r = (v if abs(v) < 1 << 31 else -1 for v in (N, d, h, o, K, r))
        p = _shapes[key] = ctypes.pointer(ExpertShape(
            N=N, d=d, h=h, o=o, K=K, r=r, dtype=_DT[dtype], activation=ACTIVATIONS[activation],
            gated=int(bool(gated))))
    return p


def expert_workspace_size(N: int, d: int, h: int, o: int, K: int, r: int, dtype=torch.float32,
                          gated: bool = False, backward: bool = False,
                          flags: int = GMM_FLAG_NONE) -> int:
    """Bytes of workspace of expert_linear (h = 0) or expert_mlp, 0 for invalid
    sizes; r = 0 is the dense form."""
    return int(_lib.load().gmm_expert_workspace_size(
        _shape(N, d, h, o, K, r, dtype, gated=gated), int(backward), int(flags)))


def expert_path(N: int, d: int, h: int, o: int, K: int, r: int, dtype=torch.float32,
                gated: bool = False, backward: bool = False, flags: int = GMM_FLAG_NONE) -> int:
    """Which kernels a call of these sizes runs: 0 CUDA cores, 1 the form for
    few points, 2 tensor cores (gmm_expert_path)."""
    path = int(_lib.load().gmm_expert_path(
        _shape(N, d, h, o, K, r, dtype, gated=gated), int(backward), int(flags)))
    if path < 0:
        raise ValueError("invalid problem size")
    return path


def _tensor(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or \
            t.device != dev or not t.is_contiguous():
        got = f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor) else t
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {dev}, got {got}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: these calls do not record autograd history; pass "
                         "detached tensors and call the _backward function")
    return t


class _Call:
    """The arguments the four calls share, checked, with the device and the
    stream they run on.  As a context it makes both current where they are
    not, so that outputs belong to the stream that writes them."""

    __slots__ = ("dev", "dtype", "N", "d", "h", "o", "K", "r", "first", "shape", "ws", "stream",
                 "guard", "side")

    def __init__(self, X, ids, resp, W1, W2, ws, activation, gated, stream):
        if not isinstance(X, torch.Tensor) or X.dim() != 2 or X.dtype not in _DT or not X.is_cuda:
            raise ValueError("X must be a contiguous cuda float32/bfloat16/float16 [N, d] tensor")
        dev, dtype, size = X.device, X.dtype, X.shape
        _tensor(X, "X", dtype, size, dev)
        N, d = size
        for w in (W1,) if W2 is None else (W1, W2):
            if not isinstance(w, torch.Tensor) or w.dim() != 3:
                raise ValueError("weights must be [K, out, in] tensors")
        K, first, _ = W1.shape
        if W2 is None:
            h, o = 0, first
            _tensor(W1, "W", dtype, (K, first, d), dev)
        else:
            if gated and first % 2:
                raise ValueError("gated: W1 must have 2h rows")
            h, o = first // 2 if gated else first, W2.shape[1]
            _tensor(W1, "W1", dtype, (K, first, d), dev)
            _tensor(W2, "W2", dtype, (K, o, h), dev)
        if ids is None:
            if resp is not None:
                raise ValueError("resp needs ids")
            if K != 1:
                raise ValueError(f"without ids there is one expert, got {K}")
            r = 0
        else:
            if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
                raise ValueError("ids must be an int32 [N, r] tensor")
            r = ids.shape[1]
            _tensor(ids, "ids", torch.int32, (N, r), dev)
            if not 1 <= r <= 8:
                raise ValueError(f"r must be 1..8, got {r}")
            if resp is not None:
                _tensor(resp, "resp", torch.float32, (N, r), dev)
        if not isinstance(ws, Workspace) or ws.view.device != dev:
            raise ValueError(f"ws must be a Workspace on {dev}")
        self.dev, self.dtype, self.ws = dev, dtype, ws
        self.N, self.d, self.h, self.o, self.K, self.r, self.first = N, d, h, o, K, r, first
        self.shape = _shape(N, d, h, o, K, r, dtype, activation, bool(gated))
        self.guard, self.side = None, stream
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, X on {dev}")
            self.guard = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != dev.index:
            self.guard = torch.cuda.device(dev)

    def bias(self, b, name, width):
        if b is not None:
            _tensor(b, name, self.dtype, (self.K, width), self.dev)

    def rows(self, t, name, width):
        return _tensor(t, name, self.dtype, (self.N, width), self.dev)

    def out(self, t, width):
        return torch.empty((self.N, width), dtype=self.dtype, device=self.dev) if t is None \
            else self.rows(t, "out", width)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        # (torch.cuda.current_stream(), without building a Stream)
        self.stream = torch._C._cuda_getCurrentRawStream(self.dev.index)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def run(self, name, fn, flags, *args):
        status = fn(self.shape, *[None if t is None else t.data_ptr() for t in args], self.ws.ptr,
                    self.ws.nbytes, int(flags), self.stream)
        if self.side is not None:   # (a failed call may have launched a part of it)
            keep_for(self.side, self.ws.buf, *args)
        check(name, status)


def _like(t):
    return None if t is None else torch.empty_like(t)


def expert_linear(X, ids, resp, W, b, ws: Workspace, activation: str = "none", residual=None,
                  out=None, flags: int = GMM_FLAG_NONE, stream=None) -> torch.Tensor:
    """y_n = sum_i resp_ni f(W_e x_n + b_e) + residual_n, e = ids_ni
    (gmm_expert_linear).  X [N, d]; ids [N, r] int32 (-1: none) or None;
    resp [N, r] fp32 or None; W [K, o, d]; b [K, o] or None; residual [N, o]
    or None.  Returns [N, o], written to ``out`` when given (which may be the
    residual)."""
    c = _Call(X, ids, resp, W, None, ws, activation, False, stream)
    c.bias(b, "b", c.o)
    if residual is not None:
        c.rows(residual, "residual", c.o)
    with c:
        Y = c.out(out, c.o)
        c.run("gmm_expert_linear", _lib.load().gmm_expert_linear, flags, X, ids, resp, W, b,
              residual, Y)
    return Y


def expert_linear_backward(dY, X, ids, resp, W, b, ws: Workspace, activation: str = "none",
                           flags: int = GMM_FLAG_NONE, stream=None):
    """Gradients of expert_linear's inputs for dY [N, o]: (dX, dW, db or None,
    dresp or None).  The residual's gradient is dY itself."""
    c = _Call(X, ids, resp, W, None, ws, activation, False, stream)
    c.bias(b, "b", c.o)
    c.rows(dY, "dY", c.o)
    with c:
        dX, dW, db, dresp = _like(X), _like(W), _like(b), _like(resp)
        c.run("gmm_expert_linear_backward", _lib.load().gmm_expert_linear_backward, flags, dY, X,
              ids, resp, W, b, dX, dW, db, dresp)
    return dX, dW, db, dresp


def expert_mlp(X, ids, resp, W1, b1, W2, b2, ws: Workspace, activation: str = "silu",
               gated: bool = False, residual=None, out=None, flags: int = GMM_FLAG_NONE,
               stream=None) -> torch.Tensor:
    """y_n = sum_i resp_ni (W2_e h + b2_e) + residual_n with h = f(W1_e x_n + b1_e),
    or, gated, h = f(a) * u for [a, u] = W1_e x_n + b1_e (gmm_expert_mlp).
    W1 [K, h or 2h, d], b1 [K, h or 2h] or None, W2 [K, o, h], b2 [K, o] or
    None; the rest as expert_linear."""
    c = _Call(X, ids, resp, W1, W2, ws, activation, gated, stream)
    c.bias(b1, "b1", c.first)
    c.bias(b2, "b2", c.o)
    if residual is not None:
        c.rows(residual, "residual", c.o)
    with c:
        Y = c.out(out, c.o)
        c.run("gmm_expert_mlp", _lib.load().gmm_expert_mlp, flags, X, ids, resp, W1, b1, W2, b2,
              residual, Y)
    return Y


def expert_mlp_backward(dY, X, ids, resp, W1, b1, W2, b2, ws: Workspace, activation: str = "silu",
                        gated: bool = False, flags: int = GMM_FLAG_NONE, stream=None):
    """Gradients of expert_mlp's inputs for dY [N, o]: (dX, dW1, db1 or None,
    dW2, db2 or None, dresp or None).  The residual's gradient is dY itself.
    Needs a workspace made with ``backward=True``."""
    c = _Call(X, ids, resp, W1, W2, ws, activation, gated, stream)
    c.bias(b1, "b1", c.first)
    c.bias(b2, "b2", c.o)
    c.rows(dY, "dY", c.o)
    with c:
        dX, dW1, db1, dW2, db2, dresp = (_like(t) for t in (X, W1, b1, W2, b2, resp))
        c.run("gmm_expert_mlp_backward", _lib.load().gmm_expert_mlp_backward, flags, dY, X, ids,
              resp, W1, b1, W2, b2, dX, dW1, db1, dW2, db2, dresp)
    return dX, dW1, db1, dW2, db2, dresp
