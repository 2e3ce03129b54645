"""Host-side checks of the experts' entry points (no GPU needed)."""
import ctypes

import pytest
import torch

import means_clustering_gmm_b200 as gmm
from means_clustering_gmm_b200 import _lib

A = 1 << 20   # a fake, 256-aligned, never-dereferenced address
E = _lib.GMM_ERR_INVALID_ARG
BF16, F32 = _lib.GMM_BF16, _lib.GMM_F32


def shape(**kw):
    return _lib.ExpertShape(**dict(dict(N=100, d=64, h=0, o=32, K=4, r=2, dtype=BF16, activation=2,
                                        gated=0), **kw))


def size(s, backward=0, flags=0):
    return _lib.load().gmm_expert_workspace_size(ctypes.byref(s), backward, flags)


BAD_SHAPES = [dict(N=0), dict(d=0), dict(o=0), dict(K=0), dict(r=-1), dict(r=9), dict(r=0),
              dict(dtype=3), dict(dtype=-1), dict(activation=4), dict(activation=-1),
              dict(gated=1), dict(gated=2, h=8), dict(h=-1), dict(d=1 << 20), dict(o=1 << 20),
              dict(h=1 << 20), dict(K=5000), dict(N=1 << 31), dict(N=1 << 30)]


@pytest.mark.parametrize("bad", BAD_SHAPES)
def test_invalid_shapes(bad):
    lib = _lib.load()
    s = shape(**bad)
    assert size(s) == 0 and size(s, 1) == 0
    assert lib.gmm_expert_path(ctypes.byref(s), 0, 0) == -1
    fn = lib.gmm_expert_mlp if s.h else lib.gmm_expert_linear
    args = (A, A, A, A, A) + ((A, A) if s.h else ()) + (A, A + 256, A, 1 << 40, 0, None)
    assert fn(ctypes.byref(s), *args) == E


def test_sizes_and_flags():
    assert 0 < size(shape()) < size(shape(), 1)
    assert size(shape(h=64)) > size(shape())
    assert size(shape(), 0, 64) == 0
    assert size(shape(r=0, K=1)) > 0
    # 16-bit operands for the tensor cores, fp32 ones for the CUDA cores
    big = shape(N=10000, h=1024, d=512, o=512)
    assert size(big, 1) < size(big, 1, _lib.GMM_FLAG_FORCE_SIMT)
    # copies where a width is not a multiple of 8
    assert size(shape(d=63)) > size(shape()) and size(shape(o=31), 1) > size(shape(), 1)
    # nothing of size N x K x width: rows grow with the pairs
    assert size(shape(N=100000, h=64, K=64), 1) < 2 * size(shape(N=100000, h=64, K=4), 1)
    assert _lib.load().gmm_expert_workspace_size(None, 0, 0) == 0


def linear(**kw):
    a = dict(s=shape(), X=A, ids=A, resp=A, W=A, b=A, res=A, Y=A + 4096, ws=A, wsb=None, fl=0)
    a.update(kw)
    wsb = size(a["s"], 0, a["fl"]) if a["wsb"] is None else a["wsb"]
    return _lib.load().gmm_expert_linear(ctypes.byref(a["s"]), a["X"], a["ids"], a["resp"], a["W"],
                                         a["b"], a["res"], a["Y"], a["ws"], wsb, a["fl"], None)


def test_linear_refusals():
    for k in ("X", "W", "Y"):
        assert linear(**{k: None}) == E
        assert linear(**{k: A + 8}) == E          # 16-byte aligned
    for k in ("ids", "resp", "b", "res"):
        assert linear(**{k: A + 1}) == E
    assert linear(ws=None) == E
    assert linear(ws=A + 64) == E
    assert linear(wsb=size(shape()) - 1) == E
    assert linear(fl=64) == E
    assert linear(fl=1) == E
    assert linear(ids=None) == E                  # r = 2 needs ids
    assert linear(s=shape(r=0, K=1)) == E         # and the dense form has none
    assert linear(s=shape(r=0, K=1), ids=None) == E   # nor weights
    assert linear(s=shape(h=64)) == E             # the mlp's shape
    assert linear(Y=A) == E                       # X itself


def test_backward_refusals():
    lib = _lib.load()
    names = ["dY", "X", "ids", "resp", "W1", "b1", "W2", "b2", "dX", "dW1", "db1", "dW2", "db2",
             "dresp"]
    need = size(shape(h=64), 1)

    def call(wsb=need, ws=A, fl=0, s=None, **kw):
        a = {n: A + 4096 * i for i, n in enumerate(names)}
        a.update(kw)
        return lib.gmm_expert_mlp_backward(ctypes.byref(s or shape(h=64)), *[a[n] for n in names],
                                           ws, wsb, fl, None)

    for k in ("dY", "X", "W1", "W2", "dX", "dW1", "dW2"):
        assert call(**{k: None}) == E
        assert call(**{k: A + 8}) == E
    for k in ("db1", "db2", "dresp", "b1", "b2", "resp"):
        assert call(**{k: None}) == E             # an input and its gradient go together
    assert call(ids=None) == E
    assert call(wsb=need - 1) == E
    assert call(ws=A + 128) == E
    assert call(fl=2) == E                        # the CUDA-core form needs more workspace
    assert call(s=shape()) == E
    assert call(dX=A + 4096) == E                 # X itself
    fwd = size(shape(h=64), 0)
    assert fwd < need and call(wsb=fwd) == E


def test_binding_refuses_on_the_host():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="X must be"):
        gmm.expert_linear(x, None, None, torch.zeros(1, 8, 8), None, None)
    with pytest.raises(ValueError, match="X must be"):
        gmm.expert_mlp(x, None, None, x, None, x, None, None)
    with pytest.raises(ValueError, match="activation"):
        gmm.experts._shape(1, 8, 0, 8, 1, 0, torch.bfloat16, "tanh")
    with pytest.raises(ValueError, match="dtype"):
        gmm.expert_workspace_size(1, 8, 0, 8, 1, 0, torch.float64)
    with pytest.raises(ValueError):
        gmm.Workspace.for_expert_linear(0, 8, 8, 1, 0, torch.float32)
    with pytest.raises(ValueError):
        gmm.expert_path(1, 8, 0, 8, 2, 0)
    bf = torch.bfloat16
    assert gmm.expert_path(64, 8, 0, 8, 9, 4, bf) == 1
    assert gmm.expert_path(64, 8, 16, 8, 9, 5, bf) == 2       # more pairs
    assert gmm.expert_path(65, 8, 16, 8, 9, 1, bf) == 2       # more points
    assert gmm.expert_path(1, 8, 16, 8, 9, 1, bf, backward=True) == 2
    assert gmm.expert_path(100, 7, 0, 8, 2, 1, bf) == 2       # on padded copies
    assert gmm.expert_path(5, 7, 0, 8, 2, 1, bf) == 2
    assert gmm.expert_path(100, 8, 0, 8, 2, 1, torch.float32) == 0
    assert gmm.expert_path(100, 8, 0, 8, 2, 1, bf, flags=gmm.GMM_FLAG_FORCE_SIMT) == 0
