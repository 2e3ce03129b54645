"""Calls with ``stream``: behind a busy stream, with every array dropped as soon
as the call returns, they give what calls on the current stream give."""
import pytest
import torch

import means_clustering_gmm_b200 as gmm

pytestmark = pytest.mark.gpu
N, D, K = 3000, 32, 12


def arrays():
    g = torch.Generator().manual_seed(3)
    X = (torch.randn(N, D, generator=g) + 4 * torch.randint(3, (N, 1), generator=g)).cuda()
    return [X, X[:K].clone(), torch.full((K, D), 3.0, device="cuda"),
            torch.full((K,), 1.0 / K, device="cuda").log()]


def em_step(X, m, v, lw, stream=None):
    return gmm.gmm_em_step(X, m, v, lw, gmm.Workspace.for_gmm(N, D, K), stream=stream)[::2]


def em_iteration(X, m, v, lw, stream=None):
    return (*gmm.em_iteration(X, m, v, lw, gmm.Workspace.for_gmm(N, D, K), stream=stream)[::2], m,
            v, lw)


def soft_assign(X, m, v, lw, stream=None):
    return gmm.soft_assign(X, m, v, lw, 3, 0.01, gmm.Workspace.for_gmm(N, D, K), stream=stream)[:2]


def batched(X, m, v, lw, stream=None):
    X, m, v, lw = X.view(2, N // 2, D), m.view(2, K // 2, D), v.view(2, K // 2, D), lw.view(2, -1)
    ws = gmm.BatchedWorkspace(2, N // 2, D, K // 2)
    out = gmm.gmm_em_step_batched(X, m, v, lw, ws, stream=stream)[::2]
    return (*out, *gmm.gmm_finalize_batched(out[0], N // 2, m, v, lw, ws, stream=stream))


def kmeans_step(X, m, v, lw, stream=None):
    return gmm.kmeans_step(X, m, gmm.Workspace.for_kmeans(1, N, D, K), stream=stream)


def init_kmeans(X, m, v, lw, stream=None):
    return gmm.init_kmeans(X, m, iters=2, want_ids=True, stream=stream)


def fit(X, m, v, lw, stream=None):
    return gmm.fit(X, m, v, lw, max_iters=3, stream=stream)[:4]


@pytest.mark.parametrize("call", [em_step, em_iteration, soft_assign, batched, kmeans_step,
                                  init_kmeans, fit])
def test_arrays_may_be_dropped_behind_a_busy_stream(call):
    want = call(*arrays())
    side = torch.cuda.Stream()
    call(*arrays(), stream=side)   # (the stream's own memory)
    torch.cuda.synchronize()
    given = arrays()
    torch.cuda.synchronize()
    read = given[:2] if call in (kmeans_step, init_kmeans) else given
    busy = {t.data_ptr(): (t.shape, t.dtype) for t in read}
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)   # clocks: 0.5 s
    got = call(*given, stream=side)
    if call is fit:   # reads its result on the host
        assert side.query()
    else:
        assert not side.query()   # (otherwise nothing is shown)
        kept = {t.data_ptr() for t in got}
        del given, read
        new = [torch.empty(s, dtype=t, device="cuda") for s, t in busy.values()]
        new += [torch.empty(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(64)]
        assert not (busy.keys() | kept) & {t.data_ptr() for t in new}
        for t in new:
            t.fill_(1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
