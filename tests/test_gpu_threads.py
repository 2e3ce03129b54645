"""Calls of different sizes at once, on host threads with a stream and a
workspace each."""
import sys
import threading

import pytest
import torch

import means_clustering_gmm_b200 as gmm

pytestmark = pytest.mark.gpu
SIMT = gmm.GMM_FLAG_FORCE_SIMT


def kmeans(K):
    g = torch.Generator().manual_seed(K)
    X = torch.randn(1, 5000, 16, generator=g).cuda()
    C = X[:, :K].contiguous()
    ws = gmm.Workspace.for_kmeans(1, 5000, 16, K)
    return lambda stream: gmm.kmeans_step(X, C, ws, stream=stream)[:2]


def em(d, K):
    g = torch.Generator().manual_seed(K)
    X = torch.randn(2000, d, generator=g).cuda()
    m, v = X[:K].contiguous(), torch.ones(K, d, device="cuda")
    lw = torch.full((K,), -float(K)).log_softmax(0).cuda()
    ws = gmm.Workspace.for_gmm(2000, d, K)
    return lambda stream: gmm.gmm_em_step(X, m, v, lw, ws, flags=SIMT, stream=stream)[:1]


@pytest.mark.parametrize("make,sizes", [(kmeans, [(8,), (4096,)]), (em, [(8, 4), (300, 40)])])
def test_threads_with_calls_of_different_sizes(make, sizes):
    failed, results = [], []

    def loop(call, stream, want):
        try:
            for i in range(4000):
                with torch.cuda.stream(stream):   # (outputs are the stream's)
                    got = call(stream)
                if i % 50 == 49:
                    stream.synchronize()
            results.append(all(torch.equal(a, b) for a, b in zip(got, want)))
        except gmm.GmmError as e:
            failed.append(e)

    threads = []
    for size in 2 * sizes:
        call = make(*size)   # a workspace of its own
        want = call(None)
        torch.cuda.synchronize()
        threads.append(threading.Thread(target=loop, args=(call, torch.cuda.Stream(), want)))
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not failed, (len(failed), failed[0])
    assert results == [True] * 4
