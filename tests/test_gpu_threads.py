"""Calls on different workspaces may run at once.  Kernels whose shared memory goes by a call's sizes are called from two
threads, each on its own stream, with sizes that differ; the calls release Python's lock, so they meet."""
import threading

import pytest
import torch

import contextual_sparsity_sparse_gb300 as cs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def at_once(makers, calls):
    """Each maker gives a call and a check of its result; both are made and called `calls` times in a thread and on a
    stream of their own."""
    errors, gate = [], threading.Barrier(len(makers))

    def work(make):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                call, check = make()
                torch.cuda.current_stream().synchronize()
                gate.wait(60)
                for _ in range(calls):
                    call()
                torch.cuda.current_stream().synchronize()
                check()
        except Exception as e:   # noqa: BLE001 (told to the main thread)
            errors.append(e)
            gate.abort()

    threads = [threading.Thread(target=work, args=(m,)) for m in makers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_cache_attention_of_small_and_large_batches():
    def maker(batch):
        def make():
            g = torch.Generator("cuda").manual_seed(batch)
            cache = cs.QCache.empty(batch, 1, 4, 64)
            rows = torch.randn(batch, 4, 1, 64, generator=g, device="cuda")
            zero = torch.zeros(batch, dtype=torch.int32, device="cuda")
            ws = cs.QCacheWorkspace(cache)
            cs.cs_qcache_append(cache, rows, rows, ws, start=zero, pos=zero)
            q = torch.randn(batch, 1, 1, 64, generator=g, device="cuda")
            length, out, first = torch.full_like(zero, 4), torch.empty_like(q), torch.empty_like(q)
            cs.cs_qcache_attention(cache, q, length, first, ws)

            def check():
                assert torch.equal(out, first) and out.any()
            return lambda: cs.cs_qcache_attention(cache, q, length, out, ws), check
        return make
    at_once([maker(1), maker(4096)], 3000)


@pytest.mark.parametrize("sizes", [(512, 8192), (2560, 5120)])
def test_predictors_of_small_and_large_layers(sizes):
    def maker(d):
        def make():
            f, r = 4096, 256
            g = torch.Generator("cuda").manual_seed(d)
            rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
            pred = cs.Predictor(rand(r, d).half(), rand(f, r).half())
            x, out, first = rand(d), torch.zeros(f, device="cuda"), torch.zeros(f, device="cuda")
            ws = cs.Workspace(d, f, r)
            cs.cs_predict(pred, x, first, ws)

            def check():
                assert torch.equal(out, first) and out.any()
            return lambda: cs.cs_predict(pred, x, out, ws), check
        return make
    at_once([maker(d) for d in sizes], 3000)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("B", [1, 2])
@pytest.mark.parametrize("sizes", [(4096, 5120), (512, 8192)])
def test_layers_of_two_widths(sizes, B, glu):
    def maker(d):
        def make():
            f = 2048
            g = torch.Generator("cuda").manual_seed(d)
            rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
            layer = cs.FfnLayer(rand(f, d).half(), rand(f, d).half(), w_up=rand(f, d).half() if glu else None)
            x, out, first = rand(B, d), torch.zeros(B, d, device="cuda"), torch.zeros(B, d, device="cuda")
            idx = torch.arange(f, dtype=torch.int32, device="cuda").repeat(B, 1)
            count = torch.full((B,), 64, dtype=torch.int32, device="cuda")
            ws = cs.Workspace(d, f, 64, B=B)
            cs.cs_sparse_ffn(layer, x, idx, count, first, ws)

            def check():
                assert torch.equal(out, first) and out.any()
            return lambda: cs.cs_sparse_ffn(layer, x, idx, count, out, ws), check
        return make
    at_once([maker(d) for d in sizes], 3000)
