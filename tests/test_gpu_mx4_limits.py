"""The 4-bit product and the expert layer give up their waits at the wait limit, and the GPU
stays usable.

The expert layer's grid waits at four barriers for the number of its CTAs; a counter that
starts at -1 never shows it, so every CTA gives up there, with what it has in flight
ended.

The product: at the shortest limit (1 us) on a weight that has to come from memory (328 MB, more than
L2 holds, for the kernel of few tokens; rows of 32768, a tile's accumulators tens of
microseconds away, for the pairs of SMs) some wait of every call lasts longer: the call
reports the timeout, ends long before the usual limit of two seconds, writes nothing
behind y, and the next call with the usual limit is right.
"""
import time

import pytest
import torch

from tests.test_gpu_parity import status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


def matrix(rows, cols, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8),
            torch.randint(117, 138, (rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,d_out", [(3, 20000), (16, 20000), (17, 20000), (64, 20000),  # up to 64 tokens a tile
                                     (129, 20000), (300, 8192), (2048, 4096)])  # pairs of SMs
def test_every_wait_ends_at_the_limit(L, M, d_out, out):
    x, w = matrix(M, 32768, 500 + M), matrix(d_out, 32768, 501)
    want = L.larosa_mx4_linear(*x, *w, dtype=out)
    buf = torch.full((M * d_out + 8192,), 7.0, dtype=out, device="cuda")
    y = buf[:M * d_out].view(M, d_out)
    st = status()
    torch.cuda.synchronize()
    for _ in range(3):
        st.zero_()
        previous = L.larosa_set_wait_limit_ns(1000)
        try:
            t0 = time.perf_counter()
            L.larosa_mx4_linear(*x, *w, y=y, dev_status=st)
            torch.cuda.synchronize()
            elapsed = time.perf_counter() - t0
        finally:
            L.larosa_set_wait_limit_ns(previous)
        assert elapsed < 1.0, elapsed
        with pytest.raises(L.LarosaError) as err:
            L.larosa_check(st)
        assert err.value.status == L.LAROSA_ERR_TIMEOUT
        assert torch.all(buf[M * d_out:] == 7.0)
        st.zero_()
        L.larosa_mx4_linear(*x, *w, y=y, dev_status=st)
        assert L.larosa_check(st) == 0 and torch.equal(y, want)


@pytest.mark.parametrize("experts", ["bf16", "f32", "mx4"])
@pytest.mark.parametrize("barrier", [0, 1, 2, 3])
def test_every_barrier_of_the_expert_layer_gives_up(L, experts, barrier):
    from tests.test_gpu_moe import Layer
    M, d, f, E, k = 9, 256, 160, 8, 3
    layer = Layer(L, M, d, f, E, "mx4" if experts == "mx4" else "plain",
                  torch.float32 if experts == "f32" else torch.bfloat16, 510)
    ws, st = L.Workspace(), status()
    want = layer.run(L, k, ws=ws, dev_status=st)
    torch.cuda.synchronize()
    ws.buf[4 * barrier:4 * barrier + 4].view(torch.int32).fill_(-1)
    previous = L.larosa_set_wait_limit_ns(1_000_000)
    try:
        t0 = time.perf_counter()
        layer.run(L, k, ws=ws, dev_status=st)
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        L.larosa_set_wait_limit_ns(previous)
    assert elapsed < 1.0, elapsed
    assert int(st.item()) == L.LAROSA_DEV_TIMEOUT
    ws.reset()
    st.zero_()
    again = layer.run(L, k, ws=ws, dev_status=st)
    assert L.larosa_check(st) == 0 and all(torch.equal(a, b) for a, b in zip(again, want))
