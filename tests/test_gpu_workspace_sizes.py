"""What the entry points ask of a workspace.

The calls on bf16 and fp32 weights never touch the 4-bit product's
coefficients and partial sums, so what they ask for does not depend on whether
the sizes suit the 4-bit format (d_out a multiple of 32): a row-major weight of
d_out - 8 columns (which the format does not take) needs the same but for the
columns themselves, at most 1 % of the partial sums and a tile's rounding.
"""
import ctypes

import pytest
import torch

import synthdata as sd
from tests.test_gpu_parity import status

pytestmark = pytest.mark.gpu

ERR_WORKSPACE = 6
SHAPES = [(1, 4096, 22016, 2458), (16, 4096, 22016, 2458), (4, 1024, 4096, 600), (16, 13824, 5120, 8295)]


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


def least(call, most):
    """The fewest workspace bytes that `call` accepts (its buffer has `most`)."""
    assert call(most) == 0
    lo, hi = 0, most  # lo refused, hi accepted
    assert call(lo) == ERR_WORKSPACE
    while hi - lo > 1:
        mid = (lo + hi) // 2
        st = call(mid)
        assert st in (0, ERR_WORKSPACE)
        lo, hi = (lo, mid) if st == 0 else (mid, hi)
    torch.cuda.synchronize()
    return hi


class Calls:
    def __init__(self, M, d_in, d_out, K):
        from activation_sparsity_b200 import larosa
        self.lib = larosa.raw_library()
        self.sizes = M, d_in, d_out, K
        t = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.W, self.x = t(d_in, d_out, dt=torch.bfloat16), t(M, d_in, dt=torch.bfloat16)
        self.x_rot, self.y, self.st = t(M, d_in), t(M, d_out), status()
        self.idx, self.val = (a.cuda() for a in sd.index_values(M, d_in, K, 5))
        self.most = int(self.lib.larosa_workspace_bytes(M, d_in, d_out, K)) + (1 << 20)
        self.buf = t(self.most, dt=torch.uint8)
        self.s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def needs(self):
        M, d_in, d_out, K = self.sizes
        p = lambda v: ctypes.c_void_p(v.data_ptr())  # noqa: E731
        z = ctypes.c_size_t
        lib, st, s = self.lib, p(self.st), self.s
        return {
            "topk_linear": least(lambda n: lib.larosa_topk_linear(
                p(self.x_rot), p(self.W), M, d_in, d_out, K, p(self.y), p(self.buf), z(n), st, 1, s), self.most),
            "rotate_topk_linear": least(lambda n: lib.larosa_rotate_topk_linear(
                p(self.x), None, p(self.W), M, d_in, d_out, K, p(self.y), p(self.buf), z(n), st, 1, s), self.most),
            "sparse_linear": least(lambda n: lib.larosa_sparse_linear(
                p(self.idx), p(self.val), M, K, p(self.W), d_in, d_out, p(self.y), p(self.buf), z(n), 1, st, s),
                self.most),
        }


@pytest.mark.parametrize("M,d_in,d_out,K", SHAPES)
def test_calls_on_wide_weights_need_nothing_for_the_4_bit_product(L, M, d_in, d_out, K):
    suits, other = Calls(M, d_in, d_out, K).needs(), Calls(M, d_in, d_out - 8, K).needs()
    for name in suits:
        assert suits[name] <= other[name] * 1.01 + 65536, (name, suits[name], other[name])


@pytest.mark.parametrize("M,d_in,d_out,K", SHAPES + [(1, 32768, 128, 20000), (5, 64, 7200, 64), (2, 4096, 4096, 2458)])
def test_workspace_bytes_serve_every_call(L, M, d_in, d_out, K):
    """The query's answer is enough for all of them, the 4-bit calls among them, and no byte
    past it is written."""
    ws_bytes = L.larosa_workspace_bytes(M, d_in, d_out, K)
    buf = torch.zeros(ws_bytes + 4096, dtype=torch.uint8, device="cuda")
    buf[ws_bytes:] = 0xA5
    ws = buf[:ws_bytes]
    W = sd.weights(d_in, d_out, 0.02, 6, torch.bfloat16, device="cuda")
    codes, scales = L.larosa_mx4_quantize(W, axis=0)
    idx, val = (a.cuda() for a in sd.index_values(M, d_in, K, 7))
    x = sd.activations(M, d_in, 8, torch.float32).cuda()
    st = status()
    calls = [lambda w: L.larosa_mx4_sparse_linear(idx, val, codes, scales, ws=w, dev_status=st),
             lambda w: L.larosa_mx4_topk_linear(x, codes, scales, K, ws=w, dev_status=st),
             lambda w: L.larosa_topk_linear(x, W, K, ws=w, dev_status=st),
             lambda w: L.larosa_sparse_linear(idx, val, W, ws=w, dev_status=st)]
    own = [call(L.Workspace()) for call in calls]
    for _ in range(2):  # one after the other on the same bytes
        for call, want in zip(calls, own):
            assert torch.equal(call(ws), want)
    assert L.larosa_check(st) == 0
    assert torch.all(buf[ws_bytes:] == 0xA5)
