"""The 4-bit operators and the expert layer together, as a served model runs
them: a prompt through a 4-bit product, decoded tokens through the rotation, the
Top-K and a 4-bit W_rot, and the expert layer, on one workspace and one stream,
eagerly and captured into a graph; and what surrounds such a run: two streams,
the debug checks, wait limits too short for any kernel.

Every stage is compared with the fp64 oracle on the values that the GPU's stage
before it handed over, with the bounds that the stages' own tests derive.
"""
import numpy as np
import pytest
import torch

import oracle
import synthdata as sd
from tests import test_gpu_moe as moe
from tests import test_gpu_mx4 as mx4
from tests import test_gpu_mx4_linear as linear
from tests.test_gpu_mx4 import unpack
from tests.test_gpu_parity import f64, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


class Model:
    """prompt [T, d] -> 4-bit product -> the last M tokens -> rotate, Top-K, 4-bit
    W_rot -> experts (4-bit), all on one workspace."""

    def __init__(self, L, T, M, d, K, experts):
        self.L, self.M, self.K = L, M, K
        self.prompt = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
        Wt = sd.weights(d, d, d ** -0.5, 200, torch.bfloat16, device="cuda")
        self.wt = L.larosa_mx4_quantize(Wt, axis=1)
        self.Qt = sd.orthogonal(d, 201).t().contiguous().to(torch.bfloat16).cuda()
        W = sd.weights(d, d, d ** -0.5, 202, torch.bfloat16, device="cuda")
        self.w = L.larosa_mx4_quantize(L.larosa_prepare_weights(self.Qt, W), axis=0)
        self.layer = moe.Layer(L, M, d, 2 * d, 8, experts, torch.bfloat16, 203)
        self.ws, self.st = L.Workspace(), status()

    def run(self):
        L, ws, st = self.L, self.ws, self.st
        self.p4 = L.larosa_mx4_quantize(self.prompt, dev_status=st)
        self.hidden = L.larosa_mx4_linear(*self.p4, *self.wt, dtype=torch.bfloat16, ws=ws, dev_status=st)
        self.rot = L.larosa_rotate(self.hidden[-self.M:], self.Qt)
        self.y = L.larosa_mx4_topk_linear(self.rot, *self.w, self.K, ws=ws, dev_status=st)
        self.layer.x.copy_(self.y)
        self.out = self.layer.run(L, 2, ws=ws, dev_status=st)

    def check(self):
        assert self.L.larosa_check(self.st) == 0
        codes, scales = oracle.mx4_quantize(f64(self.prompt), 1)
        assert np.array_equal(unpack(self.p4[0]), codes) and np.array_equal(self.p4[1].cpu().numpy(), scales)
        wt = oracle.mx4_values(unpack(self.wt[0]), self.wt[1].cpu().numpy(), 1)
        linear.check(f64(self.hidden), oracle.mx4_values(codes, scales, 1), wt, torch.bfloat16)
        idx, val = oracle.topk(f64(self.rot), self.K)
        mx4.check_y(f64(self.y), idx, val, oracle.mx4_values(unpack(self.w[0]), self.w[1].cpu().numpy(), 0))
        self.layer.check(self.out, 2)


@pytest.mark.parametrize("T,M,experts", [(3, 1, "plain"), (70, 2, "mx4"), (200, 7, "mx4"), (129, 16, "plain")])
def test_prompt_decode_and_experts(L, T, M, experts):
    m = Model(L, T, M, 256, 154, experts)
    m.prompt.copy_(sd.activations(T, 256, 210 + T))
    m.run()
    m.check()


@pytest.mark.parametrize("T,M", [(2, 1), (70, 6)])
def test_the_whole_run_captured_and_replayed(L, T, M):
    m = Model(L, T, M, 256, 154, "mx4")
    m.prompt.copy_(sd.activations(T, 256, 220))
    m.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.run()
    for seed in (221, 222, 223):
        m.prompt.copy_(sd.activations(T, 256, seed))
        g.replay()
        torch.cuda.synchronize()
        m.check()


def test_expert_layers_on_two_streams(L):
    """Calls that are in flight at the same time, each on its stream's own
    workspace, give what they give alone."""
    layers = [moe.Layer(L, 4, 256, 512, 16, kind, torch.bfloat16, 230) for kind in ("plain", "mx4")]
    want = [layer.run(L, 4) for layer in layers]
    torch.cuda.synchronize()
    outs = []
    for layer in layers:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs.append([layer.run(L, 4) for _ in range(6)])
    torch.cuda.synchronize()
    for w, group in zip(want, outs):
        assert all(torch.equal(a, b) for out in group for a, b in zip(w, out))


@pytest.mark.parametrize("E,k", [(40, 6), (128, 4), (200, 6)])
def test_close_scores_keep_their_order(L, E, k):
    """Scores that differ by 2^-26 of themselves, some of them equal."""
    layer = moe.Layer(L, 1, 64, 64, E, "plain", torch.float32, 240)
    layer.x.fill_(1.0)
    layer.wr.fill_(0.25)
    step = torch.arange(E, device="cuda") * 7 % 5  # 0 ... 4, each many times
    layer.wr[:, 63] = 0.25 + step * 2.0 ** -22
    for renormalize in (True, False):
        out = layer.run(L, k, renormalize=renormalize)
        order = sorted(range(E), key=lambda e: (-int(step[e]), e))
        assert out[1][0].tolist() == order[:k]
        layer.check(out, k, renormalize)


def test_debug_checks_see_the_lists_of_4_bit_calls(L):
    codes, scales, W = mx4.weight(L, 256, 128, 250)
    previous = L.larosa_set_debug(True)
    try:
        st = status()
        idx = torch.tensor([[3, 9, 3, 40]], dtype=torch.int32, device="cuda")
        L.larosa_mx4_sparse_linear(idx, torch.ones(1, 4, device="cuda"), codes, scales, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == L.LAROSA_DEV_LIST
        st.zero_()
        x = sd.activations(3, 256, 251, torch.float32)
        y = L.larosa_mx4_topk_linear(x.cuda(), codes, scales, 100, dev_status=st)
        assert L.larosa_check(st) == 0
        idx, val = oracle.topk(f64(x), 100)
        mx4.check_y(f64(y), idx, val, W)
    finally:
        L.larosa_set_debug(previous)


@pytest.mark.parametrize("M", [3, 40, 200])
def test_a_wait_limit_too_short_for_the_product(L, M):
    """Every wait of the 4-bit product ends at the limit, and the next call with
    the usual one is right: either the call was in time or it says that it was
    not."""
    xc, xs, x = linear.matrix(M, 8192, 260)
    wc, ws, w = linear.matrix(384, 8192, 261)
    want = L.larosa_mx4_linear(xc, xs, wc, ws)
    torch.cuda.synchronize()
    st = status()
    previous = L.larosa_set_wait_limit_ns(1000)
    try:
        y = L.larosa_mx4_linear(xc, xs, wc, ws, dev_status=st)
    finally:
        L.larosa_set_wait_limit_ns(previous)
    torch.cuda.synchronize()
    flags = int(st.item())
    assert flags == L.LAROSA_DEV_TIMEOUT or (flags == 0 and torch.equal(y, want))
    st.zero_()
    again = L.larosa_mx4_linear(xc, xs, wc, ws, dev_status=st)
    assert L.larosa_check(st) == 0 and torch.equal(again, want)
    linear.check(f64(again), x, w, torch.float32)


@pytest.mark.parametrize("axis", [0, 1])
def test_values_go_to_any_16_byte_boundary(L, axis):
    """Outputs that start 16, 32 and 48 bytes into an allocation; what lies
    around them stays."""
    x = sd.activations(64, 160, 270, torch.float32).cuda()
    codes, scales = L.larosa_mx4_quantize(x, axis=axis)
    want = L.larosa_mx4_dequantize(codes, scales, axis=axis)
    for dtype, step in ((torch.float32, 4), (torch.bfloat16, 8)):
        for k in (1, 2, 3):
            buf = torch.full((64 * 160 + 64,), 7.0, dtype=dtype, device="cuda")
            out = buf[k * step:k * step + 64 * 160].view(64, 160)
            L.larosa_mx4_dequantize(codes, scales, axis=axis, out=out)
            assert torch.equal(out, want.to(dtype))
            rest = torch.cat([buf[:k * step], buf[k * step + 64 * 160:]])
            assert torch.all(rest == 7.0)
