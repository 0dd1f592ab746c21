"""The expert layer against the fp64 oracle.

Scores are fp64 sums of exact products, so the chosen experts equal the
oracle's (the test inputs hold no scores closer than fp64 rounding except
exact ties).  Gates: exp of an fp32 difference (relative error 2^-24 of the
difference, at most 100, plus 2 ulp of exp), a sum of up to E and a division:
(E + 110) 2^-23 relative.

y: with n additions per sum, each losing at most 2^-23 of the running
magnitude (the tensor cores truncate), and G = sum |x W_gate|, V = sum
|x W_up|, the errors of g and u are dg = n_d 2^-23 G and du = n_d 2^-23 V
(n_d = d + 40); |silu'| <= 1.1, so dh <= 1.1 dg |u| + |silu(g)| du + 1.1 dg du
+ 8 2^-23 |h| (exp, division, products, the operand's pieces); and |error of y| <= sum_s
gate (sum_j (dh + (f + 40) 2^-23 |h|) |W_d| + (n_gate + k) 2^-23 sum_j |h W_d|).
A 4-bit expert's pieces add 2^-50 of the block's largest operand times the
block's largest weight, below 2^-30 of the bound's other terms here.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_mx4 import unpack
from tests.test_gpu_parity import f64, status

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


class Layer:
    """Inputs on the device and their values in fp64."""

    def __init__(self, L, M, d, f, E, experts, dtype, seed, same_router=False):
        rng = np.random.default_rng(seed)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()  # noqa: E731
        self.x = t(rng.standard_normal((M, d)))
        self.wr = t(np.zeros((E, d)) if same_router else rng.standard_normal((E, d)) * d ** -0.5)
        gu = t(rng.standard_normal((E, d, 2 * f)) * d ** -0.5)
        dn = t(rng.standard_normal((E, f, d)) * f ** -0.5)
        self.sg = self.sd = None
        if experts == "mx4":
            gu, self.sg = L.larosa_mx4_quantize(gu, axis=0)
            dn, self.sd = L.larosa_mx4_quantize(dn, axis=0)
            self.gu64 = np.stack([oracle.mx4_values(unpack(gu[e]), self.sg[e].cpu().numpy(), 0) for e in range(E)])
            self.dn64 = np.stack([oracle.mx4_values(unpack(dn[e]), self.sd[e].cpu().numpy(), 0) for e in range(E)])
        else:
            self.gu64, self.dn64 = f64(gu), f64(dn)
        self.gu, self.dn = gu, dn

    def run(self, L, k, renormalize=True, **kw):
        return L.larosa_moe_layer(self.x, self.wr, self.gu, self.dn, k, S_gu=self.sg, S_d=self.sd,
                                  renormalize=renormalize, **kw)

    def check(self, out, k, renormalize=True):
        y, idx, gate = (f64(o) for o in out)
        x, wr = f64(self.x), f64(self.wr)
        want, wi, wg = oracle.moe_layer(x, wr, self.gu64, self.dn64, k, renormalize)
        E, d, f = self.gu64.shape[0], x.shape[1], self.dn64.shape[1]
        assert np.array_equal(idx.astype(np.int64), wi)
        n_gate = E + 110
        assert np.all(np.abs(gate - wg) <= n_gate * U * wg)
        for m in range(x.shape[0]):
            bound = np.zeros(d)
            for s in range(k):
                gu, dn = self.gu64[wi[m, s]], self.dn64[wi[m, s]]
                a, mag = x[m] @ gu, np.abs(x[m]) @ np.abs(gu)
                g, u = a[:f], a[f:]
                dg, du = (d + 40) * U * mag[:f], (d + 40) * U * mag[f:]
                silu = g / (1 + np.exp(-g))
                h = np.abs(silu * u)
                dh = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + 8 * U * h
                bound += wg[m, s] * ((dh + (f + 40) * U * h) @ np.abs(dn) + (n_gate + k) * U * (h @ np.abs(dn)))
            err = np.abs(y[m] - want[m])
            assert np.all(err <= bound * (1 + 2.0 ** -30) + 1e-37), np.max(err / (bound + 1e-37))


CASES = [  # M, d, f, E, k
    (1, 8, 8, 1, 1), (1, 64, 32, 4, 2), (2, 256, 64, 8, 8), (3, 200, 72, 5, 2), (1, 256, 512, 8, 2),
    (5, 96, 1408, 60, 4), (16, 128, 96, 2, 1), (16, 64, 64, 3, 3), (9, 32, 32, 16, 2), (8, 512, 256, 512, 16),
    (13, 1024, 136, 33, 7), (4, 40, 4096, 6, 2), (1, 4096, 64, 16, 2), (16, 256, 128, 128, 8),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d,f,E,k", CASES)
def test_layer(L, dtype, M, d, f, E, k):
    layer = Layer(L, M, d, f, E, "plain", dtype, M + d + f)
    st = status()
    for renormalize in (True, False):
        out = layer.run(L, k, renormalize, dev_status=st)
        assert L.larosa_check(st) == 0
        layer.check(out, k, renormalize)
        again = layer.run(L, k, renormalize, dev_status=st)
        assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d,f,E,k", [(1, 32, 32, 1, 1), (1, 256, 512, 8, 2), (3, 96, 160, 5, 3), (16, 64, 96, 2, 2),
                                       (7, 1024, 224, 40, 4), (16, 288, 128, 64, 8), (2, 4096, 64, 4, 1)])
def test_layer_with_4_bit_experts(L, dtype, M, d, f, E, k):
    layer = Layer(L, M, d, f, E, "mx4", dtype, M + d + f)
    st = status()
    out = layer.run(L, k, dev_status=st)
    assert L.larosa_check(st) == 0
    layer.check(out, k)
    assert all(torch.equal(a, b) for a, b in zip(out, layer.run(L, k)))


@pytest.mark.parametrize("M,k", [(1, 3), (16, 4)])
def test_equal_scores_take_the_lowest_experts(L, M, k):
    layer = Layer(L, M, 64, 64, 9, "plain", torch.bfloat16, 3, same_router=True)
    out = layer.run(L, k)
    assert out[1].cpu().tolist() == [list(range(k))] * M
    layer.check(out, k)


def test_scores_closer_than_fp32_rounding_are_told_apart(L):
    """Two experts whose scores differ in the 30th bit."""
    layer = Layer(L, 1, 64, 64, 2, "plain", torch.float32, 4)
    layer.x.fill_(1.0)
    layer.wr.fill_(0.25)
    layer.wr[1, 63] = 0.25 + 2.0 ** -25  # scores 16 and 16 + 2^-25
    out = layer.run(L, 1)
    assert out[1].item() == 1
    layer.check(out, 1)


def test_all_tokens_on_one_expert(L):
    layer = Layer(L, 16, 128, 256, 4, "plain", torch.bfloat16, 5)
    layer.wr.zero_()
    layer.wr[2] = layer.x.float().mean(0).to(layer.wr.dtype) * 100
    layer.x.copy_(layer.x[:1].expand(16, -1).contiguous())
    out = layer.run(L, 1)
    layer.check(out, 1)
    assert len(set(out[1].flatten().tolist())) == 1


def test_nonfinite_scores_are_reported(L):
    layer = Layer(L, 3, 64, 64, 6, "plain", torch.float32, 6)
    layer.x[1, 5] = float("nan")
    st = status()
    y, idx, gate = layer.run(L, 2, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & L.LAROSA_DEV_NONFINITE
    assert 0 <= int(idx.min()) and int(idx.max()) < 6
    layer.x[1, 5] = 1.0
    st.zero_()
    layer.check(layer.run(L, 2, dev_status=st), 2)  # the workspace still serves the next call
    assert L.larosa_check(st) == 0


def test_one_workspace_for_calls_of_many_kinds_and_sizes(L):
    ws = L.Workspace()
    st = status()
    import synthdata as sd
    for size in ((1, 256, 512, 8, 2), (16, 64, 64, 3, 3), (1, 64, 32, 4, 2)):
        M, d, f, E, k = size
        for experts in ("plain", "mx4"):
            layer = Layer(L, M, d, f, E, experts, torch.bfloat16, 7)
            layer.check(layer.run(L, k, ws=ws, dev_status=st), k)
        x = sd.activations(1, 512, 8, torch.bfloat16)
        Qt = sd.orthogonal(512, 9).float().t().contiguous().to(torch.bfloat16).cuda()
        W = sd.weights(512, 256, 0.02, 10, torch.bfloat16).cuda()
        got = L.larosa_rotate_topk_linear(x.cuda(), Qt, W, 300, ws=ws, dev_status=st)
        want = L.larosa_rotate_topk_linear(x.cuda(), Qt, W, 300, dev_status=st)
        assert torch.equal(got, want)
    assert L.larosa_check(st) == 0


def test_captured_and_replayed_with_new_inputs(L):
    layer = Layer(L, 4, 256, 128, 16, "plain", torch.bfloat16, 11)
    ws = L.Workspace()
    layer.run(L, 4, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.run(L, 4, ws=ws)
    for seed in (12, 13, 14):
        layer.x.copy_(torch.randn(4, 256, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        layer.check(out, 4)


def test_optional_outputs_and_the_wait_limit(L):
    """idx and gate may be missing; a limit no call can keep reports a timeout
    and leaves the context usable."""
    layer = Layer(L, 2, 256, 128, 8, "plain", torch.bfloat16, 15)
    want = layer.run(L, 2)
    from activation_sparsity_b200 import larosa
    lib = larosa.raw_library()
    ws = L.Workspace()
    buf = ws.get_moe(2, 256, 128, 8, 2)
    y = torch.zeros(2, 256, device="cuda")
    st = status()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    args = (p(layer.x), p(layer.wr), p(layer.gu), None, p(layer.dn), None, 2, 256, 128, 8, 2, 1, p(y), None, None,
            p(buf), buf.numel(), p(st), 1, stream)
    assert lib.larosa_moe_layer(*args) == 0
    assert L.larosa_check(st) == 0 and torch.equal(y, want[0])
    # an arrival counter that starts at -1 never reaches the number of CTAs
    buf[:4].view(torch.int32).fill_(-1)
    previous = L.larosa_set_wait_limit_ns(2_000_000)
    try:
        assert lib.larosa_moe_layer(*args) == 0
    finally:
        L.larosa_set_wait_limit_ns(previous)
    torch.cuda.synchronize()
    assert int(st.item()) == L.LAROSA_DEV_TIMEOUT
    buf.zero_()
    st.zero_()
    y.zero_()
    assert lib.larosa_moe_layer(*args) == 0
    assert L.larosa_check(st) == 0 and torch.equal(y, want[0])
