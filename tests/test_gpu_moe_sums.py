"""The expert layer's sums: how they round, how they are dealt out, how long they get.

Rounding.  The sums of bf16 experts are fp32 sums: each addition rounds to
nearest, so errors lean to neither side.  Products of positive values show it:
additions that truncate would put every sum low.  x and the weights are
multiples of 2^-10 with eight significant bits in [1/8, 1), so a product is a multiple
of 2^-20 below 1 and sixteen of them sum exactly in fp32; what rounds is the
addition of these sums and the joins, at most n = d / 16 + 40 times, each by at
most 2^-24 of the result and without a preferred side: the mean of N independent
results' relative errors has a standard deviation below 2^-24 sqrt(n / (3 N)), and six of
those are the bound.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_moe import Layer
from tests.test_gpu_parity import f64, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


def eighths(rng, *shape):
    """bf16 values that are multiples of 2^-10 in [1/8, 1)."""
    v = rng.integers(128, 256, shape) * np.exp2(rng.integers(-10, -7, shape).astype(np.float64))
    return torch.from_numpy(v)


E, N = 8, 2048


@pytest.fixture(scope="module")
def unit():
    return torch.eye(N, dtype=torch.bfloat16, device="cuda").repeat(E, 1, 1)


def mean_error(L, x, gu, dn, want):
    """The mean relative error of y for one token on all E experts with equal gates."""
    wr = torch.zeros(E, x.shape[1], dtype=torch.bfloat16, device="cuda")
    y, idx, gate = L.larosa_moe_layer(x.cuda(), wr, gu, dn, E)
    assert torch.all(gate == 1.0 / E)
    return float(np.mean(f64(y)[0] / want - 1.0))


def test_gate_up_sums_of_bf16_experts_lean_to_neither_side(L, unit):
    """silu(64) = 64 in fp32 and Wd the identity: y is 64 times the up sums."""
    rng = np.random.default_rng(1)
    x = eighths(rng, 1, N)
    x[0, 0] = 1.0
    up = eighths(rng, E, N, N)
    gate = torch.zeros(E, N, N, dtype=torch.bfloat16)
    gate[:, 0] = 64.0
    gu = torch.cat([gate, up.to(torch.bfloat16)], dim=2).cuda()
    want = 64.0 * (x.cuda() @ up.cuda().mean(dim=0))[0].cpu().numpy()
    bias = mean_error(L, x.to(torch.bfloat16), gu, unit, want)
    assert abs(bias) <= 6 * 2.0 ** -24 * np.sqrt((N / 16 + 40) / (3 * N)), bias


def test_down_sums_of_bf16_experts_lean_to_neither_side(L):
    """x picks one row of the up weight: h is that row, known exactly."""
    rng = np.random.default_rng(2)
    x = torch.zeros(1, N, dtype=torch.float64)
    x[0, 0] = 1.0
    gu = torch.zeros(E, N, 2 * N, dtype=torch.float64)
    gu[:, 0, :N] = 64.0
    h = eighths(rng, E, N)
    gu[:, 0, N:] = h / 64.0
    dn = eighths(rng, E, N, N)
    want = (torch.bmm(h.view(E, 1, N).cuda(), dn.cuda()).mean(dim=0))[0].cpu().numpy()
    bias = mean_error(L, x.to(torch.bfloat16), gu.to(torch.bfloat16).cuda(), dn.to(torch.bfloat16).cuda(), want)
    assert abs(bias) <= 6 * 2.0 ** -24 * np.sqrt((N / 16 + 40) / (3 * N)), bias


# Units of 128 columns: some 20 groups times 128 gate and up tiles, or 44 (256 pairs on 24
# experts, more than eight to most) times 64, or 40 times 64 down tiles: more than
# the 2368 warps of the grid, whatever number of chunks is chosen, so that warps
# take further shares.  The last case has several chunks as well.
MANY = [(3, 64, 8192, 20, 16), (16, 64, 4096, 24, 16), (16, 8192, 64, 24, 16), (8, 8192, 96, 40, 16),
        (16, 608, 2080, 24, 16)]


@pytest.mark.parametrize("experts,dtype", [("mx4", torch.bfloat16), ("mx4", torch.float32),
                                           ("plain", torch.float32), ("plain", torch.bfloat16)])
@pytest.mark.parametrize("M,d,f,E,k", MANY)
def test_more_shares_than_warps(L, experts, dtype, M, d, f, E, k):
    layer = Layer(L, M, d, f, E, experts, dtype, 7 * M + d)
    st = status()
    ws = L.Workspace()
    out = layer.run(L, k, renormalize=M != 3, ws=ws, dev_status=st)
    assert L.larosa_check(st) == 0
    layer.check(out, k, renormalize=M != 3)
    for _ in range(3):
        again = layer.run(L, k, renormalize=M != 3, ws=ws, dev_status=st)
        assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("experts,dtype", [("mx4", torch.bfloat16), ("plain", torch.float32),
                                           ("plain", torch.bfloat16)])
@pytest.mark.parametrize("M,d,f,E,k", [(1, 32768, 64, 2, 1), (3, 32736, 32, 3, 2), (1, 64, 32768, 2, 2),
                                       (6, 32, 32736, 3, 1)])
def test_the_longest_rows(L, experts, dtype, M, d, f, E, k):
    layer = Layer(L, M, d, f, E, experts, dtype, 8 * M + d)
    st = status()
    out = layer.run(L, k, renormalize=False, dev_status=st)
    assert L.larosa_check(st) == 0
    layer.check(out, k, renormalize=False)
