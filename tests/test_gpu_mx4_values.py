"""How coefficients and operands are held by the 4-bit products, and what values
that are not numbers do there.

A coefficient is two f16 pieces over a power of two: p0 is its first 11 bits
(rounded), p1 the rest.  In units of its last fp32 bit a value is an integer
below 2^24, p0 a multiple of 2^13 of it and the rest an integer of at most 2^12,
of which f16 holds the odd ones only up to 2^11: a value is held to 2^-23 of
itself.  Entries far below the largest of their block meet f16's smallest step,
2^-24: after the scaling (largest in [2^14, 2^15)) and the 2^-11 of the second
piece that is an error of 2^-36, 2^-50 of the largest.
"""
import numpy as np
import pytest
import torch

import oracle
import synthdata as sd
from tests.test_gpu_mx4 import check_y, unpack, weight
from tests.test_gpu_parity import f64, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


def unit_weight(d):
    """The d x d identity in 4 bits: code 2 (1.0) on the diagonal, scales of one."""
    codes = np.zeros((d, d // 2), dtype=np.uint8)
    i = np.arange(d)
    codes[i, i // 2] = np.where(i % 2, 0x20, 0x02)
    return torch.from_numpy(codes).cuda(), torch.full((d // 32, d), 127, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("topk", [False, True])
@pytest.mark.parametrize("M", [1, 3, 6, 16])
def test_a_coefficient_is_held_to_2_to_the_minus_23(L, M, topk):
    """Through the identity, y is the coefficients as they are held."""
    d = 512
    rng = np.random.default_rng(M)
    v = (rng.integers(1 << 23, 1 << 24, (M, d)) | 1) * np.exp2(rng.integers(-40, -20, (M, d)))
    val = torch.from_numpy(v * rng.choice([-1.0, 1.0], (M, d))).float()
    codes, scales = unit_weight(d)
    if topk:
        y = L.larosa_mx4_topk_linear(val.cuda(), codes, scales, d)
    else:
        idx = torch.arange(d, dtype=torch.int32).repeat(M, 1)
        y = L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales)
    want = f64(val)
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -23 * np.abs(want))


@pytest.mark.parametrize("M", [1, 4, 9])
def test_entries_far_below_their_block(L, M):
    """Entries 2^-1 ... 2^-60 of their block's largest, and blocks down to fp32's smallest values."""
    d = 1024
    rng = np.random.default_rng(20 + M)
    v = rng.uniform(1, 2, (M, d)) * np.exp2(rng.integers(-60, 0, (M, d)).astype(np.float64))
    v[:, ::32] = 1.5
    top = np.repeat(rng.integers(-120, 90, (M, d // 32)), 32, axis=1)
    val = torch.from_numpy(np.ldexp(v, top)).float()
    codes, scales = unit_weight(d)
    idx = torch.arange(d, dtype=torch.int32).repeat(M, 1)
    y = f64(L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales))
    want = f64(val)
    largest = np.repeat(np.abs(want).reshape(M, -1, 32).max(axis=2), 32, axis=1)
    # the scale stops at 2^-100: smaller blocks keep the absolute error 2^-150 of that one
    bound = 2.0 ** -23 * np.abs(want) + 2.0 ** -50 * largest + 2.0 ** -149
    assert np.all(np.abs(y - want) <= bound)


@pytest.mark.parametrize("M", [1, 3, 7, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_coefficient_that_is_no_number_reaches_its_token_alone(L, M, bad):
    codes, scales, W = weight(L, 256, 96, 30)
    idx, val = sd.index_values(M, 256, 100, 31)
    val[M // 2, 40] = bad
    y = f64(L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales))
    others = [m for m in range(M) if m != M // 2]
    assert not np.any(np.isfinite(y[M // 2]))
    check_y(y[others], idx.numpy()[others], f64(val)[others], W)


@pytest.mark.parametrize("M", [2, 6])
def test_a_nan_block_reaches_every_token_of_a_call_that_reads_it(L, M):
    """Token 0 keeps a row of the block whose scale is NaN in column 5, the others none: the
    column is NaN for all of them, every other column right for all."""
    codes, scales, W = weight(L, 128, 64, 32)
    scales[2, 5] = 255
    idx = torch.arange(32, dtype=torch.int32).repeat(M, 1)
    idx[0] += 64
    val = torch.from_numpy(np.random.default_rng(33).standard_normal((M, 32))).float()
    y = f64(L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales))
    assert np.all(np.isnan(y[:, 5]))
    W[:, 5] = 0.0
    y[:, 5] = 0.0
    check_y(y, idx.numpy(), f64(val), W)
    y = L.larosa_mx4_sparse_linear(idx[1:].contiguous().cuda(), val[1:].contiguous().cuda(), codes, scales)
    assert not torch.isnan(y).any()  # alone they never read it


# ---------------------------------------------------------------- expert layer

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("M,d,f,E,k", [(2, 96, 160, 3, 2), (16, 288, 64, 4, 2), (7, 64, 512, 40, 6)])
def test_4_bit_experts_with_inputs_spread_inside_a_block(L, dtype, renormalize, M, d, f, E, k):
    """x from 2^-40 to 1 inside every block, up columns from 2^-30 to 1, so that h spreads too.

    With the errors of tests/test_gpu_moe.py: x is held to 2^-23 of itself and 2^-50 of its
    block's largest, which adds tx = 2^-50 sum_blocks max|x| sum_block |w| to a sum's error; h
    likewise, th = 2^-50 sum_blocks max|h| sum_block |w|.
    """
    from tests.test_gpu_moe import U, Layer
    layer = Layer(L, M, d, f, E, "mx4", dtype, 300 + d)
    rng = np.random.default_rng(301 + d)
    x = rng.standard_normal((M, d)) * np.exp2(rng.integers(-40, 1, (M, d)).astype(np.float64))
    layer.x.copy_(torch.from_numpy(x))
    # the scale bytes of the up columns, lowered by 0 ... 30
    low = rng.integers(0, 31, f)
    layer.sg[:, :, f:] -= torch.from_numpy(low).to(torch.uint8).cuda()
    layer.gu64 = np.stack([oracle.mx4_values(unpack(layer.gu[e]), layer.sg[e].cpu().numpy(), 0) for e in range(E)])
    st = status()
    out = layer.run(L, k, renormalize, dev_status=st)
    assert L.larosa_check(st) == 0
    y, idx, gate = (f64(o) for o in out)
    x64 = f64(layer.x)
    want, wi, wg = oracle.moe_layer(x64, f64(layer.wr), layer.gu64, layer.dn64, k, renormalize)
    assert np.array_equal(idx.astype(np.int64), wi)
    n_gate = E + 110
    assert np.all(np.abs(gate - wg) <= n_gate * U * wg)

    def tail(v, w):
        b = np.abs(v).reshape(-1, 32).max(axis=1)
        return 2.0 ** -50 * (b @ np.abs(w).reshape(len(b), 32, -1).sum(axis=1))

    for m in range(M):
        bound = np.zeros(d)
        for s in range(k):
            gu, dn = layer.gu64[wi[m, s]], layer.dn64[wi[m, s]]
            a, mag = x64[m] @ gu, np.abs(x64[m]) @ np.abs(gu)
            err = (d + 42) * U * mag + tail(x64[m], gu)  # two more: x and its pieces' sum
            g, u, dg, du = a[:f], a[f:], err[:f], err[f:]
            silu = g / (1 + np.exp(-g))
            h = silu * u
            dh = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + 10 * U * np.abs(h)
            over = dh @ np.abs(dn) + tail(np.abs(h) + dh, dn)
            bound += wg[m, s] * (over + (f + 42 + n_gate + k) * U * ((np.abs(h) + dh) @ np.abs(dn)))
        e = np.abs(y[m] - want[m])
        assert np.all(e <= bound * (1 + 2.0 ** -20) + 1e-37), np.max(e / (bound + 1e-37))
    again = layer.run(L, k, renormalize)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
