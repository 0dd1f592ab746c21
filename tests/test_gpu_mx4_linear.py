"""The product of two 4-bit matrices (tcgen05, block scales) against the fp64
oracle.

Products of 4-bit values and powers of two are exact; an output is a sum of
d_in of them in fp32, each addition losing at most 2^-23 of the running
magnitude (the tensor cores truncate): |error| <= (d_in + 8) 2^-23 sum |x w|,
and half a bf16 step of the result for a bf16 output.  Scales differ from
block to block and row to row, so a scale taken from another block or row
shows at once.
"""
import numpy as np
import pytest
import torch

import oracle
import synthdata as sd
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


def matrix(rows, cols, seed, lo=117, hi=137):
    """Random codes and scales 2^-10 ... 2^10, and the values they stand for."""
    rng = np.random.default_rng(seed)
    codes = torch.from_numpy(rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8))
    scales = torch.from_numpy(rng.integers(lo, hi + 1, (rows, cols // 32), dtype=np.uint8))
    return codes.cuda(), scales.cuda(), oracle.mx4_values(unpack(codes), scales.numpy(), 1)


def check(got, x, w, out):
    want = x @ w.T
    bound = (x.shape[1] + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if out == torch.bfloat16:
        bound = bound + (np.abs(want) + bound) * torch.finfo(out).eps / 2
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / (bound + 1e-300))


SHAPES = [(1, 32, 1), (1, 256, 128), (16, 256, 128), (3, 64, 40), (5, 512, 129), (17, 1024, 257), (33, 96, 130),
          (64, 2048, 384), (1, 4096, 1000), (7, 11008, 520), (16, 32768, 128), (65, 544, 127), (100, 288, 640),
          (128, 4096, 256), (129, 1056, 200), (200, 640, 5000), (257, 800, 1111), (300, 8192, 260), (1000, 256, 20000),
          (640, 512, 3001), (2048, 96, 5000), (129, 64, 40000), (384, 1536, 10240), (2050, 288, 4104)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,d_in,d_out", SHAPES)
def test_linear(L, M, d_in, d_out, out):
    xc, xs, x = matrix(M, d_in, 1 + M)
    wc, ws, w = matrix(d_out, d_in, 2 + d_out)
    st = status()
    y = L.larosa_mx4_linear(xc, xs, wc, ws, dtype=out, dev_status=st)
    assert L.larosa_check(st) == 0
    assert y.dtype == out and y.shape == (M, d_out)
    check(f64(y), x, w, out)
    assert torch.equal(y, L.larosa_mx4_linear(xc, xs, wc, ws, dtype=out))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_each_block_meets_its_own_scale(L, M):
    """One nonzero block per row, a different one in every row: the product
    picks out single scales."""
    d_in, d_out = 1024, 256
    x = np.zeros((M, d_in))
    rng = np.random.default_rng(7)
    for m in range(M):
        b = m % (d_in // 32)
        x[m, 32 * b:32 * b + 32] = rng.integers(-6, 7, 32) * 2.0 ** (m % 9 - 4)
    xc, xs = L.larosa_mx4_quantize(torch.from_numpy(x).float().cuda())
    wc, ws, w = matrix(d_out, d_in, 8)
    got = f64(L.larosa_mx4_linear(xc, xs, wc, ws))
    xq = oracle.mx4_values(*oracle.mx4_quantize(x, 1), 1)
    check(got, xq, w, torch.float32)


def test_quantised_activations_and_weights(L):
    """The use: activations and a weight to 4 bits, then their product."""
    M, d_in, d_out = 37, 4096, 512
    x = sd.activations(M, d_in, 20, torch.bfloat16)
    W = sd.weights(d_out, d_in, 0.02, 21, torch.bfloat16)
    xc, xs = L.larosa_mx4_quantize(x.cuda())
    wc, ws = L.larosa_mx4_quantize(W.cuda())
    got = f64(L.larosa_mx4_linear(xc, xs, wc, ws))
    check(got, oracle.mx4_values(*oracle.mx4_quantize(f64(x), 1), 1),
          oracle.mx4_values(*oracle.mx4_quantize(f64(W), 1), 1), torch.float32)


@pytest.mark.parametrize("M", [2, 150])
def test_nan_scale_reaches_its_row_alone(L, M):
    xc, xs, x = matrix(M, 512, 30)
    wc, ws, w = matrix(192, 512, 31)
    xs[1, 3] = 255
    ws[100, 0] = 255
    y = L.larosa_mx4_linear(xc, xs, wc, ws)
    bad = torch.isnan(y)
    want = torch.zeros_like(bad)
    want[1, :] = True
    want[:, 100] = True
    assert torch.equal(bad, want)


def test_rows_past_the_matrix_are_left_alone(L):
    M, d_in, d_out = 5, 256, 100
    xc, xs, x = matrix(M, d_in, 40)
    wc, ws, w = matrix(d_out, d_in, 41)
    buf = torch.full((M + 3, d_out), 7.0, device="cuda")
    y = buf[:M]
    L.larosa_mx4_linear(xc, xs, wc, ws, y=y)
    assert torch.all(buf[M:] == 7.0)
    check(f64(y), x, w, torch.float32)


@pytest.mark.parametrize("M", [3, 200])
def test_captured_and_replayed(L, M):
    d_in, d_out = 1024, 384
    W = sd.weights(d_out, d_in, 0.02, 50, torch.bfloat16).cuda()
    wc, ws = L.larosa_mx4_quantize(W)
    w = oracle.mx4_values(unpack(wc), ws.cpu().numpy(), 1)
    x = torch.zeros(M, d_in, dtype=torch.bfloat16, device="cuda")
    L.larosa_mx4_linear(*L.larosa_mx4_quantize(x), wc, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = L.larosa_mx4_linear(*L.larosa_mx4_quantize(x), wc, ws, dtype=torch.bfloat16)
    for seed in (51, 52):
        xn = sd.activations(M, d_in, seed, torch.bfloat16)
        x.copy_(xn)
        g.replay()
        torch.cuda.synchronize()
        check(f64(y), oracle.mx4_values(*oracle.mx4_quantize(f64(xn), 1), 1), w, torch.bfloat16)
