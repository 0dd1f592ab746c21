"""Forms of the 4-bit products that only wide weights or many tokens reach.

* up to four tokens, d_out > 6912: a CTA of the sparse product takes 256 columns, two
  warps abreast (6912 and less: 128);
* the 4-bit linear from 65 tokens on, tiles that end inside y: nothing behind
  the last row or column is written;
* the 4-bit linear on two streams at once.
"""
import numpy as np
import pytest
import torch

import oracle
import synthdata as sd
from tests import test_gpu_mx4_linear as linear
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


WIDTHS = [6880, 6912, 6944, 7200, 7424]


@pytest.mark.parametrize("d_out", WIDTHS)
@pytest.mark.parametrize("M,d_in,K", [(1, 32, 20), (1, 256, 150), (1, 2048, 1229), (2, 96, 96), (3, 256, 100),
                                      (4, 1024, 40)])
def test_sparse_linear(L, M, d_in, d_out, K):
    codes, scales, W = weight(L, d_in, d_out, 400 + d_in)
    idx, val = sd.index_values(M, d_in, K, 401 + K)
    st = status()
    y = L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales, dev_status=st)
    assert L.larosa_check(st) == 0
    check_y(f64(y), idx.numpy(), f64(val), W)
    assert torch.equal(y, L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales))


@pytest.mark.parametrize("d_out", WIDTHS)
@pytest.mark.parametrize("M,d_in,K", [(1, 256, 150), (1, 1024, 1024), (2, 64, 30), (4, 512, 307)])
def test_topk_linear(L, M, d_in, d_out, K):
    codes, scales, W = weight(L, d_in, d_out, 410 + d_in)
    x = sd.activations(M, d_in, 411, torch.float32)
    st = status()
    y = L.larosa_mx4_topk_linear(x.cuda(), codes, scales, K, dev_status=st)
    assert L.larosa_check(st) == 0
    idx, val = oracle.topk(f64(x), K)
    check_y(f64(y), idx, val, W)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,d_in,d_out", [(65, 256, 264), (100, 288, 1003), (190, 96, 20008), (193, 512, 4097),
                                          (257, 64, 333), (700, 128, 10248), (130, 256, 40)])
def test_what_lies_behind_y_is_left_alone(L, M, d_in, d_out, out):
    xc, xs, x = linear.matrix(M, d_in, 420 + M)
    wc, ws, w = linear.matrix(d_out, d_in, 421 + M)
    buf = torch.full((M * d_out + 40000,), 7.0, dtype=out, device="cuda")
    for start in (0, 16 // out.itemsize * 3):
        buf.fill_(7.0)
        y = buf[start:start + M * d_out].view(M, d_out)
        L.larosa_mx4_linear(xc, xs, wc, ws, dtype=out, y=y)
        assert torch.all(buf[:start] == 7.0) and torch.all(buf[start + M * d_out:] == 7.0)
        linear.check(f64(y), x, w, out)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_linear_on_two_streams(L, M):
    """Calls in flight at the same time, each on its stream's own workspace, give what they
    give alone."""
    sets = []
    for seed in (430, 440):
        xc, xs, _ = linear.matrix(M, 1024, seed)
        wc, ws, _ = linear.matrix(2048, 1024, seed + 1)
        sets.append((xc, xs, wc, ws))
    want = [L.larosa_mx4_linear(*s) for s in sets]
    torch.cuda.synchronize()
    ys = []
    for s in sets:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ys.append([L.larosa_mx4_linear(*s) for _ in range(6)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for w, group in zip(want, ys) for y in group)
