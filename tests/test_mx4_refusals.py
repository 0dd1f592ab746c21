"""What the 4-bit and expert entry points refuse, on the host: no call here launches work."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
FAKE = P(0x10000)          # aligned, never dereferenced: validation fails first
MISALIGNED = P(0x10008)
BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def lib():
    from activation_sparsity_b200 import build_lib
    return ctypes.CDLL(build_lib.build())


def test_quantize_and_dequantize(lib):
    q, d = lib.larosa_mx4_quantize, lib.larosa_mx4_dequantize
    assert q(FAKE, 4, 64, 1, 7, FAKE, FAKE, None, None) == 4
    assert q(None, 4, 64, 1, BF16, FAKE, FAKE, None, None) == 1
    assert q(FAKE, 4, 64, 1, BF16, None, FAKE, None, None) == 1
    assert q(FAKE, 4, 64, 2, BF16, FAKE, FAKE, None, None) == 1
    assert q(FAKE, 0, 64, 1, BF16, FAKE, FAKE, None, None) == 2
    assert q(FAKE, 4, 0, 1, BF16, FAKE, FAKE, None, None) == 2
    assert q(FAKE, 4, 48, 1, BF16, FAKE, FAKE, None, None) == 3
    assert q(FAKE, 40, 64, 0, F32, FAKE, FAKE, None, None) == 3
    assert q(MISALIGNED, 4, 64, 1, BF16, FAKE, FAKE, None, None) == 3
    assert q(FAKE, 4, 64, 1, BF16, FAKE, MISALIGNED, None, None) == 3
    assert d(FAKE, FAKE, 4, 64, 1, 9, FAKE, None) == 4
    assert d(FAKE, None, 4, 64, 1, BF16, FAKE, None) == 1
    assert d(FAKE, FAKE, 4, 64, -1, BF16, FAKE, None) == 1
    assert d(FAKE, FAKE, -4, 64, 1, BF16, FAKE, None) == 2
    assert d(FAKE, FAKE, 4, 33, 1, BF16, FAKE, None) == 3
    assert d(FAKE, FAKE, 4, 64, 1, BF16, MISALIGNED, None) == 3


def test_sparse_and_topk_linear(lib):
    s, t = lib.larosa_mx4_sparse_linear, lib.larosa_mx4_topk_linear
    z = ctypes.c_size_t(1 << 20)
    assert s(FAKE, FAKE, 1, 4, None, FAKE, 64, 64, FAKE, FAKE, z, None, None) == 1
    assert s(None, FAKE, 1, 4, FAKE, FAKE, 64, 64, FAKE, FAKE, z, None, None) == 1
    assert s(FAKE, FAKE, 17, 4, FAKE, FAKE, 64, 64, FAKE, FAKE, z, None, None) == 2
    assert s(FAKE, FAKE, 1, 65, FAKE, FAKE, 64, 64, FAKE, FAKE, z, None, None) == 2
    assert s(FAKE, FAKE, 1, 4, FAKE, FAKE, 65536, 64, FAKE, FAKE, z, None, None) == 2
    assert s(FAKE, FAKE, 1, 4, FAKE, FAKE, 48, 64, FAKE, FAKE, z, None, None) == 3
    assert s(FAKE, FAKE, 1, 4, FAKE, FAKE, 64, 40, FAKE, FAKE, z, None, None) == 3
    assert s(FAKE, FAKE, 1, 4, MISALIGNED, FAKE, 64, 64, FAKE, FAKE, z, None, None) == 3
    assert s(FAKE, FAKE, 1, 4, FAKE, FAKE, 64, 64, MISALIGNED, FAKE, z, None, None) == 3
    assert s(FAKE, FAKE, 1, 4, FAKE, FAKE, 64, 64, FAKE, None, z, None, None) in (5, 6)  # 5: no device to plan for
    assert t(None, FAKE, FAKE, 1, 64, 64, 4, FAKE, FAKE, z, None, None) == 1
    assert t(FAKE, FAKE, FAKE, 0, 64, 64, 4, FAKE, FAKE, z, None, None) == 2
    assert t(FAKE, FAKE, FAKE, 1, 64, 72, 4, FAKE, FAKE, z, None, None) == 3


def test_linear(lib):
    need = lib.larosa_mx4_linear_workspace_bytes
    need.restype = ctypes.c_size_t

    def call(xc=FAKE, xs=FAKE, wc=FAKE, ws_=FAKE, M=4, d_in=64, d_out=64, y=FAKE, ws=FAKE, nb=1 << 24, dt=F32):
        return lib.larosa_mx4_linear(xc, xs, wc, ws_, M, d_in, d_out, y, ws, ctypes.c_size_t(nb), None, dt, None)

    assert call(dt=5) == 4
    assert call(xs=None) == 1 and call(wc=None) == 1 and call(y=None) == 1
    assert call(M=0) == 2 and call(M=1 << 21) == 2 and call(d_in=65536) == 2 and call(d_out=0) == 2
    assert call(d_in=72) == 3 and call(xc=MISALIGNED) == 3 and call(ws_=MISALIGNED) == 3 and call(y=MISALIGNED) == 3
    assert call(ws=None) == 6 and call(ws=MISALIGNED) == 6
    assert call(M=300, nb=need(300, 64, 64) - 1) == 6
    assert need(300, 64, 64) > need(4, 64, 64) > 0 and need(4, 72, 64) == 0


def test_moe_layer(lib):
    f = lib.larosa_moe_layer
    lib.larosa_moe_workspace_bytes.restype = ctypes.c_size_t

    def call(x=FAKE, wr=FAKE, gu=FAKE, sg=None, dn=FAKE, sd=None, M=2, d=64, ff=96, E=8, k=2, re=1, y=FAKE, ws=FAKE,
             nb=1 << 30, dt=BF16):
        return f(x, wr, gu, sg, dn, sd, M, d, ff, E, k, re, y, None, None, ws, ctypes.c_size_t(nb), None, dt, None)

    assert call(dt=3) == 4
    assert call(x=None) == 1 and call(wr=None) == 1 and call(dn=None) == 1 and call(y=None) == 1
    assert call(sg=FAKE) == 1 and call(sd=FAKE) == 1 and call(re=2) == 1
    assert call(M=0) == 2 and call(M=17) == 2 and call(d=0) == 2 and call(d=32776) == 2 and call(ff=32776) == 2
    assert call(E=0) == 2 and call(E=513) == 2 and call(k=0) == 2 and call(k=9) == 2 and call(E=64, k=17) == 2
    assert call(d=60) == 3 and call(ff=100) == 3 and call(sg=FAKE, sd=FAKE, d=72) == 3
    assert call(gu=MISALIGNED) == 3 and call(y=MISALIGNED) == 3
    need = lib.larosa_moe_workspace_bytes(2, 64, 96, 8, 2)
    assert need > 0 and lib.larosa_moe_workspace_bytes(2, 64, 96, 8, 9) == 0
    assert call(ws=None) == 6 and call(nb=need - 1) == 6 and call(ws=MISALIGNED) == 6


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import activation_sparsity_b200 as L
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        L.larosa_mx4_quantize(x)
    with pytest.raises(ValueError):
        L.larosa_mx4_dequantize(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    from activation_sparsity_b200 import larosa
    with pytest.raises(ValueError):
        larosa._mx4_shapes((4, 48), 1)
    with pytest.raises(ValueError):
        larosa._mx4_shapes((40, 64), 0)
    with pytest.raises(ValueError):
        larosa._mx4_shapes((4, 64), 2)
    with pytest.raises(ValueError):
        larosa._mx4_shapes((64,), 1)
    assert larosa._mx4_shapes((2, 64, 96), 0) == ((2, 64, 48), (2, 2, 96), 128, 96)
    assert larosa._mx4_shapes((2, 3, 96), 1) == ((2, 3, 48), (2, 3, 3), 6, 96)
