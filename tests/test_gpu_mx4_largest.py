"""The 4-bit sparse products and the expert layer on the largest weights they take: offsets of
2^30 bytes within a weight (32768 x 65536), and of more than 2^32 into a stack of
experts.  The values of the rows and experts in question are worked out on the
device in 64 bits, from the format's definition.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_parity import f64, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


def values(codes, scales):
    """Rows of codes with the scale bytes of each row's block, in fp64."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], dim=-1).flatten(-2)
    return v * torch.exp2(scales.double() - 127)


@pytest.fixture(scope="module")
def weight():
    g = torch.Generator(device="cuda")
    g.manual_seed(600)
    d_in, d_out = 32768, 65536
    return (torch.randint(0, 256, (d_in, d_out // 2), generator=g, device="cuda", dtype=torch.uint8),
            torch.randint(117, 138, (d_in // 32, d_out), generator=g, device="cuda", dtype=torch.uint8))


@pytest.mark.parametrize("M,topk", [(1, False), (1, True), (3, False), (6, False), (16, False), (16, True)])
def test_sparse_products(L, weight, M, topk):
    codes, scales = weight
    d_in, K = codes.shape[0], 200
    rng = np.random.default_rng(601 + M)
    idx = np.stack([np.sort(np.append(rng.choice(d_in - 1, K - 1, replace=False), d_in - 1)) for _ in range(M)])
    val = rng.standard_normal((M, K)).astype(np.float32)
    st = status()
    if topk:
        x = np.zeros((M, d_in), dtype=np.float32)
        np.put_along_axis(x, idx, val, axis=1)
        y = L.larosa_mx4_topk_linear(torch.from_numpy(x).cuda(), codes, scales, K, dev_status=st)
    else:
        y = L.larosa_mx4_sparse_linear(torch.from_numpy(idx.astype(np.int32)).cuda(), torch.from_numpy(val).cuda(),
                                       codes, scales, dev_status=st)
    assert L.larosa_check(st) == 0
    for m in range(M):
        i = torch.from_numpy(idx[m]).cuda()
        W = values(codes[i], scales[i // 32]).cpu().numpy()
        # an addition per kept row, plus what the form adds (see tests/test_gpu_mx4.py)
        mag = np.abs(val[m].astype(np.float64)) @ np.abs(W)
        top = np.max(np.abs(val[m])) * np.max(np.abs(W))
        bound = (52 + d_in // 32) * 2.0 ** -23 * mag + K * 2.0 ** -50 * top
        err = np.abs(f64(y[m]) - val[m].astype(np.float64) @ W)
        assert np.all(err <= bound)


@pytest.mark.parametrize("experts", ["mx4", "bf16"])
def test_experts_far_into_their_stack(L, experts):
    d = f = 8192
    E, k = (72, 2) if experts == "mx4" else (20, 2)
    g = torch.Generator(device="cuda")
    g.manual_seed(610)
    x = torch.randn(1, d, generator=g, device="cuda").to(torch.bfloat16)
    wr = torch.zeros(E, d, dtype=torch.bfloat16, device="cuda")
    wr[E - 1], wr[E - 2] = x[0] / 4096, x[0] / 8192  # scores of about 2, 1 and 0
    if experts == "mx4":
        gu = torch.randint(0, 256, (E, d, f), generator=g, device="cuda", dtype=torch.uint8)
        dn = torch.randint(0, 256, (E, f, d // 2), generator=g, device="cuda", dtype=torch.uint8)
        sg = torch.randint(115, 121, (E, d // 32, 2 * f), generator=g, device="cuda", dtype=torch.uint8)
        s2 = torch.randint(115, 121, (E, f // 32, d), generator=g, device="cuda", dtype=torch.uint8)
        of = lambda c, s: values(c, s.repeat_interleave(32, dim=0))  # noqa: E731
        gu64, dn64 = (lambda e: of(gu[e], sg[e])), (lambda e: of(dn[e], s2[e]))
        assert gu.numel() > 1 << 32
    else:
        gu = torch.empty(E, d, 2 * f, dtype=torch.bfloat16, device="cuda").normal_(0, d ** -0.5, generator=g)
        dn = torch.empty(E, f, d, dtype=torch.bfloat16, device="cuda").normal_(0, f ** -0.5, generator=g)
        sg = s2 = None
        gu64, dn64 = (lambda e: gu[e].double()), (lambda e: dn[e].double())
        assert gu.numel() * 2 > 1 << 32
    st = status()
    y, idx, gate = L.larosa_moe_layer(x, wr, gu, dn, k, S_gu=sg, S_d=s2, dev_status=st)
    assert L.larosa_check(st) == 0
    assert idx[0].tolist() == [E - 1, E - 2]
    scores = x.double()[0] @ wr.double().t()
    want_gate = torch.softmax(scores[[E - 1, E - 2]], dim=0)
    U = 2.0 ** -23
    assert torch.all((gate[0].double() - want_gate).abs() <= (E + 110) * U * want_gate)
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    bound = torch.zeros(d, dtype=torch.float64, device="cuda")
    for s, e in enumerate((E - 1, E - 2)):  # the bound of tests/test_gpu_moe.py
        w = gu64(e)
        a, mag = x.double()[0] @ w, x.double()[0].abs() @ w.abs()
        u, G = a[f:], a[:f]
        dg, du = (d + 40) * U * mag[:f], (d + 40) * U * mag[f:]
        silu = G * torch.sigmoid(G)
        h = silu * u
        dh = 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + 8 * U * h.abs()
        w = dn64(e)
        want += want_gate[s] * (h @ w)
        bound += want_gate[s] * ((dh + (f + 40 + E + 110 + k) * U * h.abs()) @ w.abs())
        # 4-bit operands: 2^-50 of their block's largest
        bound += want_gate[s] * 2.0 ** -50 * 32 * h.abs().max() * w.abs().sum(dim=0)
    assert torch.all((y[0].double() - want).abs() <= bound * (1 + 2.0 ** -20))
