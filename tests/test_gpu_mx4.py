"""The microscaled 4-bit format and the sparse linear with a 4-bit weight,
against the fp64 oracle.

Quantising is exact integer work on powers of two: codes and scales equal the
oracle's bit for bit, and reading back equals its values (a bf16 or fp32 holds
every 4-bit value).

Sparse linear: a coefficient is held to 2^-24 of itself (or 2^-50 of the
largest of its block), products of the pieces are exact, and a sum's additions
each lose at most 2^-23 of the running magnitude (the tensor cores truncate).
An output passes through at most 34 additions in a block (two 16-term steps),
one per block of its warp (an eighth of the CTA's) and 16 in the reductions,
so |error| <= (52 + blocks) 2^-23 sum |v w|, with the second term of the
coefficients added.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import synthdata as sd
from tests.test_gpu_parity import f64, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from activation_sparsity_b200 import build_lib
    build_lib.build()
    import activation_sparsity_b200 as L
    torch.cuda.init()
    return L


def unpack(codes: torch.Tensor) -> np.ndarray:
    c = codes.cpu().numpy()
    out = np.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=np.int64)
    out[..., 0::2], out[..., 1::2] = c & 15, c >> 4
    return out


def spread(rows, cols, seed, dtype, lo=-30, hi=30):
    """Gaussian entries times powers of two that vary from entry to entry."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(lo, hi + 1, (rows, cols)) // 6)
    x[rng.random((rows, cols)) < 0.05] = 0.0
    return torch.from_numpy(x).to(dtype)


# ---------------------------------------------------------------- the format

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("axis,rows,cols", [(1, 1, 32), (1, 1, 4096), (1, 3, 96), (1, 777, 1056), (1, 37, 11008),
                                            (0, 32, 32), (0, 32, 96), (0, 96, 4128), (0, 4096, 32), (0, 256, 1024)])
def test_quantize_is_the_oracles_bit_for_bit(L, dtype, axis, rows, cols):
    x = spread(rows, cols, rows + cols, dtype)
    st = status()
    codes, scales = L.larosa_mx4_quantize(x.cuda(), axis=axis, dev_status=st)
    assert L.larosa_check(st) == 0
    wc, ws = oracle.mx4_quantize(f64(x), axis)
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(unpack(codes), wc)
    for out in (torch.float32, torch.bfloat16):
        got = f64(L.larosa_mx4_dequantize(codes, scales, axis=axis, dtype=out))
        assert np.array_equal(got, oracle.mx4_values(wc, ws, axis))


@pytest.mark.parametrize("axis", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_borders(L, axis, dtype):
    """Ties, saturation, zeros of both signs, subnormals and the largest values."""
    vals = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, -5.0, 6.0, -0.0, 0.0, 4.0]
    rows = []
    for e in (-140, -133, -127, -126, -125, -120, -1, 0, 1, 60, 124):
        r = np.zeros(32)
        r[:len(vals)] = np.ldexp(vals, e)
        rows.append(r)
    rows.append(np.full(32, 2.0 ** 127 * (2 - 2.0 ** -7)))  # the largest bf16
    rows.append(np.zeros(32))
    x = torch.from_numpy(np.stack(rows)).to(dtype)
    x = x if axis == 1 else x.t().contiguous().repeat(1, 32)
    codes, scales = L.larosa_mx4_quantize(x.cuda(), axis=axis)
    wc, ws = oracle.mx4_quantize(f64(x), axis)
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(unpack(codes), wc)
    got = f64(L.larosa_mx4_dequantize(codes, scales, axis=axis))
    assert np.array_equal(got, oracle.mx4_values(wc, ws, axis))


@pytest.mark.parametrize("axis", [0, 1])
def test_nonfinite_block_is_reported_and_reads_back_as_nan(L, axis):
    x = spread(64, 64, 5, torch.float32)
    x[3, 40], x[50, 7] = float("nan"), float("-inf")
    st = status()
    codes, scales = L.larosa_mx4_quantize(x.cuda(), axis=axis, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == L.LAROSA_DEV_NONFINITE
    wc, ws = oracle.mx4_quantize(f64(x), axis)
    assert np.array_equal(scales.cpu().numpy(), ws) and np.array_equal(unpack(codes), wc)
    for dt in (torch.float32, torch.bfloat16):
        got = f64(L.larosa_mx4_dequantize(codes, scales, axis=axis, dtype=dt))
        assert np.array_equal(np.isnan(got), np.isnan(oracle.mx4_values(wc, ws, axis)))


def test_every_code_and_scale_reads_back(L):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :256].contiguous().cuda()  # 512 columns
    scales = torch.arange(256, dtype=torch.uint8).repeat(16, 1).t().contiguous().cuda()
    got = f64(L.larosa_mx4_dequantize(codes, scales))
    want = oracle.mx4_values(unpack(codes), scales.cpu().numpy(), 1)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    assert np.array_equal(got, want, equal_nan=True)


def test_stacked_matrices_are_their_rows_in_turn(L):
    x = torch.stack([spread(64, 96, s, torch.bfloat16) for s in (1, 2, 3)]).cuda()
    for axis in (0, 1):
        codes, scales = L.larosa_mx4_quantize(x, axis=axis)
        for i in range(3):
            c, s = L.larosa_mx4_quantize(x[i].contiguous(), axis=axis)
            assert torch.equal(codes[i], c) and torch.equal(scales[i], s)
        assert L.larosa_mx4_dequantize(codes, scales, axis=axis).shape == x.shape


# ---------------------------------------------------------------- sparse linear

def weight(L, d_in, d_out, seed, std=0.02):
    W = sd.weights(d_in, d_out, std, seed, torch.float32)
    codes, scales = L.larosa_mx4_quantize(W.cuda(), axis=0)
    return codes, scales, oracle.mx4_values(unpack(codes), scales.cpu().numpy(), 0)


def check_y(got, idx, val, W):
    d_in = W.shape[0]
    for m in range(got.shape[0]):
        i, v = idx[m], val[m]
        want = v @ W[i] if len(i) else np.zeros(W.shape[1])
        mag = np.abs(v) @ np.abs(W[i]) if len(i) else np.zeros(W.shape[1])
        top = (np.max(np.abs(v)) if len(v) else 0.0) * np.max(np.abs(W), initial=0.0)
        bound = (52 + d_in // 32) * 2.0 ** -23 * mag + len(i) * 2.0 ** -50 * top
        assert np.all(np.abs(got[m] - want) <= bound + 1e-37), np.max(np.abs(got[m] - want) / (bound + 1e-37))


SHAPES = [(1, 32, 32, 1), (1, 32, 32, 32), (1, 64, 96, 0), (1, 256, 544, 100), (2, 256, 160, 17),
          (3, 512, 128, 300), (4, 1024, 256, 600), (5, 1024, 288, 700), (8, 2048, 128, 2048), (9, 1024, 128, 50),
          (16, 1024, 416, 600), (16, 64, 32, 64), (13, 4096, 1024, 2458), (1, 4096, 4096, 2458),
          (1, 11008, 4096, 6605), (1, 32768, 128, 20000), (16, 13824, 512, 8295)]


@pytest.mark.parametrize("M,d_in,d_out,K", SHAPES)
def test_sparse_linear(L, M, d_in, d_out, K):
    codes, scales, W = weight(L, d_in, d_out, 40 + d_in)
    idx, val = sd.index_values(M, d_in, K, 41 + K)
    st = status()
    y = L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales, dev_status=st)
    assert L.larosa_check(st) == 0
    check_y(f64(y), idx.numpy(), f64(val), W)
    again = L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales)
    assert torch.equal(y, again)


def test_unordered_lists_and_zero_values(L):
    codes, scales, W = weight(L, 512, 256, 50)
    idx, val = sd.index_values(3, 512, 200, 51)
    perm = torch.randperm(200, generator=torch.Generator().manual_seed(1))
    val[:, ::3] = 0.0
    val[1] = 0.0  # a token that keeps nothing
    y0 = L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales)
    y1 = L.larosa_mx4_sparse_linear(idx[:, perm].contiguous().cuda(), val[:, perm].contiguous().cuda(), codes, scales)
    assert torch.equal(y0, y1)
    assert not y0[1].any()
    check_y(f64(y0), idx.numpy(), f64(val), W)


def test_wide_ranges_of_coefficients_and_scales(L):
    """Coefficients 2^-40 ... 2^40 and column scales 2^-60 ... 2^20."""
    rng = np.random.default_rng(8)
    d_in, d_out, M, K = 256, 128, 5, 200
    codes = torch.from_numpy(rng.integers(0, 256, (d_in, d_out // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(67, 148, (d_in // 32, d_out), dtype=np.uint8)).cuda()
    W = oracle.mx4_values(unpack(codes), scales.cpu().numpy(), 0)
    idx, val = sd.index_values(M, d_in, K, 9)
    val = val * torch.from_numpy(np.exp2(rng.integers(-40, 41, (M, K)))).float()
    got = f64(L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales))
    i, v = idx.numpy(), f64(val)
    for m in range(M):
        want = v[m] @ W[i[m]]
        mag = np.abs(v[m]) @ np.abs(W[i[m]])
        # 2^-50 of the block's largest coefficient against the column's largest entry in the block
        tail = np.zeros(d_out)
        for b in range(d_in // 32):
            here = (i[m] // 32) == b
            if here.any():
                tail += 32 * np.max(np.abs(v[m][here])) * 2.0 ** -50 * np.max(np.abs(W[32 * b:32 * b + 32]), axis=0)
        assert np.all(np.abs(got[m] - want) <= (52 + d_in // 32) * 2.0 ** -23 * mag + tail)


def test_nan_scale_reaches_only_its_column(L):
    codes, scales, W = weight(L, 128, 64, 60)
    scales[2, 5] = 255
    idx = torch.arange(128, dtype=torch.int32).view(1, -1)
    val = torch.ones(1, 128)
    y = L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales)
    bad = torch.isnan(y[0]).nonzero().flatten().tolist()
    assert bad == [5]
    # rows 64 .. 95 not kept: the block with the NaN scale is not read
    y = L.larosa_mx4_sparse_linear(idx[:, :64].contiguous().cuda(), val[:, :64].contiguous().cuda(), codes, scales)
    assert not torch.isnan(y).any()


def test_index_out_of_range_is_reported_and_skipped(L):
    codes, scales, W = weight(L, 128, 64, 61)
    idx = torch.tensor([[3, 128, -1, 7]], dtype=torch.int32)
    val = torch.tensor([[1.0, 5.0, 5.0, 2.0]])
    st = status()
    y = L.larosa_mx4_sparse_linear(idx.cuda(), val.cuda(), codes, scales, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == L.LAROSA_DEV_INDEX
    check_y(f64(y), np.array([[3, 7]]), np.array([[1.0, 2.0]]), W)


@pytest.mark.parametrize("M,d_in,d_out,K", [(1, 256, 512, 154), (1, 4096, 1024, 2458), (2, 512, 128, 0),
                                            (6, 1024, 256, 1024), (16, 2048, 128, 1229)])
def test_topk_linear(L, M, d_in, d_out, K):
    codes, scales, W = weight(L, d_in, d_out, 70)
    x = sd.activations(M, d_in, 71, torch.float32)
    ws = L.Workspace()
    st = status()
    y = L.larosa_mx4_topk_linear(x.cuda(), codes, scales, K, ws=ws, dev_status=st)
    assert L.larosa_check(st) == 0
    idx, val = oracle.topk(f64(x), K)
    check_y(f64(y), idx, val, W)


def test_rotated_path_with_a_quantised_weight(L):
    """The decode path as a user runs it: rotate, select, multiply by the 4-bit W_rot."""
    d_in, d_out, M, K = 512, 256, 4, 308
    Q = sd.orthogonal(d_in, 80).float()
    W = sd.weights(d_in, d_out, 0.02, 81, torch.float32)
    x = sd.activations(M, d_in, 82, torch.float32)
    Qt = Q.t().contiguous().cuda()
    W_rot = L.larosa_prepare_weights(Qt, W.cuda())
    codes, scales = L.larosa_mx4_quantize(W_rot, axis=0)
    x_rot = L.larosa_rotate(x.cuda(), Qt)
    y = L.larosa_mx4_topk_linear(x_rot, codes, scales, K)
    idx, val = oracle.topk(f64(x_rot), K)
    check_y(f64(y), idx, val, oracle.mx4_values(unpack(codes), scales.cpu().numpy(), 0))


def test_captured_and_replayed_with_new_inputs(L):
    codes, scales, W = weight(L, 1024, 256, 90)
    x = torch.zeros(2, 1024, device="cuda")
    ws = L.Workspace()
    st = status()
    y = L.larosa_mx4_topk_linear(x, codes, scales, 600, ws=ws, dev_status=st)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c, s = L.larosa_mx4_quantize(x, dev_status=st)
        back = L.larosa_mx4_dequantize(c, s)
        L.larosa_mx4_topk_linear(x, codes, scales, 600, y=y, ws=ws, dev_status=st)
    for seed in (91, 92):
        xn = sd.activations(2, 1024, seed, torch.float32)
        x.copy_(xn)
        g.replay()
        assert L.larosa_check(st) == 0
        idx, val = oracle.topk(f64(xn), 600)
        check_y(f64(y), idx, val, W)
        assert np.array_equal(f64(back), oracle.mx4_values(*oracle.mx4_quantize(f64(xn), 1), 1))


def test_calls_on_two_streams(L):
    codes, scales, W = weight(L, 2048, 512, 95)
    idx, val = sd.index_values(1, 2048, 1200, 96)
    idx, val = idx.cuda(), val.cuda()
    want = L.larosa_mx4_sparse_linear(idx, val, codes, scales)
    torch.cuda.synchronize()
    ys = []
    for _ in range(2):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ys.append([L.larosa_mx4_sparse_linear(idx, val, codes, scales) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for group in ys for y in group)
