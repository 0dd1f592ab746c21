"""Arguments of the 4-bit and expert calls in Python: what is taken, what is refused."""
from unittest import mock

import pytest
import torch


def test_what_is_no_tensor_is_refused_as_such():
    """Like every call of the binding: a ValueError that names the argument."""
    import activation_sparsity_b200 as L
    t = torch.zeros(32, 16, dtype=torch.uint8)
    for call in (lambda: L.larosa_mx4_dequantize(None, t), lambda: L.larosa_mx4_linear(None, t, t, t),
                 lambda: L.larosa_mx4_sparse_linear(t, t, None, t), lambda: L.larosa_mx4_topk_linear(t, None, t, 3),
                 lambda: L.larosa_mx4_quantize(None), lambda: L.larosa_moe_layer(None, t, t, t, 1)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_workspace_sizes_are_kept_apart_by_call():
    """Two calls with the same number of sizes, and the same sizes, each get their own query."""
    from activation_sparsity_b200 import larosa
    ws = larosa.Workspace.__new__(larosa.Workspace)
    ws.device, ws.buf, ws._need = torch.device("cuda", 0), torch.zeros(1000, dtype=torch.uint8), {}
    ws._outgrown, ws._capture = [], 0
    lib = mock.Mock(first=lambda *a: 10 + len(a), second=lambda *a: 20 + len(a), none=lambda *a: 0)
    lib.larosa_status_string.return_value = lib.larosa_last_error_string.return_value = b""
    with mock.patch.object(torch.cuda, "device"), mock.patch.object(larosa, "_lib", lib):
        for _ in range(2):
            assert ws._sized(("first", 1, 2, 3)) is ws.buf and ws._sized(("second", 1, 2, 3)) is ws.buf
        assert ws._need == {("first", 1, 2, 3): 13, ("second", 1, 2, 3): 23}
        with pytest.raises(larosa.LarosaError):
            ws._sized(("none", 1, 2, 3))


@pytest.mark.gpu
def test_a_single_token_may_have_one_dimension():
    import activation_sparsity_b200 as L
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(96, dtype=dtype, device="cuda")
        codes, scales = L.larosa_mx4_quantize(x)
        c, s = L.larosa_mx4_quantize(x.view(1, 96))
        assert codes.shape == (1, 48) and torch.equal(codes, c) and torch.equal(scales, s)
        W = L.larosa_mx4_quantize(torch.randn(40, 96, device="cuda"))
        assert L.larosa_mx4_linear(codes, scales, *W).shape == (1, 40)
        with pytest.raises(ValueError):
            L.larosa_mx4_quantize(x, axis=0)  # one row is no block


@pytest.mark.gpu
def test_an_output_of_another_type_than_asked_for_is_refused():
    import activation_sparsity_b200 as L
    f32, bf16 = torch.float32, torch.bfloat16
    x = L.larosa_mx4_quantize(torch.randn(3, 64, device="cuda"))
    W = L.larosa_mx4_quantize(torch.randn(16, 64, device="cuda"))
    for asked, given in ((f32, bf16), (bf16, f32)):
        y = torch.zeros(3, 16, dtype=given, device="cuda")
        with pytest.raises(TypeError):
            L.larosa_mx4_linear(*x, *W, dtype=asked, y=y)
        out = torch.zeros(3, 64, dtype=given, device="cuda")
        with pytest.raises(TypeError):
            L.larosa_mx4_dequantize(*x, dtype=asked, out=out)
        assert not y.any() and not out.any()
        assert L.larosa_mx4_linear(*x, *W, dtype=given, y=y) is y
        assert L.larosa_mx4_linear(*x, *W, y=y) is y  # without a type: y's
        assert L.larosa_mx4_dequantize(*x, out=out) is out
        assert L.larosa_mx4_linear(*x, *W, dtype=asked).dtype == asked
    assert L.larosa_mx4_linear(*x, *W).dtype == f32 and L.larosa_mx4_dequantize(*x).dtype == f32
