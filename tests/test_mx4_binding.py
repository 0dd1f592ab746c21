"""Arguments of the 4-bit and expert calls in Python: what is taken, what is refused."""
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
