"""Refusals of the Python layer of the training and quantising operators, before the native binding (CPU only)."""
import pytest
import torch

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.mark.parametrize("dtype,ydt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float16),
                                       (torch.float64, torch.bfloat16)])
@pytest.mark.parametrize("quantised", [False, True])
def test_dtype_that_is_not_the_outputs(dtype, ydt, quantised):
    a = torch.zeros((4, 32), dtype=torch.int8 if quantised else torch.bfloat16)
    s = torch.ones((4,)) if quantised else None
    with pytest.raises(ValueError, match="dtype"):
        om.int8_matmul(a, torch.zeros((6, 32), dtype=torch.int8), torch.ones((6,)), a_scale=s, dtype=dtype,
                       Y=torch.empty((4, 6), dtype=ydt))
