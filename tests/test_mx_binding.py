"""What the MXFP4 binding refuses before it calls the library (CPU)."""
import pytest
import torch

from bit_gemm_nvfp4_amd import mx


@pytest.mark.parametrize("shape", [(0,), (2,), (4, 1)])
@pytest.mark.parametrize("name, dtype", [("src_scale", torch.float32), ("flags", torch.int32)])
def test_a_scale_or_flags_word_is_one_element(name, dtype, shape):
    # an empty one has no address and would count as not given, a scale per row would be taken for one of the tensor
    cpu = torch.device("cpu")
    with pytest.raises(AssertionError, match=name):
        mx._opt(torch.ones(shape, dtype=dtype), cpu, name, dtype)
    one = torch.ones(1, dtype=dtype)
    assert mx._opt(one, cpu, name, dtype) == one.data_ptr() and mx._opt(one.view(()), cpu, name, dtype) == one.data_ptr()
    with pytest.raises(AssertionError):
        mx._opt(one.double(), cpu, name, dtype)
