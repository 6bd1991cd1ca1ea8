"""The binding takes no address of a tensor that has no memory: 0 would stand for an
argument left out (no GPU needed)."""
import pytest
import torch

from attention_forward_gb300 import fa

CPU = -1  # what get_device() says of a CPU tensor


def test_a_functionalized_tensor_is_refused_by_name():
    x = torch.ones(3, dtype=torch.int32)
    said = []

    def body(y):
        with pytest.raises(ValueError, match="start must be a tensor with memory"):
            fa._ptr(y, "start", CPU, torch.int32, (3,))
        said.append(True)
        return y + 1

    torch.func.functionalize(body)(x)
    assert said == [True] and fa._ptr(x, "start", CPU, torch.int32, (3,)) == x.data_ptr()


def test_tensors_of_no_elements_have_no_address_to_check():
    x = torch.ones(0, dtype=torch.int32)
    assert fa._ptr(x, "start", CPU, torch.int32, (0,)) == x.data_ptr()
