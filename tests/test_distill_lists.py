"""The binding's marshalling of the clients' lists (CPU): arrays of another type than the kernels
read are refused, since what they would read is not what the caller wrote."""
import numpy as np
import pytest
import torch

import server_side_fedavg_gb300 as fa


def lists(index, value, dtype_value="f32"):
    return fa.distill_lists([index], [value], [4], [1.0], dtype_value)


def test_indices_as_torch_topk_gives_them_are_refused():
    top = torch.randn(3, 10).topk(4)
    with pytest.raises(TypeError, match="int32"):
        lists(top.indices, top.values)
    arr, n, _, keep = lists(top.indices.int(), top.values)
    assert n == 1 and arr[0].index == keep[0][0].data_ptr() and arr[0].value == keep[1][0].data_ptr()


@pytest.mark.parametrize("index", [torch.zeros(3, 4), torch.zeros(3, 4, dtype=torch.int16), torch.zeros(3, 4, dtype=torch.bool),
                                   np.zeros((3, 4)), np.zeros((3, 4), np.int64), np.zeros((3, 4), np.float32)])
def test_other_indices_are_refused(index):
    with pytest.raises(TypeError, match="int32"):
        lists(index, torch.zeros(3, 4))


@pytest.mark.parametrize("value,dtype", [
    (torch.zeros(3, 4, dtype=torch.float64), "f32"), (torch.zeros(3, 4, dtype=torch.bfloat16), "f32"),
    (torch.zeros(3, 4, dtype=torch.float16), "bf16"), (torch.zeros(3, 4), "bf16"), (torch.zeros(3, 4, dtype=torch.int32), "f32"),
    (np.zeros((3, 4)), "f32"), (np.zeros((3, 4), np.float16), "bf16"), (np.zeros((3, 4), np.int32), "f32")])
def test_values_of_another_type_are_refused(value, dtype):
    with pytest.raises(TypeError, match=dtype):
        lists(torch.zeros(3, 4, dtype=torch.int32), value, dtype)


def test_what_the_kernels_read_is_taken():
    i = torch.zeros(3, 4, dtype=torch.int32)
    lists(i, torch.zeros(3, 4))
    lists(i, torch.zeros(3, 4, dtype=torch.bfloat16), "bf16")
    lists(np.zeros((3, 4), np.int32), np.zeros((3, 4), np.float32))
    lists(i, np.zeros((3, 4), np.uint16), "bf16")         # bf16 bits: numpy has no such type
    lists(i, torch.zeros(3, 4, dtype=torch.uint16), "bf16")
    lists(4096, 8192)                                       # plain addresses
    lists(None, None)                                       # refused by the call itself
