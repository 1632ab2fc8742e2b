"""Arguments of the operators around the Mamba-2 SSD that a call does not use, and of
types that it does not take.  No GPU needed: the pointers are never used."""
import ctypes

import pytest
import torch

import selective_state_space_38_b200 as ssm


def _p(i):
    return ctypes.c_void_p(0x10000000 + i * 0x1000000)


@pytest.mark.parametrize("sequences", [0, -1, 1 << 31, -(1 << 62)])
def test_steps_ignore_the_number_of_sequences(sequences):
    """A step has no cu_seqlens, and its call goes by no count of sequences: one that the packed forms would refuse
    comes as far as the check behind it (rows of out over the cache)."""
    lib = ssm.get_lib()
    dims = ssm.Conv1dDims(tokens=4, dim=128, sequences=sequences, slots=4, x_stride=128, y_stride=128, width=4, silu=1, act_dtype=1)
    assert lib.ssm_conv1d_step(_p(4), _p(5), _p(1), _p(2), None, _p(4), ctypes.byref(dims), None) == 1
    dims = ssm.SsdPackedDims(tokens=4, sequences=sequences, slots=4, heads=8, headdim=64, groups=2, dstate=128, x_stride=512,
                             dt_stride=8, b_stride=256, c_stride=256, y_stride=512, act_dtype=1)
    args = [_p(10), None, _p(1), _p(2), None, 1, _p(3), _p(4), _p(5), None, _p(10)]
    assert lib.ssm_ssd_step(*args, ctypes.byref(dims), None) == 1


def test_tables_that_are_no_tensors_or_of_other_types():
    from selective_state_space_38_b200.mamba2 import _tables
    cu, cpu = torch.tensor([0, 3, 5], dtype=torch.int32), torch.device("cpu")
    assert _tables(cu, None, torch.tensor([True, False]), cpu)[3] == 2
    assert _tables(cu, None, torch.tensor([1, 0], dtype=torch.uint8), cpu)[3] == 2
    for has_initial in ([True, False], True, torch.tensor([1, 0])):
        with pytest.raises(TypeError, match="has_initial"):
            _tables(cu, None, has_initial, cpu)
    with pytest.raises(ValueError, match="has_initial"):
        _tables(cu, None, torch.tensor([True]), cpu)
    with pytest.raises(TypeError, match="slots"):
        _tables(cu, [0, 1], None, cpu)


def test_sizes_of_what_is_no_tensor_or_of_another_rank():
    from selective_state_space_38_b200.mamba2 import _size
    assert _size(torch.zeros(6, 4), 1, 2, "conv_w") == 4
    with pytest.raises(TypeError, match="conv_w"):
        _size([[0.0] * 4], 1, 2, "conv_w")
    for shape in ((6,), (6, 1, 4)):
        with pytest.raises(ValueError, match="conv_w"):
            _size(torch.zeros(shape), 1, 2, "conv_w")
