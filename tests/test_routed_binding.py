"""The binding of the low-rank adapters' call (no GPU needed): its list of column counts is
whole numbers of 32 bits, whatever earlier calls passed.
"""
import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def w4():
    __graft_entry__.build()
    import weight_only_int4_w4a16_gb300 as w4
    return w4


def call(w4, parts):
    f16 = torch.float16
    return w4.w4a16_lora(torch.zeros((2, 128), dtype=f16), torch.zeros((4, 16, 128), dtype=f16),
                         torch.zeros((4, 96, 16), dtype=f16), torch.ones(4),
                         torch.zeros(2, dtype=torch.int32), parts=parts)


def test_parts_of_more_than_32_bits(w4):
    # (the low 32 bits of these are the 96 columns)
    for parts in ([2 ** 32 + 96], (96 - 2 ** 32,), [64, 2 ** 40 + 32]):
        with pytest.raises(ValueError, match="fit 32 bits"):
            call(w4, parts)


def test_parts_that_are_not_whole_numbers(w4):
    with pytest.raises(ValueError, match="x must live on a CUDA device"):
        call(w4, [96])  # (past the check of parts)
    for parts in ([96.0], [torch.tensor(96.0)], ["96"]):
        with pytest.raises(TypeError):
            call(w4, parts)
    with pytest.raises(ValueError, match="x must live on a CUDA device"):
        call(w4, torch.tensor([64, 32]))
