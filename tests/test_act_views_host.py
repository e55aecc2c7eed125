"""Which tensors the activation calls' binding takes as a matrix of 16-bit values (CPU).

CPU tensors stand for device tensors: the binding's device is told to be theirs,
and only the check is run.
"""

import pytest
import torch

from zero_sharded_mixed_flat_amd import abi

B, S, C = 3, 4, 40


def _x(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _take(x, rows, cols, stride):
    assert abi._matrix(x, rows, cols, stride, x.get_device(), "x") == x.data_ptr()


GOOD = {
    "a matrix": lambda: (_x(12, C), 12, C, C),
    "more than is asked": lambda: (_x(12, C), 7, 31, C),
    "columns of a wider one": lambda: (_x(12, C)[:, 8:20], 12, 12, C),
    "every third row": lambda: (_x(12, C)[::3], 4, C, 3 * C),
    "one row of many": lambda: (_x(12, C)[5], 1, C, C),
    "one row, any stride": lambda: (_x(12, C)[5:6], 1, C, 77),
    "one column": lambda: (_x(12, C)[:, 3:4], 12, 1, C),
    "one column of a transposed matrix": lambda: (_x(C, 12).t()[:, :1], 12, 1, 1),
    "a batch of sequences": lambda: (_x(B, S, C), B * S, C, C),
    "a batch of sequences, some columns": lambda: (_x(B, S, C)[:, :, 4:30], B * S, 26, C),
    "one sequence first": lambda: (_x(1, S, C).transpose(0, 1), S, C, C),
    "heads apart": lambda: (_x(12, 4, 10), 12, 40, 40),
    "heads apart, of a wider product": lambda: (_x(12, 100)[:, 20:60].view(12, 4, 10), 12, 40, 100),
    "flat memory": lambda: (_x(1000), 12, 33, 83),
    "flat memory behind a batch of one": lambda: (_x(1, 1000), 12, 33, 83),
}


@pytest.mark.parametrize("case", GOOD)
def test_taken(case):
    _take(*GOOD[case]())


BAD = {
    # a view's rows in another order than its memory's
    "a transposed batch": (lambda: (_x(B, S, C).transpose(0, 1), B * S, C, C), "apart"),
    "sequences cut short": (lambda: (_x(B, S, C)[:, :3], B * 3, C, C), "apart"),
    "heads first": (lambda: (_x(12, 4, 10).transpose(0, 1), 48, 10, 10), "apart"),
    "an expanded row": (lambda: (_x(1, C).expand(12, C), 12, C, C), "apart"),
    "an expanded batch": (lambda: (_x(1, S, C).expand(B, S, C), B * S, C, C), "apart"),
    # less than the call says, with memory behind it
    "too few columns": (lambda: (_x(12, C)[:, :20], 12, 30, C), "holds"),
    "too few rows": (lambda: (_x(12, C)[:2], 10, C, C), "holds"),
    "too few rows of a wide matrix": (lambda: (_x(12, 2 * C)[:2, :C], 10, C, 2 * C), "holds"),
    "too few sequences": (lambda: (_x(B, S, C)[:2], B * S, C, C), "holds"),
    "too few columns of a batch": (lambda: (_x(B, S, C)[:, :, :20], B * S, 30, C), "holds"),
    "one row of many, all asked": (lambda: (_x(12, C)[0], 12, C, C), "holds"),
    "one row asked, wider": (lambda: (_x(12, C)[0:1, :20], 1, 30, C), "holds"),
    "flat memory, its last row short": (lambda: (_x(1000), 12, 100, 82), "holds"),
    # as before
    "a transposed matrix": (lambda: (_x(C, 12).t(), 12, C, C), "adjacent"),
    "every second column": (lambda: (_x(12, 2 * C)[:, ::2], 12, C, 2 * C), "adjacent"),
    "another stride": (lambda: (_x(12, C + 2)[:, :C], 12, C, C), "apart"),
    "a matrix of other rows": (lambda: (_x(6, 2 * C), 12, C, C), "apart"),
    "fp32": (lambda: (torch.zeros(12, C), 12, C, C), "16-bit"),
}


@pytest.mark.parametrize("case", BAD)
def test_refused(case):
    make, match = BAD[case]
    with pytest.raises(ValueError, match=match):
        _take(*make())
