"""Whole numbers of other types that trees and caches take: what does not fit 32
bits stays out of range (a token of 2^32 + 5 is not 5), and what is no whole
number is refused."""

import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_verification_decode_gb300 import api  # noqa: E402

CPU = torch.device("cpu")


def test_wide_numbers_keep_their_side():
    x = torch.tensor([0, 1, -1, 2**31 - 1, 2**31, 2**32, 2**32 + 5, 2**63 - 1, -2**31, -2**31 - 1, -2**32 + 5, -2**63])
    top, low = 2**31 - 1, -2**31
    assert api._words(x, CPU, "x").tolist() == [0, 1, -1, top, top, top, top, top, low, low, low, low]
    assert x[6] == 2**32 + 5  # the caller's stay


@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8, torch.int16, torch.uint16, torch.int32, torch.uint32, torch.int64, torch.uint64])
def test_numbers_that_fit(dtype):
    x = torch.tensor([0, 5, 100], dtype=dtype)
    y = api._words(x, CPU, "x")
    assert y.dtype == torch.int32 and y.tolist() == [0, 5, 100]


def test_wide_unsigned_numbers():
    x = torch.tensor([7, 2**31 - 1, 2**31, 2**32 - 1], dtype=torch.int64)
    top = 2**31 - 1
    assert api._words(x.to(torch.uint32), CPU, "x").tolist() == [7, top, top, top]
    assert api._words(torch.tensor([7, 2**32 + 5, 2**63, 2**64 - 1], dtype=torch.uint64), CPU, "x").tolist() == [7, top, top, top]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bool, torch.complex64])
def test_other_types_are_refused(dtype):
    with pytest.raises(ValueError, match="whole numbers"):
        api._words(torch.zeros(3, dtype=dtype), CPU, "x")
