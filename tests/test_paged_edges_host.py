"""Arithmetic that paged attention relies on, without a GPU."""
import torch


def test_every_bf16_value_in_two_8_bit_parts():
    """An e4m3 and an e5m2 part hold all bf16 values up to 2^8 exactly from 2^-6 on, and the
    rest to 2^-14: each element of a row whose largest is 2^7 or more to 2^-21 of it."""
    x = torch.arange(0x4380, dtype=torch.int16).view(torch.bfloat16).float()
    assert x[0] == 0 and x[-1] < 256 and x[-1] * 1.004 > 256
    first = x.to(torch.float8_e4m3fn).float()
    rest = x - first
    off = (rest - rest.to(torch.float8_e5m2).float()).abs()
    assert off[x >= 2.0 ** -6].max() == 0 and off.max() <= 2.0 ** -14
