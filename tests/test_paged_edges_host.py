"""Arithmetic that paged attention relies on and refusals of its entry points, without a
GPU (every call here is refused or does no device work)."""
from decimal import Decimal, getcontext

import pytest
import torch

import exact_attention_51_gb300 as ea
from exact_attention_51_gb300 import build as eabuild


@pytest.fixture(scope="module", autouse=True)
def built():
    eabuild.build()


def test_every_bf16_value_in_two_8_bit_parts():
    """An e4m3 and an e5m2 part hold all bf16 values up to 2^8 exactly from 2^-6 on, and the
    rest to 2^-14: each element of a row whose largest is 2^7 or more to 2^-21 of it."""
    x = torch.arange(0x4380, dtype=torch.int16).view(torch.bfloat16).float()
    assert x[0] == 0 and x[-1] < 256 and x[-1] * 1.004 > 256
    first = x.to(torch.float8_e4m3fn).float()
    rest = x - first
    off = (rest - rest.to(torch.float8_e5m2).float()).abs()
    assert off[x >= 2.0 ** -6].max() == 0 and off.max() <= 2.0 ** -14


A = 1 << 20  # fake, aligned "device" addresses (never dereferenced)


@pytest.mark.parametrize("kw", [dict(drop=-1), dict(ms=0), dict(ms=10001), dict(T=0), dict(splits=65), dict(d=96)])
def test_paged_selftest_refuses(kw):
    a = dict(T=6, d=64, splits=1, drop=0, ms=50) | kw
    lib = ea.load_library()
    assert lib.attn_selftest_fwd_fp8_paged_dropped_load(
        A, 8 * 64, 64, A + (1 << 34), A + (1 << 35), A + (1 << 36), A + (1 << 37), A + (1 << 30), 7, A + (1 << 31), A + (1 << 32),
        A + (1 << 38), A + (1 << 39), 3, a["T"], 8, 2, a["d"], 9, 16, 2, 100, 0.125, 1, a["splits"], None, 0, a["drop"], a["ms"],
        None) == ea.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("entry", ["attn_rope", "attn_rope_bwd"])
@pytest.mark.parametrize("stride", [1 << 62, 1 << 46, (1 << 61) + 5])
def test_rope_refuses_position_strides_that_wrap(entry, stride):
    """As of x and y: (B - 1) strides of 2^62 wrap to 0 for B = 5, an extent that overlaps nothing."""
    st = (3 * 5 * 64, 5 * 64, 64)
    rc = getattr(ea.load_library(), entry)(A, A + (1 << 30), 0, 5, 3, 5, 64, *st, *st, A + (1 << 34), stride, 0, A + (1 << 35), 64,
                                           0, 1.0, None)
    assert rc == ea.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rot_dim=(1 << 32) + 64), dict(rot_dim=-(1 << 32) + 64), dict(rot_dim=1 << 40), dict(rot_dim=-64),
                                dict(scaling="yarn", factor=2.0, original_positions=(1 << 32) + 4096)])
def test_phases_refuse_what_does_not_fit(kw):
    """Not taken for what is left of them in 32 bits, nor allocated first."""
    with pytest.raises(ea.AttnError):
        ea.attn_rope_phases(**({"rot_dim": 64, "device": "cpu"} | kw))


def test_paged_sizes_of_what_does_not_fit():
    big = 1 << 32
    assert ea.attn_fwd_fp8_paged_workspace_size(6, 8, 2, 64, 4, 11) > 0
    for i, n in enumerate((6, 8, 2, 64, 4, 11)):
        a = [6, 8, 2, 64, 4, 11]
        a[i] = n + big
        assert ea.attn_fwd_fp8_paged_workspace_size(*a) == 0
    sizes = [1, 32, 8, 128, 16, 1, 131072, 152]
    assert ea.attn_fwd_fp8_paged_num_splits(*sizes) > 1
    for i, n in enumerate(sizes):
        a = list(sizes)
        a[i] = n + big
        assert ea.attn_fwd_fp8_paged_num_splits(*a) == 1


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 1e6), (512, 1.5), (96, 500000.0)])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 4.0)])
def test_phases_within_a_fraction_of_a_turn(rot, base, scaling, factor):
    """f / 2 pi = base^-e / 2 pi to 2^-52 of a turn, in steps of fp64 (2^-53 of the value each): pow's
    result, 2; 2 pi, the division and the scaling, 3; and as errors of the exponent and of
    NTK's base (3) reach f times e ln(base) and e, at most 1 / e and 1 of f, 4 more: 9 steps of 0.16 at most."""
    if scaling == "ntk" and rot == 2:
        return
    getcontext().prec = 40
    got, _ = ea.attn_rope_phases(rot, base=base, scaling=scaling, factor=factor, device="cpu")
    b = Decimal(base)
    if scaling == "ntk":
        b *= (Decimal(factor).ln() * rot / (rot - 2)).exp()
    for i, u in enumerate(got.tolist()):
        f = (b.ln() * Decimal(-2 * i) / rot).exp() / (Decimal(factor) if scaling == "linear" else 1)
        assert abs(Decimal(u) / 2 ** 64 - f / (2 * PI)) <= Decimal(2) ** -52


def test_paged_selftest_refuses_what_the_gpu_cannot_read():
    c, s, i = torch.zeros((2, 1, 16, 64), dtype=torch.uint8), torch.zeros((2, 1)), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    rest = dict(max_q=1, max_kv=16, num_splits=1, drop_load=0)
    with pytest.raises(ValueError):
        ea.attn_selftest_fwd_fp8_paged_dropped_load(q, c, c, s, s, i[None], i[:1], i, **rest)
    with pytest.raises(TypeError):
        ea.attn_selftest_fwd_fp8_paged_dropped_load(q.float(), c, c, s, s, i[None], i[:1], i, **rest)
