"""Attention over the paged e4m3 cache where its arithmetic is at an edge, against
the 64-bit definition: queries that are not numbers, factors of any size, rows of Q
whose elements differ much."""
import math

import pytest
import torch

import exact_attention_51_gb300 as ea
from test_gpu_paged import assert_close, case, clean_status, on_gpu, reference  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [3, 70])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_rows_without_keys_are_empty_whatever_their_query(new, d, value):
    """More causal queries than keys: the first see none, and give O = 0 and LSE = -inf
    even where their Q is not a number, among rows that see keys."""
    c = case([new - 1], [new], 4, 2, d, 16, seed=60)
    want = reference(c)
    dev = on_gpu(c)
    dev["q"][0, :3, 5] = value
    for splits in (1, 2, 9):
        assert_close(ea.attn_fwd_fp8_paged(**dev, max_q=new, max_kv=128, num_splits=splits), want)


@pytest.mark.parametrize("new", [3, 70])
def test_rows_whose_pages_are_all_hidden_are_empty_whatever_their_query(new):
    c = case([new], [new], 4, 2, 64, 128, seed=61)
    dev = on_gpu(c)
    dev["q"][:] = math.nan
    dev["block_table"][0, 0] = -5
    for splits in (1, 2):
        o, lse = ea.attn_fwd_fp8_paged(**dev, max_q=new, max_kv=256, num_splits=splits)
        assert ea.attn_fwd_device_status() == (ea.ATTN_ERR_BAD_INDEX, 0x202)
        assert o.eq(0).all() and lse.eq(-math.inf).all()


@pytest.mark.parametrize("new", [3, 70])
@pytest.mark.parametrize("q,k,scale", [(1.0, 2.0 ** 60, 0.0), (2.0 ** -100, 2.0 ** 60, 0.125),
                                       (1.0, 2.0 ** -60, 2.0 ** 60), (1.0, 2.0 ** -60, 0.0)])
def test_score_factors_of_any_size(new, q, k, scale):
    """Small factors of Q and the scale against large keys, and the other way round: no
    factor is held at a bound of its own, and a masked key stays one however small they are."""
    c = case([200, 90], [1, new], 4, 2, 64, 16, seed=62, spread=0)
    c["q"] = (c["q"].double() * q).to(torch.bfloat16)
    c["ks"] = torch.full_like(c["ks"], k)
    want = reference(c, scale=scale)
    dev = on_gpu(c)
    for splits in (1, 2, 9):
        assert_close(ea.attn_fwd_fp8_paged(**dev, max_q=new, max_kv=200, scale=scale, num_splits=splits), want)


@pytest.mark.parametrize("new", [3, 70])
@pytest.mark.parametrize("q", [2.0 ** -110, 2.0 ** -124, 2.0 ** -131, 2.0 ** 126])
def test_rows_of_q_at_the_ends_of_bf16(new, q):
    """As exact as other rows, subnormal ones too (whose few digits bf16 has rounded already)."""
    c = case([200, 90], [1, new], 4, 2, 64, 16, seed=64, spread=0)
    c["q"] = (c["q"].double().clamp(-1.9, 1.9) * q).to(torch.bfloat16)
    c["ks"] = torch.full_like(c["ks"], 2.0 ** 40 if q < 1 else 2.0 ** -60)
    scale = 2.0 ** -10 / q * (2.0 ** -40 if q < 1 else 2.0 ** 60)
    want = reference(c, scale=scale)
    dev = on_gpu(c)
    for splits in (1, 2, 9):
        assert_close(ea.attn_fwd_fp8_paged(**dev, max_q=new, max_kv=200, scale=scale, num_splits=splits), want)
