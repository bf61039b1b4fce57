"""Paged attention's abort paths, without a fault: a load that every block leaves out, so
that a bounded wait runs out.  Every role leaves its waits, copies and products in flight end,
clusters keep their barriers in step, the kernel returns, and the next call is right."""
import time

import pytest
import torch

import exact_attention_51_gb300 as ea
from test_gpu_paged import case, clean_status, on_gpu  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

FEW = {0x141, 0x142}
MANY = set(range(0x151, 0x158))


def check(dev, max_q, max_kv, splits, drops, codes, causal=True):
    want = ea.attn_fwd_fp8_paged(**dev, max_q=max_q, max_kv=max_kv, num_splits=splits, causal=causal)
    assert ea.attn_fwd_device_status() == (ea.ATTN_OK, 0)
    for drop in drops:
        t0 = time.perf_counter()
        assert ea.attn_selftest_fwd_fp8_paged_dropped_load(**dev, max_q=max_q, max_kv=max_kv, num_splits=splits, causal=causal,
                                                           drop_load=drop, timeout_ms=50) == ea.ATTN_OK
        st, detail = ea.attn_fwd_device_status()
        elapsed = time.perf_counter() - t0
        assert st == ea.ATTN_ERR_TIMEOUT and detail in codes, (drop, st, hex(detail))
        assert 0.04 <= elapsed < 5.0, elapsed
        assert ea.attn_fwd_device_status() == (ea.ATTN_OK, 0)
        got = ea.attn_fwd_fp8_paged(**dev, max_q=max_q, max_kv=max_kv, num_splits=splits, causal=causal)
        assert ea.attn_fwd_device_status() == (ea.ATTN_OK, 0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# one block for all keys, a cluster whose blocks some rows leave without keys, shares in the workspace
SPLITS = pytest.mark.parametrize("splits", [1, 3, 11], ids=["one", "cluster", "workspace"])


@SPLITS
@pytest.mark.parametrize("page", [16, 64], ids=["own copies", "a warp's copies"])
@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 8), (256, 8)])
def test_few_rows(d, Hq, page, splits):
    dev = on_gpu(case([3000, 5, 1200], [2, 1, 1], Hq, 2, d, page, seed=90))
    # the first stage, one behind the ring's first round, and, in one block for all, one far back
    check(dev, 2, 3000, splits, (0, 1, 14) if splits == 1 else (0, 1), FEW)


@pytest.mark.parametrize("splits", [1, 3, 7], ids=["one", "cluster", "workspace"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows(d, splits):
    dev = on_gpu(case([2100, 40, 1200], [150, 40, 33], 6, 2, d, 32, seed=91))
    # keys and values of the first tile, of the next, and, in one block for all, of one far back
    check(dev, 150, 2100, splits, (0, 1, 2, 3, 20, 21) if splits == 1 else (0, 1, 2, 3), MANY)


@pytest.mark.parametrize("d,tokens", [(64, 270), (128, 270), (256, 134)])
def test_last_wave(d, tokens):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = -(-(sms + 9) // 5)
    dev = on_gpu(case([2048] * B, [tokens] * B, 3, 3, d, 128, seed=92))
    check(dev, tokens, 2048, 1, (0, 3), MANY)
