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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [4, 5, 70])
def test_rows_of_q_with_one_large_element(new, d):
    """One channel of Q is 2^12 to 2^17 times the rest, and the keys have nothing in it, so
    that the scores are those of the small elements alone.

    Sixteen rows and fewer hold Q in fp16, exact here.  More rows hold it as an e4m3 and
    an e5m2 part.  A row's largest element is at 2^7 at least.  What the e4m3 part leaves of an element of 2^-6 or
    more is at most 8 steps of bf16: 3 digits, which e5m2 has.  Of a smaller one it leaves at most 2^-10, where
    e5m2's steps are 2^-13: off by 2^-14 at most, 2^-21 of the row's largest."""
    g = torch.Generator().manual_seed(63)
    c = case([90], [new], 4, 1, d, 16, seed=63, spread=0)
    small = torch.tensor([2.0 ** -5, 2.0 ** -7, 2.0 ** -9, 2.0 ** -11, -2.0 ** -10, 2.0 ** -11])  # (the last: all alike)
    rows = torch.arange(new * 4).view(new, 4)
    c["q"] = (small[rows % 6][..., None] * (1 + torch.rand((new, 4, d), generator=g))).to(torch.bfloat16)
    c["q"][rows % 6 == 5] = 2.0 ** -11
    c["q"][..., 0] = 64.0
    keys = (0.25 + torch.rand((c["kc"].shape[0], 1, 16, d), generator=g)) * torch.rand((c["kc"].shape[0], 1, 16, 1), generator=g)
    keys[..., 0] = 0
    c["kc"] = keys.to(torch.float8_e4m3fn)
    c["ks"] = torch.ones_like(c["ks"])
    scale = 8.0
    o, lse, tol_o, tol_l = reference(c, scale=scale)
    if new * 4 > 16:
        # a weight carries its score's error, and so does the normaliser; sum w |v| is below the largest |v|
        seen = torch.cat([c["kc"][int(p), 0].double() for p in c["table"][0, :6]])[:90]
        e = 2.0 ** -21 * 64 * seen.abs().sum(-1).max() * scale
        values = torch.cat([c["vc"][int(p), 0].double() * c["vs"][int(p), 0] for p in c["table"][0, :6]])[:90]
        tol_o, tol_l = tol_o + 2 * e * values.abs().max(), tol_l + 2 * e
    dev = on_gpu(c)
    for splits in (1, 2, 9):
        assert_close(ea.attn_fwd_fp8_paged(**dev, max_q=new, max_kv=90, scale=scale, num_splits=splits), (o, lse, tol_o, tol_l))


@pytest.mark.parametrize("new", [3, 70])
def test_scales_of_v_a_hundred_powers_apart(new):
    """Blocks of V of 2^-50 to 2^50: the weights of the small ones count all the same."""
    g = torch.Generator().manual_seed(66)
    c = case([300, 90], [1, new], 4, 2, 64, 16, seed=66, spread=0)
    c["vs"] = 2.0 ** torch.randint(0, 2, c["vs"].shape, generator=g).float().mul(100).sub(50)
    want = reference(c, scale=0.5)
    dev = on_gpu(c)
    for splits in (1, 2, 9):
        assert_close(ea.attn_fwd_fp8_paged(**dev, max_q=new, max_kv=300, scale=0.5, num_splits=splits), want)


@pytest.mark.parametrize("d,tokens", [(64, 270), (128, 270), (256, 134)])
def test_last_wave_sees_what_was_written_right_before(d, tokens):
    """A wave of blocks and a few more, whose keys pairs of blocks share: lengths, page
    numbers, queries and the cache are written by the launches right before, without a wait, and read
    as after one."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = -(-(sms + 9) // 5)  # two tiles of each of three heads: a wave and a fifth
    g = torch.Generator().manual_seed(65)
    c = case([2048 + 16 * (b % 5) for b in range(B)], [tokens] * B, 3, 3, d, 128, seed=65)
    dev = on_gpu(c)
    pages = c["kc"].shape[0]
    dev["block_table"] = torch.cat([dev["block_table"].clamp(min=0), dev["block_table"].clamp(min=0)[:, :1]], 1).contiguous()
    tables = [dev["block_table"].clone(), dev["block_table"].flip(0).contiguous()]
    lens = [dev["kv_len"].clone(), dev["kv_len"].flip(0).contiguous()]
    kv = torch.randn((6, 2, 8, 3, d), generator=g).to(torch.bfloat16).cuda()
    start = [dev[k].clone() for k in ("q", "k_cache", "v_cache", "k_scale", "v_scale")]

    def run(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        for k, t in zip(("q", "k_cache", "v_cache", "k_scale", "v_scale"), start):
            dev[k].view(torch.uint8).copy_(t.view(torch.uint8))
        got = []
        for i in range(6):
            # eight tokens over the beginning of a page that some sequence has
            slots = (i * 7 % pages) * 128 + torch.arange(8, dtype=torch.int32, device="cuda")
            dev["q"].mul_(-1.25)
            dev["block_table"].copy_(tables[i % 2])
            dev["kv_len"].copy_(lens[i % 2])
            sync()
            ea.attn_paged_append_fp8(kv[i, 0], kv[i, 1], slots, dev["k_cache"], dev["v_cache"], dev["k_scale"], dev["v_scale"])
            sync()
            got += ea.attn_fwd_fp8_paged(**dev, max_q=tokens, max_kv=2112, num_splits=1)
            sync()
            dev["kv_len"].zero_()
            dev["block_table"].zero_()
            sync()
        return got

    want = run(True)
    assert not torch.equal(want[0], want[2])
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
