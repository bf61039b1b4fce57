"""Writes of the rotary and paged-cache calls into the caller's tensors are counted as
torch's own in-place operations are."""
import pytest
import torch

import exact_attention_51_gb300 as ea
from test_gpu_paged import case, clean_status, on_gpu  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_versions_of_what_is_written():
    ph, _ = ea.attn_rope_phases(64)
    c = on_gpu(case([40, 9], [2, 3], 4, 2, 64, 16, seed=80))
    kv = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    cache = [c[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")]
    x = torch.randn((1, 2, 5, 64), device="cuda")
    out, o, lse = torch.empty_like(x), torch.empty_like(c["q"]), torch.empty((5, 4), device="cuda")
    every = [*cache, kv, slots, ph, x, out, o, lse, *c.values()]

    def changed(call):
        before = [t._version for t in every]
        call()
        return {id(t) for t, v in zip(every, before) if t._version != v}

    assert changed(lambda: ea.attn_rope(x, ph)) == set()
    assert changed(lambda: ea.attn_rope(x, ph, out=out)) == {id(out)}
    assert changed(lambda: ea.attn_rope_bwd(x, ph, out=x)) == {id(x)}
    assert changed(lambda: ea.attn_paged_append_fp8(kv, kv, slots, *cache)) == {id(t) for t in cache}
    assert changed(lambda: ea.attn_fwd_fp8_paged(**c, max_q=3)) == set()
    assert changed(lambda: ea.attn_fwd_fp8_paged(**c, max_q=3, out=o, lse=lse)) == {id(o), id(lse)}
    with pytest.raises(ea.AttnError):  # refused: not written
        ea.attn_rope(x, ph, position0=(1 << 31) - 2, out=out)
    assert changed(lambda: ea.attn_paged_append_fp8(kv[:0], kv[:0], slots[:0], *cache)) == set()


def test_a_saved_value_that_was_rotated_in_place_is_refused():
    ph, _ = ea.attn_rope_phases(64)
    x = torch.randn((1, 2, 5, 64), device="cuda", requires_grad=True) * 2
    y = x.square().sum()
    ea.attn_rope(x, ph, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors_are_written_anywhere():
    ph, _ = ea.attn_rope_phases(64)
    with torch.inference_mode():
        cache = [torch.zeros((2, 2, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
        cache += [torch.zeros((2, 2), device="cuda") for _ in range(2)]
        x = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
        slots = torch.arange(3, dtype=torch.int32, device="cuda")
        ea.attn_paged_append_fp8(x, x, slots, *cache)
        ea.attn_rope(x.transpose(0, 1)[None], ph, out=x.transpose(0, 1)[None])
    first = cache[0].clone()
    ea.attn_paged_append_fp8(x, x, slots, *cache)  # (x was rotated since)
    ea.attn_rope(x.transpose(0, 1)[None], ph, out=x.transpose(0, 1)[None])
    assert not torch.equal(cache[0], first)
