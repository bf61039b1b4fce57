"""The rotary and paged-cache calls on a stream that is not torch's current one."""
import pytest
import torch

import exact_attention_51_gb300 as ea
from test_gpu_paged import case, clean_status, on_gpu  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def busy_blocks(sizes):
    """Blocks of these sizes that the current stream still writes NaN to when they are
    freed: torch's allocator may give them out again, to this stream."""
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    for b in blocks:
        b.fill_(0xff)


def test_what_a_call_allocates_is_of_its_stream():
    """The call's stream does not wait for the current one, as it need not where the
    inputs were there long before; its output, LSE and workspace are not what
    the current stream still uses."""
    c = case([900, 77], [1, 4], 8, 2, 128, 16, seed=70)
    dev = on_gpu(c)
    ph, _ = ea.attn_rope_phases(128)
    x = torch.randn((1, 8, 40, 128), device="cuda").to(torch.bfloat16)
    want = [*ea.attn_fwd_fp8_paged(**dev, max_q=4, num_splits=12), ea.attn_rope(x, ph), ea.attn_rope_bwd(x, ph)]
    need = ea.attn_fwd_fp8_paged_workspace_size(5, 8, 2, 128, 4, 12)
    sizes = [need] + [t.numel() * t.element_size() for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        busy_blocks(sizes)
        got = [*ea.attn_fwd_fp8_paged(**dev, max_q=4, num_splits=12, stream=stream), ea.attn_rope(x, ph, stream=stream),
               ea.attn_rope_bwd(x, ph, stream=stream)]
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_results_are_not_given_out_again_while_the_caller_uses_them():
    """A result that is freed while the caller's stream still reads it is not what the
    next call on the other stream gets."""
    ph, _ = ea.attn_rope_phases(128)
    x = torch.randn((2, 8, 4096, 128), device="cuda").to(torch.bfloat16)
    y = torch.full_like(x, 3.0)
    want = ea.attn_rope(x, ph)
    copy = torch.zeros_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = ea.attn_rope(x, ph, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copy.copy_(first)
    del first
    for _ in range(4):
        ea.attn_rope(y, ph, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
