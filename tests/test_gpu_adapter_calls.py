"""Calls of the adapter, gated-activation and input-gradient entries at the edges of what
they document: buffers beside and over one another, captured calls and their workspaces,
waits that give up, long sums."""
import pytest
import torch

from test_gpu_adapters import (LoraCase, U, _no_kernel_errors, assert_within, mixed_ids, normal, packed,  # noqa: F401
                               rng, segment_ids)
from w8_a8_quantized_b200 import aq

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ buffers

@pytest.mark.parametrize("M", [9, 300])
def test_rows_side_by_side_in_one_buffer(M):
    """Inputs and outputs as column ranges of one buffer give the bits of separate tensors."""
    N, K, F = 256, 384, 512
    c = LoraCase(M, N, K, [8, 24], mixed_ids(M, 2, M), seed=M)
    s = torch.empty(M, 24, device="cuda")
    y = normal(rng(1), M, N)
    want = aq.aq_lora_apply(c.ad, c.x, c.ids, y, s=s)
    buf = torch.zeros(M, K + 2 * N + K, dtype=torch.bfloat16, device="cuda")
    x, y2, out, dx = buf[:, :K], buf[:, K:K + N], buf[:, K + N:K + 2 * N], buf[:, K + 2 * N:]
    x.copy_(c.x), y2.copy_(y)
    assert torch.equal(aq.aq_lora_apply(c.ad, x, c.ids, y2, out=out), want)
    dy = y2.copy_(c.dy)
    want = aq.aq_lora_backward(c.ad, c.dy, c.ids, s, c.x)
    got = aq.aq_lora_backward(c.ad, dy, c.ids, s, x, dx=dx)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    w, _ = packed(N, K, 128, 0.5, 2)
    assert torch.equal(aq.aq_linear_backward(w, dy, out=dx), aq.aq_linear_backward(w, c.dy))
    both = normal(rng(3), M, 2 * F)
    kept = aq.aq_silu_mul_quant(both[:, :F], both[:, F:], keep=True)
    want = aq.aq_silu_mul_quant(both[:, :F].contiguous(), both[:, F:].contiguous(), keep=True)
    assert all(torch.equal(p, q) for p, q in zip(kept, want))
    grads = torch.zeros(M, 3 * F, dtype=torch.bfloat16, device="cuda")
    grads[:, 2 * F:] = normal(rng(4), M, F, scale=0.01)
    want = aq.aq_silu_mul_backward(grads[:, 2 * F:].contiguous(), *kept[2:])
    got = aq.aq_silu_mul_backward(grads[:, 2 * F:], *kept[2:], dgate=grads[:, :F], dup=grads[:, F:2 * F])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_outputs_over_inputs_are_refused():
    M, N = 130, 256
    c = LoraCase(M, N, N, [8], segment_ids(M, 1, 1), seed=5)
    s = torch.empty(M, 8, device="cuda")
    aq.aq_lora_apply(c.ad, c.x, c.ids, s=s)
    w, _ = packed(N, N, 128, 0.5, 2)
    dy, x = c.dy.clone(), c.x.clone()
    for call in (lambda: aq.aq_lora_backward(c.ad, dy, c.ids, s, x, add=dy, dx=dy),
                 lambda: aq.aq_lora_backward(c.ad, dy, c.ids, s, x, dx=dy),
                 lambda: aq.aq_lora_backward(c.ad, dy, c.ids, s, x, dx=x),
                 lambda: aq.aq_linear_backward(w, dy, add=dy, out=dy),
                 lambda: aq.aq_linear_backward(w, dy, out=dy),
                 lambda: aq.aq_lora_apply(c.ad, x, c.ids, out=x)):
        with pytest.raises(aq.AqError):
            call()
    assert torch.equal(dy, c.dy) and torch.equal(x, c.x)
