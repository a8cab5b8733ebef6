"""ak_linear_attention in a training loop: what autograd records against the backward entry point, bit for bit."""
from __future__ import annotations

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dim", [(torch.float32, 64), (torch.bfloat16, 128), (torch.bfloat16, 80)])
@pytest.mark.parametrize("with_state", [False, True])
def test_recorded_gradients_are_those_of_the_backward_call(dtype, dim, with_state):
    torch.manual_seed(1)
    t, h, n = 200, 3, 2
    w = torch.randn(t, 3 * h * dim, device="cuda", dtype=dtype).requires_grad_()  # a packed projection's output
    ld = -torch.rand(h, device="cuda")
    off = torch.tensor([0, 130, t], dtype=torch.int32, device="cuda")
    s0 = torch.randn(n, h, dim, dim, device="cuda").requires_grad_() if with_state else None
    do, ds = torch.randn(t, h, dim, device="cuda").to(dtype), torch.randn(n, h, dim, dim, device="cuda")
    q, k, v = w.view(t, 3, h, dim).unbind(1)
    o, final = ak.ak_linear_attention(q, k, v, ld, offsets=off, state=s0, scale=0.3, final_state=with_state)
    inputs = [w] + ([s0] if with_state else [])
    got = torch.autograd.grad([o] + ([final] if with_state else []), inputs, [do] + ([ds] if with_state else []))
    with torch.no_grad():
        # (a call that is asked for its final state carries it more exactly, and its outputs round otherwise)
        plain, _ = ak.ak_linear_attention(q, k, v, ld, offsets=off, state=s0, scale=0.3, final_state=with_state)
        dq, dk, dv, d0 = ak.ak_linear_attention_backward(do, q, k, v, ld, offsets=off, state=s0, scale=0.3,
                                                         dstate_out=ds if with_state else None)
    assert torch.equal(o, plain) and not plain.requires_grad
    assert torch.equal(got[0], torch.stack([dq, dk, dv], 1).reshape(t, -1))
    if with_state:
        assert torch.equal(got[1], d0)


def test_a_step_of_gradient_descent_reaches_the_weights():
    """A key head shared by all query heads, a loss of a sum (a gradient with strides of zero)."""
    torch.manual_seed(2)
    t, h, d = 90, 4, 64
    q, v = (torch.randn(t, h, d, device="cuda") for _ in range(2))
    k = torch.randn(t, 1, d, device="cuda", requires_grad=True)
    ld = torch.full((h,), -0.1, device="cuda")
    o, _ = ak.ak_linear_attention(q, k.expand(t, h, d), v, ld)
    o.sum().backward()
    _, dk, _, _ = ak.ak_linear_attention_backward(torch.ones_like(o), q, k.detach().expand(t, h, d), v, ld)
    assert torch.equal(k.grad, dk.sum(1, keepdim=True))
    pool = torch.zeros(t, h, d, d, device="cuda")
    with pytest.raises(RuntimeError, match="no gradient"):
        ak.ak_linear_attention_step(q.requires_grad_(), v, v, ld, pool).sum().backward()
    assert not pool.requires_grad
