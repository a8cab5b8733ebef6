"""opts.check of the attention calls: a sound call returns AK_OK and the bits of the call without it, whatever limit of
the device-side waits it is given."""
from __future__ import annotations

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 64)])
@pytest.mark.parametrize("windows", [0, 1, 4])
@pytest.mark.parametrize("limit", [0, 1])
def test_a_checked_call_ends_well(dtype, dim, windows, limit):
    """A limit of 1 ns is below any copy's latency: the kernel waits for its own work as long as that takes."""
    torch.manual_seed(dim + windows)
    t, h, n = 700, 2, 3
    q, k, v, do = (torch.randn(t, h, dim, device="cuda").to(dtype) for _ in range(4))
    ld = -torch.rand(h, device="cuda")
    off = torch.tensor([0, 300, 301, t], dtype=torch.int32, device="cuda")
    s0, ds = torch.randn(2, n, h, dim, dim, device="cuda")
    same = dict(offsets=off, state=s0)
    plain, checked = dict(target_blocks=windows), dict(target_blocks=windows, check=True, wait_limit_ns=limit)
    for call in (lambda o: ak.ak_linear_attention(q, k, v, ld, final_state=True, opts=o, **same),
                 lambda o: ak.ak_linear_attention_backward(do, q, k, v, ld, dstate_out=ds, opts=o, **same)):
        for a, b in zip(call(plain), call(checked)):
            assert torch.isfinite(b).all() and torch.equal(a, b)
    one = lambda o: ak.ak_linear_attention_step(q[:n], k[:n], v[:n], ld, s0.clone(), opts=o)
    assert torch.equal(one(None), one(dict(check=True)))


def test_the_other_sequence_operators_with_check():
    i = torch.tensor([3, 0, 5], dtype=torch.int32, device="cuda")
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    r = ak.ak_batch_layout(torch.zeros_like(i), i, table, torch.arange(4, dtype=torch.int32, device="cuda"), block_size=4,
                           max_tokens=8, opts=dict(check=True))
    assert r.offsets.tolist() == [0, 3, 3, 8] and r.counts.tolist() == [8, 3]
    p = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]], device="cuda")
    t, a = ak.ak_verify_drafts(p, torch.ones(1, 1, dtype=torch.int32, device="cuda"), torch.full((1, 1), 0.5, device="cuda"),
                               torch.ones(1, 2, device="cuda"), opts=dict(check=True))
    assert t.tolist() == [[1, 0]] and a.tolist() == [1]
