"""What the sequence operators' binding hands to the C entry points, on the host: tensors that call themselves CUDA
tensors stand in for device memory, and nothing is launched."""
from __future__ import annotations

import weakref

import pytest
import torch

import mapreduce_prefix_scan_gb300 as ak
from mapreduce_prefix_scan_gb300 import sequence


class _Cuda(torch.Tensor):
    """Host memory under a device's name."""
    index = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


class _OtherCuda(_Cuda):
    index = 1


def _cuda(t):
    return t.as_subclass(_Cuda)


STREAM_OF = sequence._stream_of


class _Library:
    """Records every entry point's arguments; `sizes` are the answers of the workspace queries."""

    def __init__(self, sizes=256, during=None):
        self.calls, self.sizes, self.during = {}, sizes, during

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("workspace_size"):
                out = args[-1]
                (out._obj if hasattr(out, "_obj") else out).value = self.sizes
            else:
                self.calls[name] = args
                if self.during:
                    self.during(name, args)
            return 0
        return entry


@pytest.fixture
def host(monkeypatch):
    """The binding over host memory; the fixture's value installs a stand-in for the library."""
    monkeypatch.setattr(sequence, "_empty", lambda size, dtype, device, stream: _cuda(torch.empty(size, dtype=dtype)))
    monkeypatch.setattr(sequence, "_stream_of", lambda stream, t: 0)
    # (autograd's engine hands on plain tensors)
    backward, named = sequence.ak_linear_attention_backward, lambda t: None if t is None else _cuda(t)
    monkeypatch.setattr(sequence, "ak_linear_attention_backward", lambda do, *a, dstate_out=None, **kw: backward(
        named(do), *a, dstate_out=named(dstate_out), **kw))

    def use(library):
        monkeypatch.setattr(sequence._abi, "load", lambda: library)
        return library
    return use


def _int(*shape):
    return _cuda(torch.zeros(shape, dtype=torch.int32))


def _layout(table, n, **kw):
    return ak.ak_batch_layout(_int(n), _int(n), table, _int(4), block_size=16, max_tokens=8, **kw)


OVERLAPPING = {
    "one row for all": lambda n, w: _cuda(torch.full((1, w), -1, dtype=torch.int32)).expand(n, w),
    "windows of one row": lambda n, w: _cuda(torch.zeros(n + w, dtype=torch.int32)).unfold(0, w, 1)[:n],
}


@pytest.mark.parametrize("rows", OVERLAPPING)
def test_a_table_whose_rows_overlap_is_not_given_another_stride(host, rows):
    """The C entry point has to see the stride that it refuses (below the width: test_batch_layout_refusals)."""
    L = host(_Library())
    table = OVERLAPPING[rows](5, 7)
    _layout(table, 5)
    assert L.calls["ak_batch_layout"][4] == table.stride(0) < 7


def test_table_strides_are_handed_over_as_they_are(host):
    """A single row's stride says nothing: its width stands for it."""
    L = host(_Library())
    wide = _int(5, 9)
    for table, stride in ((wide[:, 1:8], 9), (_int(5, 7), 7), (_int(1, 7), 7), (wide[:1, :4], 4), (wide[:, :1], 9)):
        _layout(table, table.shape[0])
        assert L.calls["ak_batch_layout"][4] == stride and L.calls["ak_batch_layout"][5] == table.shape[1]


def _attention(t=70, h=2, d=64, dtype=torch.float32):
    rows = lambda: _cuda(torch.zeros(t, h, d, dtype=dtype))
    return rows(), rows(), rows(), _cuda(torch.zeros(h))


CALLS = {
    "ak_batch_layout": lambda: _layout(_int(5000, 3), 5000),
    "ak_linear_attention": lambda: ak.ak_linear_attention(*_attention()),
    "ak_linear_attention_backward": lambda: ak.ak_linear_attention_backward(_attention()[0], *_attention()),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_workspace_lives_until_the_entry_point_returns(host, monkeypatch, name):
    """It is released to the allocator only after every launch has been queued."""
    made, alive = [], []

    def empty(size, dtype, device, stream):
        t = _cuda(torch.empty(size, dtype=dtype))
        if dtype is torch.uint8:
            made.append((t.data_ptr(), weakref.ref(t)))
        return t

    monkeypatch.setattr(sequence, "_empty", empty)
    host(_Library(sizes=4096, during=lambda _, args: alive.extend(ref() is not None for p, ref in made if p in args)))
    CALLS[name]()
    assert alive == [True]


def _verify(n=3, k=2, vocab=11, **kw):
    a = dict(target_probs=torch.zeros(n, k + 1, vocab), draft_tokens=torch.zeros(n, k, dtype=torch.int32),
             uniform=torch.zeros(n, k), noise=torch.ones(n, vocab), draft_probs=torch.zeros(n, k, vocab),
             draft_counts=torch.zeros(n, dtype=torch.int32), tokens=torch.zeros(n, k + 1, dtype=torch.int32),
             accepted=torch.zeros(n, dtype=torch.int32))
    return {name: kw.get(name, _cuda(x)) for name, x in a.items()}


def test_arrays_of_another_shape_with_as_many_elements_are_refused(host):
    """[drafts, requests] in place of [requests, drafts] would be read in the wrong order."""
    L = host(_Library())
    for name, shape in (("uniform", (2, 3)), ("tokens", (1, 9)), ("uniform", (3, 2, 1)), ("tokens", (9, 1))):
        good = _verify()[name]
        with pytest.raises(ValueError):
            ak.ak_verify_drafts(**_verify(**{name: good.reshape(shape)}))
    assert not L.calls
    ak.ak_verify_drafts(**_verify())
    ak.ak_verify_drafts(**_verify(uniform=_cuda(torch.zeros(6)), tokens=_cuda(torch.zeros(9, dtype=torch.int32))))  # flat
    ak.ak_verify_drafts(**_verify(k=1, uniform=_cuda(torch.zeros(1, 3))))  # one order only
    assert L.calls


def _named_calls():
    """Each entry point with all of its tensor arguments by name."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    rows, state = (lambda: torch.zeros(9, 2, 64)), (lambda: torch.zeros(2, 2, 64, 64))
    qkv = lambda: dict(q=rows(), k=rows(), v=rows(), log_decay=torch.zeros(2))
    ws = lambda: torch.zeros(4096, dtype=torch.uint8)
    return {
        "ak_batch_layout": (dict(ctx_lens=i32(3), new_lens=i32(3), block_table=i32(3, 4), free_blocks=i32(5), offsets=i32(4),
                                 slots=torch.zeros(8, dtype=torch.int64), positions=i32(8), requests=i32(8), counts=i32(2),
                                 workspace=ws()), dict(block_size=16, max_tokens=8)),
        "ak_verify_drafts": (_verify(), {}),
        "ak_linear_attention": (dict(qkv(), offsets=i32(3), state=state(), out=rows(), state_out=state(), workspace=ws()), {}),
        "ak_linear_attention_backward": (dict(qkv(), do=rows(), offsets=i32(3), state=state(), dstate_out=state(), dq=rows(),
                                              dk=rows(), dv=rows(), dstate=state(), workspace=ws()), {}),
        "ak_linear_attention_step": (dict(qkv(), state=torch.zeros(9, 2, 64, 64), slots=i32(9), out=rows()), {}),
    }


ARGUMENTS = [(call, name) for call, (tensors, _) in _named_calls().items() for name in tensors]


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_an_argument_on_another_device_is_refused(host, call, name):
    L = host(_Library())
    tensors, rest = _named_calls()[call]
    tensors = {n: _cuda(t) for n, t in tensors.items()}
    getattr(ak, call)(**tensors, **rest)  # all on one device
    assert L.calls.pop(call)
    for stray in (tensors[name].as_subclass(torch.Tensor), tensors[name].as_subclass(_OtherCuda)):
        with pytest.raises(ValueError):
            getattr(ak, call)(**dict(tensors, **{name: stray}), **rest)
    assert not L.calls


def test_a_workspace_that_is_not_its_own_memory_is_refused(host):
    L = host(_Library(sizes=4096))
    for ws in (_cuda(torch.zeros(1, dtype=torch.uint8)).expand(4096), _cuda(torch.zeros(8192, dtype=torch.uint8))[::2]):
        with pytest.raises(ValueError):
            ak.ak_linear_attention(*_attention(), workspace=ws)
    assert not L.calls
    ak.ak_linear_attention(*_attention(), workspace=_cuda(torch.zeros(4096, dtype=torch.uint8)))
    assert L.calls


def _backward(*results):
    """A gradient of ones, with strides of zero as that of a sum has."""
    torch.autograd.backward(results, [_cuda(torch.ones(1)).expand(x.shape) for x in results])


def _with_grad(*tensors):
    return [t.requires_grad_() for t in tensors]


def test_gradients_are_recorded(host):
    """A call on tensors that ask for gradients runs the backward entry point on its inputs, its output's gradient and
    its final state's."""
    L = host(_Library(sizes=4096))
    q, k, v, ld = _attention()
    _with_grad(q, k, v)
    state = _cuda(torch.zeros(1, 2, 64, 64)).requires_grad_()
    o, final = ak.ak_linear_attention(q, k, v, ld, state=state, final_state=True, scale=0.5, max_len=64)
    assert o.requires_grad and final.requires_grad and "ak_linear_attention_backward" not in L.calls
    _backward(o, final)
    a = L.calls["ak_linear_attention_backward"]
    assert (a[0].scale, a[0].max_len, a[0].tokens) == (0.5, 64, 70) and a[1].token_stride == 128
    assert [x.data for x in a[2:5]] == [x.data_ptr() for x in (q, k, v)] and a[5] == ld.data_ptr() and a[7] == state.data_ptr()
    assert a[8] is not None and a[12] is not None
    assert [x.data for x in a[9:12]] == [x.grad.data_ptr() for x in (q, k, v)]
    assert all(x.grad.shape == x.shape for x in (q, k, v, state))
    # an output alone; a final state alone
    for pick in (0, 1):
        L.calls.clear()
        got = ak.ak_linear_attention(q, k, v, ld, final_state=True)
        _backward(got[pick])
        assert L.calls["ak_linear_attention_backward"][1].data and (L.calls["ak_linear_attention_backward"][8] is None) == (pick == 0)


def test_a_shared_head_gets_the_sum_of_its_gradients(host):
    host(_Library())
    q, k, v, ld = _attention(h=4)
    one = _cuda(torch.zeros(70, 1, 64)).requires_grad_()
    o, _ = ak.ak_linear_attention(q, one.expand(70, 4, 64), v, ld)
    _backward(o)
    assert one.grad.shape == one.shape


def test_what_has_no_gradient_says_so(host):
    host(_Library())
    q, k, v, ld = _attention()
    _with_grad(q, k, v)
    out, state = _cuda(torch.empty(70, 2, 64)), _cuda(torch.zeros(1, 2, 64, 64))
    pool = _cuda(torch.zeros(70, 2, 64, 64))
    for make in (lambda: ak.ak_linear_attention(q, k, v, ld, out=out)[0],
                 lambda: ak.ak_linear_attention(q, k, v, ld, state=state, state_out=state)[0],
                 lambda: ak.ak_linear_attention(q, k, v, ld, stream=7)[0],
                 lambda: ak.ak_linear_attention(q, k, v, ld.clone().requires_grad_())[0],
                 lambda: ak.ak_linear_attention_step(q, k, v, ld, pool),
                 lambda: ak.ak_linear_attention_step(q, k, v, ld, pool, out=out)):
        o = make()
        assert o.requires_grad
        with pytest.raises(RuntimeError, match="gradient"):
            _backward(o)
    assert not (out.requires_grad or state.requires_grad or pool.requires_grad)
    # without a record nothing changes
    with torch.no_grad():
        assert ak.ak_linear_attention(q, k, v, ld, out=out)[0] is out
        assert ak.ak_linear_attention_step(q, k, v, ld, pool, out=out) is out
    assert ak.ak_linear_attention(*_attention(), out=out)[0] is out


@pytest.mark.parametrize("call", _named_calls())
@pytest.mark.parametrize("current,refused", [(0, False), (1, True)])
def test_tensors_of_a_device_that_is_not_current_are_refused(host, monkeypatch, call, current, refused):
    """The kernels run on the current device, whatever stream they are given."""
    L = host(_Library())
    monkeypatch.setattr(sequence, "_stream_of", STREAM_OF)
    monkeypatch.setattr(sequence, "_device", lambda: current, raising=False)
    tensors, rest = _named_calls()[call]
    tensors = {n: _cuda(t) for n, t in tensors.items()}
    if refused:
        with pytest.raises(ValueError, match="current CUDA device"):
            getattr(ak, call)(**tensors, **rest, stream=7)
    else:
        getattr(ak, call)(**tensors, **rest, stream=7)
    assert (call in L.calls) != refused
