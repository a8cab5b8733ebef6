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
    where = torch.device("cuda", 0)

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return self.where


def _cuda(t):
    return t.as_subclass(_Cuda)


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
