"""Outputs that lie in inputs other than the entry points allow: refused on the host, before anything touches a device."""
from __future__ import annotations

import ctypes

import pytest

from test_decoding_abi import L, R, _shape  # noqa: F401


def test_a_recurrence_in_place_has_its_input_rows(L):  # noqa: F811
    """One row of x for all tokens, or rows further apart, and outputs from the same address on: rows would be written
    before they are read."""
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV, ak_rows

    def fwd(x, h, tokens):
        a = _shape(tokens=tokens, seqs=0)
        g = ak_rows(0x800000, 64)
        return L.ak_gated_recurrence(R(a), R(ak_rows(*x)), R(g), 0x2000, None, R(ak_rows(*h)), None, None, None)

    for xs, hs in ((0, 64), (64, 128), (128, 64), (63, 64)):
        assert fwd((0x10000, xs), (0x10000, hs), 100) == INV, (xs, hs)
