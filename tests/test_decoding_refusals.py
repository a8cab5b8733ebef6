"""Outputs that lie in inputs other than the entry points allow: refused on the host, before anything touches a device."""
from __future__ import annotations

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


def test_a_beam_step_in_its_own_tensors_keeps_as_many_beams(L):  # noqa: F811
    """With another number of them one request's outputs lie in another's inputs."""
    from mapreduce_prefix_scan_gb300._abi import AK_ERR_INVALID_ARG as INV

    def call(keep, s=0x2000, d=0x3001, m=0x4000, os=0x5000, od=0x8001, ol=0x9000):
        return L.ak_beam_select(0x100000, 400, 100, 0, 2, 4, 100, keep, s, d, m, 5, 0.5, os, 0x6000, 0x7000, od, ol, None, None)

    for keep in (1, 3, 5, 32):
        assert call(keep, os=0x2000) == INV and call(keep, od=0x3001) == INV and call(keep, ol=0x4000) == INV
