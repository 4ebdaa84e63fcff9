"""fathom_kv_attention refuses outputs that overlap its queries or each other (no GPU: the
check is on addresses alone and comes before anything is looked at there)."""

import ctypes

import pytest

from bit_plane_kv_scan_b200 import build as fbuild
from bit_plane_kv_scan_b200 import fathom as F
from test_kv_host import _attn, _batch

Q = 1 << 20
ROW = 32 * 128 * 2  # bytes of a row of 32 heads, bf16


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return F.lib()


def _call(L, stride=0, **kw):
    a = _attn(batch=_batch(), q=Q, q_stride=stride, **kw)  # 4 rows
    assert L.fathom_kv_attention(ctypes.byref(a), None, 0, None) == F.ERR_INVALID_ARGUMENT
    return L.fathom_last_error()


@pytest.mark.parametrize("at", [Q, Q - 16, Q + 16, Q - 4 * ROW + 16, Q + 4 * ROW - 16])
def test_out_over_q(L, at):
    assert b"out overlaps q" in _call(L, out=at)


@pytest.mark.parametrize("at", [Q, Q - 4 * 32 * 4 + 4, Q + 4 * ROW - 4])
def test_lse_over_q(L, at):
    assert b"lse overlaps q" in _call(L, out=Q + (1 << 20), lse=at)


def test_lse_over_out(L):
    out = Q + (1 << 20)
    assert b"lse overlaps out" in _call(L, out=out, lse=out + 4 * ROW - 4)


def test_strided_queries_reach_to_their_last_row(L):
    assert b"out overlaps q" in _call(L, stride=5 * ROW // 2, out=Q + 16 * ROW - 16)
    assert b"overlaps" not in _call(L, stride=5 * ROW // 2, out=Q + 16 * ROW)


def test_neighbours_are_no_overlap(L):
    for out, lse in ((Q + 4 * ROW, Q - 4 * 32 * 4), (Q - 4 * ROW, Q + 4 * ROW)):
        assert b"overlaps" not in _call(L, out=out, lse=lse)  # (the cache's pointer is what it refuses)
