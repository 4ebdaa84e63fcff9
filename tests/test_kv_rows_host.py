"""Rows that the paged cache's calls refuse before the library sees them, and handles whose
fields stay (no GPU)."""

import pytest
import torch

from bit_plane_kv_scan_b200 import fathom as F


def _setup(rows):
    k = torch.zeros((4, 2, 32, 64), dtype=torch.bfloat16)
    cache = F.KVCache(k, k.clone())
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return cache, F.KVBatch(i32(rows, 4), i32(rows))


def _broadcast(rows, heads):
    return torch.zeros((1, heads, 64), dtype=torch.bfloat16).expand(rows, heads, 64)


def _overlapping(rows, heads):
    return torch.zeros(4096, dtype=torch.bfloat16).as_strided((rows, heads, 64), (64, 64, 1))


@pytest.mark.parametrize("make", [_broadcast, _overlapping])
@pytest.mark.parametrize("which", ["k", "v", "q"])
def test_append_refuses_rows_that_overlap(which, make):
    cache, batch = _setup(5)
    x = {n: torch.zeros((5, h, 64), dtype=torch.bfloat16) for n, h in (("k", 2), ("v", 2), ("q", 8))}
    x[which] = make(5, x[which].shape[1])
    with pytest.raises(ValueError, match="%s: rows overlap" % which):
        F.kv_append(cache, batch, x["k"], x["v"], q=x["q"])


@pytest.mark.parametrize("make", [_broadcast, _overlapping])
def test_attention_refuses_rows_that_overlap(make):
    cache, batch = _setup(5)
    with pytest.raises(ValueError, match="q: rows overlap"):
        F.kv_attention(cache, batch, make(5, 8))


def test_row_strides():
    one = torch.zeros((1, 8, 64))
    assert F._rows_of(one, "q", 1, 64) == 0
    assert F._rows_of(one.expand(1, 8, 64), "q", 1, 64) == 0
    assert F._rows_of(torch.zeros((5, 8, 64)), "q", 5, 64) == 512
    assert F._rows_of(torch.zeros((5, 16, 64))[:, 3:11], "q", 5, 64) == 1024
    assert F._rows_of(torch.zeros((0, 8, 64)), "q", 0, 64) == 0


def test_handles_keep_what_they_were_made_from():
    """The library's arguments are made once: a field that is replaced would not be seen."""
    cache, batch = _setup(5)
    before = batch.args_for(cache)
    for name, value in (("seq_len", torch.ones(5, dtype=torch.int32)), ("page_table", batch.page_table.clone()),
                        ("q_start", torch.arange(6, dtype=torch.int32)), ("num_rows", 4), ("max_rows", 2), ("max_len", 7)):
        with pytest.raises(AttributeError, match="KVBatch.%s is fixed" % name):
            setattr(batch, name, value)
    with pytest.raises(AttributeError, match="KVCache.k is fixed"):
        cache.k = cache.k.clone()
    batch.q_start = None    # what it is
    batch.seq_len += 3      # in place: the same tensor
    assert batch.args_for(cache) is before and before.seq_len == batch.seq_len.data_ptr()
