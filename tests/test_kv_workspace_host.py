"""The attention's workspace follows what a call divides and widens, not its rows or bounds
alone (no GPU)."""

import ctypes

import pytest

from bit_plane_kv_scan_b200 import build as fbuild
from bit_plane_kv_scan_b200 import fathom as F
from test_kv_host import _attn, _batch, _cache

MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return F.lib()


def size(L, rows, max_rows, max_len, seqs=1, dtype=F.BF16, d=128, **kw):
    a = _attn(_cache(dtype=dtype, d=d),
              _batch(num_seqs=seqs, q_start=16, num_rows=rows, max_rows=max_rows, max_len=max_len,
                     table_width=-(-max_len // 64)), **kw)
    n = L.fathom_kv_attention_workspace_size(ctypes.byref(a))
    assert n >= 256, L.fathom_last_error()
    return n


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 100, 1500, 4096, 6000, 8192, 32000, 32700])
@pytest.mark.parametrize("window", [0, 4096])
def test_a_prompt_divides_one_wave_of_units_at_most(L, rows, d, window):
    # 148 blocks of 256 columns (128 beyond 128 dimensions; a decoded token: 4736 of 4), each
    # (d + 2) floats a column, and 4 bytes a mark
    units = -(-rows * 4 // (256 if d <= 128 else 128)) * 8
    assert size(L, rows, rows, 131072, d=d, window=window) <= 148 * 256 * (d + 2) * 4 + 148 * 4 * units + 4096


def test_decoded_tokens_beside_a_long_prompt(L):
    # the few-rows launch leaves results for the columns that it may have, not for the prompt's
    assert size(L, 8193, 8192, 1 << 20, seqs=2) <= 64 * MB
    assert size(L, 64 * 1000 + 63, 64000, 1 << 20, seqs=64) <= 64 * MB


def test_widened_keys_are_those_that_a_window_sees(L):
    # 49 tiles of 128 keys for the window and the rows, 8 KV heads, K and V in bf16: 26 MB
    loose = size(L, 2048, 2048, 1 << 20, dtype=F.E4M3, window=4096)
    assert loose <= 64 * MB
    assert size(L, 2048, 2048, 1 << 20, dtype=F.E4M3, window=4096, sinks=300) > loose
    # where everything is seen: at most 4 GiB, or one pair
    assert size(L, 2048, 2048, 1 << 20, dtype=F.E4M3) <= (4 << 30) + 64 * MB
    assert size(L, 2048, 2048, 1 << 20, dtype=F.E4M3) >= 4 << 30
