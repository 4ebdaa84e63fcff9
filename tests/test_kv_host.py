"""The paged cache's calls without a GPU: what they refuse before any launch, what
they size, and the reference that the GPU tests compare with."""

import ctypes

import numpy as np
import pytest
import torch

import kv_reference as R
from bit_plane_kv_scan_b200 import build as fbuild
from bit_plane_kv_scan_b200 import fathom as F


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return F.lib()


def _cache(**kw):
    a = dict(k=None, v=None, k_scale=None, v_scale=None, dtype=F.BF16, num_pages=100, page_tokens=64,
             h_kv=8, d=128)
    a.update(kw)
    return F.KvCacheArgs(**a)


def _batch(**kw):
    a = dict(page_table=None, seq_len=None, q_start=None, num_seqs=4, table_width=16, num_rows=4,
             max_rows=1, max_len=1024)
    a.update(kw)
    return F.KvBatchArgs(**a)


def _attn(cache=None, batch=None, **kw):
    a = dict(cache=cache or _cache(), batch=batch or _batch(), q=None, q_dtype=F.BF16, h_q=32, q_stride=0,
             softmax_scale=0.1, window=0, sinks=0, out=None, lse=None)
    a.update(kw)
    return F.KvAttentionArgs(**a)


def _app(cache=None, batch=None, **kw):
    a = dict(cache=cache or _cache(), batch=batch or _batch(), k=None, v=None, kv_dtype=F.BF16, k_stride=0,
             v_stride=0, q=None, q_out=None, q_dtype=F.BF16, h_q=32, q_stride=0, inv_freq=None,
             rotary_pairs=0, interleaved=0)
    a.update(kw)
    return F.KvAppendArgs(**a)


SHAPES = [
    (dict(dtype=F.F32), {}, F.ERR_INVALID_ARGUMENT, b"dtype"),
    (dict(dtype=9), {}, F.ERR_INVALID_ARGUMENT, b"dtype"),
    (dict(d=100), {}, F.ERR_UNSUPPORTED, b"d="),
    (dict(d=288), {}, F.ERR_UNSUPPORTED, b"d="),
    (dict(h_kv=0), {}, F.ERR_INVALID_ARGUMENT, b"h_kv"),
    (dict(num_pages=0), {}, F.ERR_INVALID_ARGUMENT, b"num_pages"),
    (dict(page_tokens=0), {}, F.ERR_INVALID_ARGUMENT, b"page_tokens"),
    (dict(page_tokens=24), {}, F.ERR_INVALID_ARGUMENT, b"page_tokens"),
    ({}, dict(num_seqs=-1), F.ERR_INVALID_ARGUMENT, b"num_seqs"),
    ({}, dict(table_width=-1), F.ERR_INVALID_ARGUMENT, b"table_width"),
    ({}, dict(num_rows=-1), F.ERR_INVALID_ARGUMENT, b"num_rows"),
    ({}, dict(max_rows=5), F.ERR_INVALID_ARGUMENT, b"max_rows"),
    ({}, dict(max_len=-1), F.ERR_INVALID_ARGUMENT, b"max_len"),
    ({}, dict(max_len=(1 << 30) + 1), F.ERR_INVALID_ARGUMENT, b"max_len"),
    ({}, dict(num_rows=5), F.ERR_INVALID_ARGUMENT, b"q_start"),
    ({}, {}, F.ERR_INVALID_ARGUMENT, b"cache.k"),
]


@pytest.mark.parametrize("cache,batch,status,word", SHAPES)
def test_both_calls_refuse_bad_shapes(L, cache, batch, status, word):
    a = _attn(_cache(**cache), _batch(**batch))
    assert L.fathom_kv_attention(ctypes.byref(a), None, 0, None) == status
    assert word in L.fathom_last_error()
    if word != b"cache.k":
        assert L.fathom_kv_attention_workspace_size(ctypes.byref(a)) == 0
    p = _app(_cache(**cache), _batch(**batch))
    assert L.fathom_kv_append(ctypes.byref(p), None) == status
    assert word in L.fathom_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(h_q=30), b"h_q"), (dict(h_q=0), b"h_q"), (dict(q_dtype=F.E4M3), b"dtype"),
    (dict(q_stride=100), b"stride"), (dict(softmax_scale=float("nan")), b"softmax_scale"),
    (dict(window=-1), b"window"), (dict(sinks=-1), b"sinks")])
def test_attention_refuses(L, kw, word):
    a = _attn(**kw)
    assert L.fathom_kv_attention(ctypes.byref(a), None, 0, None) == F.ERR_INVALID_ARGUMENT
    assert word in L.fathom_last_error()
    assert L.fathom_kv_attention_workspace_size(ctypes.byref(a)) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(kv_dtype=F.E4M3), b"dtype"), (dict(k_stride=8), b"stride"), (dict(v_stride=-1024), b"stride"),
    (dict(rotary_pairs=65, inv_freq=16), b"rotary_pairs"), (dict(rotary_pairs=-1), b"rotary_pairs"),
    (dict(rotary_pairs=8), b"inv_freq"), (dict(q=16, h_q=0), b"h_q"), (dict(q=16, q_dtype=7), b"dtype"),
    (dict(q=16, q_stride=5), b"stride")])
def test_append_refuses(L, kw, word):
    a = _app(**kw)
    assert L.fathom_kv_append(ctypes.byref(a), None) == F.ERR_INVALID_ARGUMENT
    assert word in L.fathom_last_error()


def test_null_and_host_pointers_are_refused(L):
    assert L.fathom_kv_attention(None, None, 0, None) == F.ERR_INVALID_ARGUMENT
    assert L.fathom_kv_append(None, None) == F.ERR_INVALID_ARGUMENT
    assert L.fathom_kv_attention_workspace_size(None) == 0
    buf = ctypes.create_string_buffer(4096)
    a = _app(_cache(k=ctypes.addressof(buf)))
    assert L.fathom_kv_append(ctypes.byref(a), None) == F.ERR_INVALID_ARGUMENT
    assert b"device pointer" in L.fathom_last_error()


def test_nothing_to_do_is_ok(L):
    for batch in (_batch(num_seqs=0, num_rows=0, max_rows=0), _batch(num_seqs=0, num_rows=0, max_rows=0,
                                                                   max_len=0, table_width=0),
                  _batch(q_start=16, num_rows=9, max_rows=0)):
        assert L.fathom_kv_append(ctypes.byref(_app(batch=batch)), None) == F.OK
        assert L.fathom_kv_attention(ctypes.byref(_attn(batch=batch)), None, 0, None) == F.OK


def test_workspace_size_follows_the_bounds(L):
    def size(**kw):
        attn = {k: kw.pop(k) for k in ("window", "sinks") if k in kw}
        return L.fathom_kv_attention_workspace_size(ctypes.byref(_attn(batch=_batch(**kw), **attn)))
    assert size() >= 256 and size() % 256 == 0
    long = size(max_len=1 << 20, table_width=1 << 14)
    assert long > 4 * 32 * 128 * 4  # split: partial results
    assert size(max_len=1 << 20, table_width=1 << 14, window=128) < long
    assert size(max_len=0) >= 256


def test_python_checks():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k = z(4, 2, 32, 64)
    with pytest.raises(TypeError):
        F.KVCache(k.float(), k.float())
    with pytest.raises(ValueError):
        F.KVCache(k, z(4, 2, 32, 32))
    with pytest.raises(ValueError):
        F.KVCache(z(4, 2, 24, 64), z(4, 2, 24, 64))
    with pytest.raises(ValueError):
        F.KVCache(k.transpose(0, 1), k.transpose(0, 1))
    with pytest.raises(TypeError):
        F.KVCache(k, k, z(4, 2, 2, t=torch.uint8), z(4, 2, 2, t=torch.uint8))
    k8 = z(4, 2, 32, 64, t=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(TypeError):
        F.KVCache(k8, k8)
    with pytest.raises(ValueError):
        F.KVCache(k8, k8, z(4, 2, 1, t=torch.uint8), z(4, 2, 1, t=torch.uint8))
    cache = F.KVCache(k, k.clone())
    assert F.KVCache(k8, k8.clone(), *(z(4, 2, 2, t=torch.uint8) for _ in range(2))).args.dtype == F.E4M3
    with pytest.raises(TypeError):
        F.KVBatch(torch.zeros((2, 4), dtype=torch.int64), i32(2))
    with pytest.raises(ValueError):
        F.KVBatch(i32(2, 4), i32(3))
    with pytest.raises(ValueError):
        F.KVBatch(i32(2, 4), i32(2), i32(2), num_rows=2)
    with pytest.raises(ValueError):
        F.KVBatch(i32(2, 4), i32(2), i32(3))
    batch = F.KVBatch(i32(2, 4), i32(2))
    assert (batch.num_rows, batch.max_rows, batch.args_for(cache).max_len) == (2, 1, 128)
    with pytest.raises(ValueError):
        F.kv_attention(cache, batch, z(3, 4, 64))
    with pytest.raises(ValueError):
        F.kv_attention(cache, batch, z(2, 4, 128)[..., ::2])
    with pytest.raises(ValueError):
        F.kv_append(cache, batch, z(2, 3, 64), z(2, 3, 64))
    with pytest.raises(ValueError):
        F.kv_append(cache, batch, z(2, 2, 64), z(2, 2, 64, t=torch.float32))
    with pytest.raises(TypeError):
        F.kv_append(cache, batch, z(2, 2, 64), z(2, 2, 64), inv_freq=z(32, t=torch.float64))


# ------------------------------------------------------- the reference's pins --

def test_reference_codes_are_the_nearest():
    x = np.random.default_rng(0).normal(size=4000) * 2.0 ** np.random.default_rng(1).integers(-12, 10, 4000)
    got = R.e4m3_value(R.e4m3_code(x))
    every = R.e4m3_value(np.arange(256, dtype=np.uint8))
    every = every[np.isfinite(every)]
    best = np.abs(every[None] - np.clip(x, -448, 448)[:, None]).min(1)
    np.testing.assert_array_equal(np.abs(got - np.clip(x, -448, 448)), best)
    # ties go to the even code: 1.0625 lies between 1 (code 0x38) and 1.125 (0x39)
    assert R.e4m3_code(np.array([1.0625, 1.1875, -1.0625])).tolist() == [0x38, 0x3a, 0xb8]


def test_reference_scale_byte():
    # 256 * 2^(x - 127) just holds the largest element
    for big, x in ((256.0, 127), (256.5, 128), (128.0, 126), (1.0, 119), (0.0, 8), (1e-38, 8), (3e38, 246)):
        assert R.block_byte(big) == x


def test_reference_rotation_by_hand():
    # a quarter turn takes (1, 0) to (0, 1); dimension 4.. stay
    x = np.array([[[1.0, 2.0, 0.0, 0.0, 7.0, 8.0]]])
    f = [np.pi / 2, np.pi]
    out, _ = R.rotate(x, [1], f, False)
    np.testing.assert_allclose(out[0, 0], [0, -2, 1, 0, 7, 8], atol=1e-12)
    out, _ = R.rotate(x, [1], f, True)
    np.testing.assert_allclose(out[0, 0], [-2, 1, 0, 0, 7, 8], atol=1e-12)


def test_reference_attention_by_hand():
    # two tokens, equal scores: the mean; with window 1 and no sinks the second sees itself alone
    k = torch.zeros((1, 1, 16, 32), dtype=torch.bfloat16)
    v = k.clone()
    v[0, 0, 0], v[0, 0, 1] = 1.0, 3.0
    c = R.Cache(k, v)
    q = np.ones((1, 1, 32))
    out, lse, _, _ = R.attention(c, [[0]], [(0, 1, 2)], q, 1.0)
    assert out[0, 0, 0] == 2.0 and lse[0, 0] == np.log(2.0)
    out, lse, _, _ = R.attention(c, [[0]], [(0, 1, 2)], q, 1.0, window=1)
    assert out[0, 0, 0] == 3.0 and lse[0, 0] == 0.0
    out, lse, _, _ = R.attention(c, [[0]], [(0, 1, 2)], q, 1.0, window=1, sinks=1)
    assert out[0, 0, 0] == 2.0
    out, lse, _, _ = R.attention(c, [[5]], [(0, 1, 2)], q, 1.0)
    assert out[0, 0, 0] == 0.0 and np.isneginf(lse[0, 0])
