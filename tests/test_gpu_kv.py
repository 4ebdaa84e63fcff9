"""The paged cache's calls on the GPU against tests/kv_reference.py (fp64; its
docstring derives the tolerances)."""

import math

import numpy as np
import pytest
import torch

import kv_reference as R

pytestmark = pytest.mark.gpu

F = None
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
# What the weights that meet V are rounded to.  bf16 queries: bf16 (2^-8) where the cache is
# bf16, and in the many-rows kernel, which multiplies in bf16 whatever the cache is; fp16
# (2^-11) in the few-rows kernel over e4m3, so 2^-8 bounds both.  fp32 queries: split, 2^-21.
WEIGHT = {(BF16, BF16): 2.0 ** -8, (F8, BF16): 2.0 ** -8, (BF16, F32): 2.0 ** -21, (F8, F32): 2.0 ** -21}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global F
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import bit_plane_kv_scan_b200 as fb
    from bit_plane_kv_scan_b200 import build
    build.build()
    F = fb
    F.lib()
    yield


def make_cache(rng, pages, page, h_kv, d, dtype):
    """A cache of random values (every page, so that strays show)."""
    if dtype == BF16:
        k, v = (torch.from_numpy(rng.normal(size=(pages, h_kv, page, d)).astype(np.float32)).to(BF16)
                for _ in range(2))
        return F.KVCache(k.cuda(), v.cuda())
    k, v = (torch.from_numpy(rng.normal(size=(pages, h_kv, page, d)).astype(np.float32) * 60).to(F8)
            for _ in range(2))
    s = [torch.from_numpy(rng.integers(118, 124, size=(pages, h_kv, page // 16)).astype(np.uint8))
         for _ in range(2)]
    return F.KVCache(k.cuda(), v.cuda(), s[0].cuda(), s[1].cuda())


def ref_cache(c):
    return R.Cache(c.k, c.v, c.k_scale, c.v_scale)


def make_batch(rng, pages, page, lens, rows=None, width=None, num_rows=None, max_len=None):
    """Pages in random order; rows: new tokens of each sequence (None: one each, no q_start)."""
    width = width or max(1, max(-(-n // page) for n in lens))
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(lens):
        w = -(-n // page)
        table[s, :w] = order[at:at + w]
        at += w
    start = None if rows is None else np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    t = torch.from_numpy(table).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    if rows is None:
        return F.KVBatch(t, n, max_len=max_len), table, R.sequences(lens, None)
    b = F.KVBatch(t, n, torch.from_numpy(start).cuda(), num_rows=num_rows or int(start[-1]),
                  max_rows=max(max(rows), 1), max_len=max_len)
    return b, table, R.sequences(lens, start)


def randn(rng, *shape, dtype=BF16, scale=1.0):
    return torch.from_numpy((rng.normal(size=shape) * scale).astype(np.float32)).to(dtype).cuda()


def check_attention(got, want, what=""):
    out, lse = R.f64(got[0]), R.f64(got[1])
    ref, rl, tol, ltol = want
    held = ~np.isnan(rl)
    fin = held & np.isfinite(rl)
    assert np.isneginf(lse[held & ~fin]).all() and (out[held & ~fin] == 0).all(), what + " empty rows"
    e = np.abs(out[held] - ref[held]) / tol[held].clip(1e-30)
    assert e.max(initial=0) <= 1, "%s: out off by %g tolerances" % (what, e.max())
    e = np.abs(lse[fin] - rl[fin]) / ltol[fin]
    assert e.max(initial=0) <= 1, "%s: lse off by %g tolerances" % (what, e.max())


# ----------------------------------------------------------------- append --

def check_append(before, cache, table, seqs, k, v, inv_freq, interleaved):
    """The cache after the call: what the reference writes, everything else as it was."""
    want = before
    done = want.append(table, seqs, R.f64(k), R.f64(v),
                       None if inv_freq is None else R.f64(inv_freq), interleaved)
    for side in range(2):
        x = (cache.k, cache.v)[side]
        got = R.bytes_of(x) if want.e4m3 else R.f64(x)
        exp = (want.k, want.v)[side]
        if want.e4m3:
            np.testing.assert_array_equal((cache.k_scale, cache.v_scale)[side].cpu().numpy(), want.scales[side])
        for page, slot, val, mag in done[side]:
            rot = R.ROT * mag if side == 0 and inv_freq is not None else 0 * mag
            if not want.e4m3:
                err = np.abs(got[page, :, slot] - val)
                assert (err <= rot + R.half_step(BF16) * np.abs(val)).all(), (side, page, slot, err.max())
            else:
                s = 2.0 ** (want.scales[side][page, :, slot // 16].astype(int) - 127.0)[:, None]
                err = np.abs(R.e4m3_value(got[page, :, slot]) * s - val)
                step = np.maximum(2.0 ** -4 * np.abs(val), 2.0 ** -10 * s)
                assert (err <= (rot * (1 + 2.0 ** -4) + step)).all(), (side, page, slot, err.max())
            exp[page, :, slot] = got[page, :, slot]
        np.testing.assert_array_equal(got, exp)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,h_kv,G,page,lens,rows,pairs,inter,kvt,qt", [
    (128, 8, 4, 64, [100, 1, 17, 640], None, 64, False, BF16, BF16),
    (128, 2, 4, 16, [300, 40, 33], [300, 0, 2], 64, False, BF16, BF16),
    (64, 1, 7, 48, [97, 16, 200, 5], [90, 16, 1, 3], 16, False, F32, F32),
    (96, 3, 1, 32, [70, 70], [33, 15], 48, True, BF16, F32),
    (32, 2, 2, 16, [31], [31], 5, False, BF16, BF16),
    (32, 1, 1, 16, [31, 50], [30, 17], 5, True, F32, BF16),
    (256, 1, 2, 128, [515], [260], 128, False, BF16, BF16),
    (160, 2, 1, 32, [77, 12], [50, 12], 0, False, F32, F32),
])
def test_append(dtype, d, h_kv, G, page, lens, rows, pairs, inter, kvt, qt):
    rng = np.random.default_rng(d + page)
    pages = sum(-(-n // page) for n in lens) + 3
    cache = make_cache(rng, pages, page, h_kv, d, BF16 if dtype == "bf16" else F8)
    batch, table, seqs = make_batch(rng, pages, page, lens, rows)
    T = batch.num_rows
    k, v = (randn(rng, T, h_kv, d, dtype=kvt, scale=3) for _ in range(2))
    q = randn(rng, T, h_kv * G, d, dtype=qt)
    f = torch.from_numpy((1e4 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)).cuda() if pairs else None
    before = ref_cache(cache)
    qo = F.kv_append(cache, batch, k, v, q=q, inv_freq=f, interleaved=inter)
    torch.cuda.synchronize()
    check_append(before, cache, table, seqs, k, v, f, inter)
    pos = np.concatenate([np.arange(n - m, n) for _, m, n in seqs])
    want, mag = R.rotate(R.f64(q), pos, None if f is None else R.f64(f), inter)
    err = np.abs(R.f64(qo) - want)
    assert (err <= R.ROT * mag + R.half_step(qt) * np.abs(want)).all(), err.max()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("skew", [0, 1])
def test_append_parts_of_a_fused_projection(dtype, skew):
    """k, v and q as slices of one [rows, (h_q + 2 h_kv) d (+ 1)] tensor; an odd row
    stride leaves nothing aligned."""
    rng = np.random.default_rng(5)
    h_kv, G, d, page, lens, rows = 2, 2, 64, 32, [50, 9], [20, 9]
    cache = make_cache(rng, 8, page, h_kv, d, BF16 if dtype == "bf16" else F8)
    batch, table, seqs = make_batch(rng, 8, page, lens, rows)
    wide = randn(rng, 29, 8 * d + skew)
    part = lambda a, b: wide[:, a * d + skew:b * d + skew].unflatten(1, (b - a, d))  # noqa: E731
    q, k, v = part(0, 4), part(4, 6), part(6, 8)
    f = torch.from_numpy((1e4 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    before = ref_cache(cache)
    qo = F.kv_append(cache, batch, k, v, q=q, inv_freq=f)
    torch.cuda.synchronize()
    check_append(before, cache, table, seqs, k, v, f, False)
    pos = np.concatenate([np.arange(n - m, n) for _, m, n in seqs])
    want, mag = R.rotate(R.f64(q), pos, R.f64(f), False)
    assert (np.abs(R.f64(qo) - want) <= R.ROT * mag + 2.0 ** -8 * np.abs(want)).all()
    # in place, from a contiguous copy: the same bits
    mine = q.contiguous()
    assert F.kv_append(cache, batch, k, v, q=mine, inv_freq=f, q_out=mine) is mine
    assert torch.equal(mine, qo)


def test_append_far_positions():
    """Angles of positions near 2^30: formed in 64 bits."""
    rng = np.random.default_rng(6)
    page, d = 1 << 20, 32
    k8 = torch.zeros((1, 1, page, d), dtype=BF16, device="cuda")
    cache = F.KVCache(k8, torch.zeros_like(k8))
    width = 1 << 10
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 0  # only the last page exists
    n = (1 << 30) - 5
    batch = F.KVBatch(table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    k, v, q = (randn(rng, 1, h, d) for h in (1, 1, 2))
    f = torch.from_numpy((1e6 ** (-np.arange(16) / 16)).astype(np.float32)).cuda()
    qo = F.kv_append(cache, batch, k, v, q=q, inv_freq=f)
    torch.cuda.synchronize()
    for got, x in ((qo, q), (cache.k[0, :, (n - 1) % page][None], k)):
        want, mag = R.rotate(R.f64(x), [n - 1], R.f64(f), False)
        assert (np.abs(R.f64(got) - want) <= R.ROT * mag + 2.0 ** -8 * np.abs(want)).all()
    assert int((cache.k != 0).any(-1).sum()) == 1


def test_append_token_by_token_e4m3():
    """A block's scale grows as larger tokens come in, and its older codes move."""
    rng = np.random.default_rng(7)
    h_kv, d, page = 2, 32, 32
    cache = F.KVCache.empty(4, page, h_kv, d, dtype=F8)
    want = ref_cache(cache)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    batch = F.KVBatch(table, n)
    for i in range(70):
        n += 1
        k, v = (randn(rng, 1, h_kv, d, scale=2.0 ** ((i % 16) - 8)) for _ in range(2))
        before = ref_cache(cache)
        F.kv_append(cache, batch, k, v)
        torch.cuda.synchronize()
        check_append(before, cache, table.cpu().numpy(), [(0, 1, i + 1)], k, v, None, False)
        want.append(table.cpu().numpy(), [(0, 1, i + 1)], R.f64(k), R.f64(v))
    for side, x in ((0, cache.k), (1, cache.v)):  # no rotation: every code as the reference has it
        np.testing.assert_array_equal(R.bytes_of(x), (want.k, want.v)[side])


def test_append_special_values_e4m3():
    """Zeros, an infinity (saturates), a NaN (stays), the smallest and largest scales."""
    d = 32
    cache = F.KVCache.empty(6, 16, 1, d, dtype=F8)
    x = torch.zeros((6, 1, d), dtype=F32, device="cuda")
    x[1] = 1e-38
    x[2] = 3e38
    x[3, 0, 0], x[3, 0, 1:] = math.inf, 1.0
    x[4, 0, 0], x[4, 0, 1:] = math.nan, -2.0
    x[5] = -0.0
    table = torch.arange(6, dtype=torch.int32, device="cuda")[:, None].contiguous()
    batch = F.KVBatch(table, torch.ones(6, dtype=torch.int32, device="cuda"))
    F.kv_append(cache, batch, x, x)
    torch.cuda.synchronize()
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert s[:, 0, 0].tolist() == [8, 8, 246, 119, 120, 8]
        val = c[:, 0, 0].float()
        assert (val[0] == 0).all() and (val[5] == 0).all()
        assert (val[2] == 448).all() and val[3, 0] == 448 and (val[3, 1:] == 256).all()
        assert torch.isnan(val[4, 0]) and (val[4, 1:] == -256).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_leaves_what_it_must(dtype):
    """Bad pages, lengths and row ranges, rows behind the last sequence: nothing is
    written for them, and the others are as ever."""
    rng = np.random.default_rng(8)
    h_kv, d, page = 1, 32, 16
    cache = make_cache(rng, 12, page, h_kv, d, BF16 if dtype == "bf16" else F8)
    lens = [20, 40, 18, 5, 35, 3]
    table = np.array([[0, 99, 1], [2, 3, -1], [4, 5, 6], [7, 8, 9], [10, 11, 0], [9, -7, 1]], dtype=np.int32)
    start = np.array([0, 20, 30, 31, 34, 35, 36], dtype=np.int32)
    bad = list(lens)
    bad[3] = -4  # counts as empty: its rows have negative positions
    bad[4] = 1000  # beyond max_len: the same
    T = 40       # rows 36 .. 39 are nobody's
    batch = F.KVBatch(torch.from_numpy(table).cuda(), torch.tensor(bad, dtype=torch.int32).cuda(),
                      torch.from_numpy(start).cuda(), num_rows=T, max_rows=20, max_len=48)
    k, v = (randn(rng, T, h_kv, d) for _ in range(2))
    q = randn(rng, T, 2, d)
    qo = torch.full_like(q, 7.0)
    f = torch.full((16,), 0.01, device="cuda")
    before = ref_cache(cache)
    F.kv_append(cache, batch, k, v, q=q, inv_freq=f, q_out=qo)
    torch.cuda.synchronize()
    eff = [n if 0 <= n <= 48 else 0 for n in bad]
    seqs = R.sequences(eff, start)
    check_append(before, cache, table, seqs, k, v, f, False)
    assert (qo[36:] == 7.0).all()
    pos = np.concatenate([np.arange(n - m, n) for _, m, n in seqs])
    want, mag = R.rotate(R.f64(q)[:36], pos, R.f64(f), False)
    assert (np.abs(R.f64(qo)[:36] - want) <= R.ROT * mag + 2.0 ** -8 * np.abs(want)).all()
    # rows out of range: only the sequences whose rows are in bounds are written
    wild = torch.tensor([0, 50, 30, 31, -3, 35, 36], dtype=torch.int32, device="cuda")
    batch = F.KVBatch(batch.page_table, batch.seq_len, wild, num_rows=T, max_rows=20, max_len=48)
    F.kv_append(cache, batch, k, v, q=q, inv_freq=f)
    torch.cuda.synchronize()


# -------------------------------------------------------------- attention --

CASES = [
    # d, h_kv, G, page, lens, rows, window, sinks
    (128, 8, 4, 64, [100, 1, 17, 640], None, 0, 0),
    (128, 2, 4, 16, [300, 40, 33, 20], [3, 0, 33, 9], 0, 0),
    (128, 1, 4, 128, [700], [300], 0, 0),
    (128, 1, 8, 64, [129, 513], [129, 130], 100, 5),
    (128, 2, 7, 64, [1000, 15, 400], None, 64, 4),
    (64, 1, 1, 48, [97, 16, 200, 5], [90, 16, 1, 3], 0, 0),
    (64, 2, 2, 256, [515, 300], [257, 300], 33, 16),
    (64, 1, 32, 64, [100], [20], 17, 0),
    (96, 3, 1, 32, [70, 70], [33, 15], 16, 1),
    (32, 2, 2, 16, [31, 0, 1], [31, 0, 1], 1, 0),
    (256, 1, 2, 128, [515], [40], 0, 0),
    (256, 1, 4, 16, [90, 33], None, 20, 100),
    (160, 2, 1, 32, [77, 12], [50, 12], 5, 3),
    (192, 1, 3, 16, [200], None, 0, 0),
    (224, 1, 2, 16, [65], [3], 30, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dtype, qt):
    d, h_kv, G, page, lens, rows, window, sinks = CASES[case]
    rng = np.random.default_rng(case)
    ct, qt = BF16 if dtype == "bf16" else F8, BF16 if qt == "bf16" else F32
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(rng, pages, page, h_kv, d, ct)
    batch, table, seqs = make_batch(rng, pages, page, lens, rows)
    q = randn(rng, batch.num_rows, h_kv * G, d, dtype=qt, scale=1.5)
    scale = 1.0 / math.sqrt(d)
    got = F.kv_attention(cache, batch, q, scale, window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = R.attention(ref_cache(cache), table, seqs, R.f64(q), scale, window, sinks, WEIGHT[ct, qt],
                       R.half_step(qt))
    check_attention(got, want, "case %d" % case)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("G,page,lens,rows,window,sinks", [
    (4, 16, [300], [150], 0, 0), (7, 48, [257, 40], [257, 11], 50, 3), (1, 128, [700, 1, 0], [129, 1, 0], 0, 0)])
def test_attention_many_rows(d, G, page, lens, rows, window, sinks, dtype):
    """Every width of the many-rows kernel: small and odd pages, several units and tiles,
    ragged sequences."""
    rng = np.random.default_rng(d + G)
    ct = BF16 if dtype == "bf16" else F8
    pages = sum(-(-n // page) for n in lens) + 1
    cache = make_cache(rng, pages, page, 2, d, ct)
    batch, table, seqs = make_batch(rng, pages, page, lens, rows)
    q = randn(rng, batch.num_rows, 2 * G, d, scale=1.5)
    got = F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / math.sqrt(d), window, sinks, WEIGHT[ct, BF16])
    check_attention(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("lens,rows,window", [
    ([700, 33, 1200, 5, 90, 64], [1, 1, 200, 5, 90, 16], 0), ([40, 800, 41], [15, 300, 1], 70),
    ([3000, 20, 20, 20, 20], [1, 15, 16, 17, 0], 0)])
def test_attention_prompts_beside_decoded_tokens(lens, rows, window, qt, dtype):
    """Long and short sequences in one batch: each goes to the kernel for its rows, a few
    on either side of where that changes (16 rows of 4 heads)."""
    rng = np.random.default_rng(21)
    ct, qt = BF16 if dtype == "bf16" else F8, BF16 if qt == "bf16" else F32
    cache = make_cache(rng, 70, 64, 2, 128, ct)
    batch, table, seqs = make_batch(rng, 70, 64, lens, rows, num_rows=sum(rows) + 3)
    q = randn(rng, batch.num_rows, 8, 128, dtype=qt)
    out, lse = torch.full_like(q, 7.0), torch.full((batch.num_rows, 8), 7.0, device="cuda")
    F.kv_attention(cache, batch, q, window=window, sinks=3, out=out, lse=lse)
    torch.cuda.synchronize()
    want = R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / math.sqrt(128), window, 3, WEIGHT[ct, qt],
                       R.half_step(qt))
    check_attention((out, lse), want)
    assert (out[-3:] == 7.0).all() and (lse[-3:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attention_many_heads_of_one_kv_head(dtype):
    """64 and more query heads a KV head: one decoded token fills a many-rows unit."""
    rng = np.random.default_rng(22)
    ct = BF16 if dtype == "bf16" else F8
    for G, lens in ((64, [900, 3]), (130, [200])):
        cache = make_cache(rng, 20, 64, 1, 64, ct)
        batch, table, seqs = make_batch(rng, 20, 64, lens)
        q = randn(rng, len(lens), G, 64)
        got = F.kv_attention(cache, batch, q)
        torch.cuda.synchronize()
        want = R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / 8, weight_step=WEIGHT[ct, BF16])
        check_attention(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (500, 20), (3000, 0), (5000, 100)])
def test_attention_split_over_blocks(dtype, window, sinks):
    """A context long enough that several blocks share it, with max_len far above
    some sequences' lengths."""
    rng = np.random.default_rng(11)
    ct = BF16 if dtype == "bf16" else F8
    d, h_kv, G, page = 128, 1, 4, 64
    lens = [9001, 37, 4096]
    pages = sum(-(-n // page) for n in lens)
    cache = make_cache(rng, pages, page, h_kv, d, ct)
    batch, table, seqs = make_batch(rng, pages, page, lens, [2, 1, 1], width=400)
    q = randn(rng, 4, h_kv * G, d, scale=2)
    got = F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    again = F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / math.sqrt(d), window, sinks,
                       WEIGHT[ct, BF16])
    check_attention(got, want)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def poison(cache, table, seqs, sees):
    """NaN and infinities into every token that no row of the sequence may see, and
    into every page that nobody has."""
    k, v = cache.k.clone(), cache.v.clone()
    page = k.shape[2]
    mask = torch.ones(k.shape[0], page, dtype=torch.bool)
    for s, (_, m, n) in enumerate(seqs):
        for j in range(n):
            if any(sees(p, j) for p in range(n - m, n)):
                mask[table[s][j // page], j % page] = False
    mask = mask.cuda()[:, None, :, None].expand(k.shape)
    if k.dtype == BF16:
        k[mask] = math.nan
        v[mask] = math.inf
    else:
        k.view(torch.uint8)[mask] = 0x7f
        v.view(torch.uint8)[mask] = 0xff
    return F.KVCache(k, v, cache.k_scale, cache.v_scale)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,window,sinks", [(None, 0, 0), (None, 30, 3), ([150, 2, 9], 0, 0),
                                              ([150, 33, 1], 40, 5)])
def test_attention_unseen_values_do_not_matter(dtype, qt, rows, window, sinks):
    rng = np.random.default_rng(12)
    ct, qt = BF16 if dtype == "bf16" else F8, BF16 if qt == "bf16" else F32
    cache = make_cache(rng, 12, 64, 2, 128, ct)
    batch, table, seqs = make_batch(rng, 12, 64, [201, 77, 9], rows)
    q = randn(rng, batch.num_rows, 8, 128, dtype=qt)
    sees = lambda p, j: j <= p and (not window or j > p - window or j < sinks)  # noqa: E731
    want = F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    got = F.kv_attention(poison(cache, table, seqs, sees), batch, q, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("m,bad,window,sinks", [(20, 195, 0, 0), (200, 120, 0, 0), (150, 60, 50, 3),
                                               (150, 2, 50, 3), (200, 199, 0, 0)])
def test_attention_later_tokens_do_not_reach_earlier_rows(dtype, m, bad, window, sinks):
    """One token holds NaN and infinities: the rows that do not see it are what the
    reference has without it (many rows: the unit is done again by the other kernel, whose
    rounding differs, so the tolerance is the reference's and not zero), and those that
    see it are not finite."""
    rng = np.random.default_rng(13)
    ct = BF16 if dtype == "bf16" else F8
    n, d, page = 200, 128, 64
    cache = make_cache(rng, 5, page, 1, d, ct)
    batch, table, seqs = make_batch(rng, 5, page, [n], [m])
    q = randn(rng, m, 4, d)
    want = F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    v = cache.v.clone()
    at = (table[0][bad // page], 0, bad % page)
    if ct == BF16:
        v[at] = math.inf
        v[at][0] = math.nan
    else:
        v.view(torch.uint8)[at] = 0x7f
    got = F.kv_attention(F.KVCache(cache.k, v, cache.k_scale, cache.v_scale), batch, q, window=window, sinks=sinks)
    torch.cuda.synchronize()
    p = torch.arange(n - m, n, device="cuda")
    sees = (bad <= p) & ((p - bad < window) | (bad < sinks) if window else torch.ones_like(p, dtype=torch.bool))
    assert not torch.isfinite(got[0][sees]).any()
    ref = list(R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / math.sqrt(d), window, sinks,
                           WEIGHT[ct, BF16]))
    check_attention(want, ref)
    held = np.isfinite(ref[1]).copy()
    ref[1][sees.cpu().numpy()] = np.nan  # compare the others alone
    assert held.all()
    check_attention(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attention_bad_pages_lengths_and_rows(dtype):
    """A page outside the pool is not seen; bad lengths count as empty; rows that no
    sequence has stay; the status counts the sequences that broke a bound."""
    rng = np.random.default_rng(14)
    ct = BF16 if dtype == "bf16" else F8
    cache = make_cache(rng, 6, 16, 1, 64, ct)
    table = np.array([[0, 99, 1], [2, -1, 3], [4, 5, 0], [5, 4, 3]], dtype=np.int32)
    lens = [45, 20, 1000, 60]  # 1000 > max_len; 60 is beyond the table's 48
    start = np.array([0, 5, 6, 9, 12], dtype=np.int32)
    T = 14
    batch = F.KVBatch(torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                      torch.from_numpy(start).cuda(), num_rows=T, max_rows=5, max_len=64)
    q = randn(rng, T, 4, 64)
    out, lse = torch.full_like(q, 7.0), torch.full((T, 4), 7.0, device="cuda")
    ws = F.Workspace()
    F.kv_attention(cache, batch, q, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    seqs = R.sequences([45, 20, 0, 60], start)
    want = R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / 8, weight_step=WEIGHT[ct, BF16])
    check_attention((out, lse), want)
    assert (out[12:] == 7.0).all() and (lse[12:] == 7.0).all()
    with pytest.raises(F.FathomError) as e:
        F.check_device_status(ws)
    assert e.value.status == F.ERR_DEVICE_CHECK and "1 faults" in str(e.value)
    good = F.KVBatch(batch.page_table, torch.tensor([45, 20, 1, 48], dtype=torch.int32).cuda(), batch.q_start,
                     num_rows=T, max_rows=5, max_len=64)
    F.kv_attention(cache, good, q, out=out, lse=lse, workspace=ws)
    F.check_device_status(ws)


def test_attention_extreme_scores():
    """Scores far apart, equal, and an empty-headed scale of 0; values near fp32's ends."""
    rng = np.random.default_rng(15)
    for ct in (BF16, F8):
        cache = make_cache(rng, 3, 64, 1, 64, ct)
        batch, table, seqs = make_batch(rng, 3, 64, [150], [3])
        for qs, scale in ((300.0, 0.5), (1e-30, 1.0), (1.0, 0.0), (1.0, -0.3)):
            q = randn(rng, 3, 2, 64, scale=qs)
            got = F.kv_attention(cache, batch, q, scale)
            torch.cuda.synchronize()
            want = R.attention(ref_cache(cache), table, seqs, R.f64(q), scale, weight_step=WEIGHT[ct, BF16])
            check_attention(got, want, "%s %g %g" % (ct, qs, scale))


def test_attention_flat_weights_over_a_long_cache():
    """One key far above 60000 flat ones, which together outweigh it: weights of 2^-15 and
    less of the largest still count."""
    d, n = 64, 60000
    for ct in (BF16, F8):
        k = torch.zeros((1, 1, 60032, d), device="cuda")
        k[0, 0, 0, 0] = 8.0
        v = torch.ones((1, 1, 60032, d), device="cuda")
        v[0, 0, 0] = -1.0
        cache = F.KVCache.empty(1, 60032, 1, d, dtype=ct)
        batch = F.KVBatch(torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"),
                          torch.tensor([0, n], dtype=torch.int32, device="cuda"), num_rows=n)
        F.kv_append(cache, batch, k[0, 0, :n, None].contiguous(), v[0, 0, :n, None].contiguous())
        one = F.KVBatch(batch.page_table, batch.seq_len)
        q = torch.zeros((1, 1, d), dtype=BF16, device="cuda")
        q[0, 0, 0] = 1.25
        for top in (10.0, 11.09, 16.0, 20.0):  # the largest score above the others
            out, lse = F.kv_attention(cache, one, q, top / 10.0)
            w = math.exp(top)
            want = (n - 1 - w) / (n - 1 + w)
            assert abs(float(out[0, 0, 5]) - want) <= 2.0 ** -8 + 2.0 ** -7, (ct, top)
            assert abs(float(lse) - math.log(n - 1 + w)) <= 1e-4


def test_offsets_beyond_32_bits():
    """Pages whose elements lie beyond 2^32 of the cache's start."""
    rng = np.random.default_rng(16)
    h_kv, page, d = 8, 256, 128
    per = h_kv * page * d
    pages = (1 << 32) // per + 3
    k = torch.zeros((pages, h_kv, page, d), dtype=torch.uint8, device="cuda").view(F8)
    s = torch.full((pages, h_kv, page // 16), 120, dtype=torch.uint8, device="cuda")
    cache = F.KVCache(k, k, s, s)  # one tensor for both: the append writes v last or first, both the same
    lens = [300]
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    batch = F.KVBatch(table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      torch.tensor([0, 300], dtype=torch.int32, device="cuda"), num_rows=300)
    x = randn(rng, 300, h_kv, d)
    F.kv_append(cache, batch, x, x)
    q = randn(rng, 300, 8, d)
    got = F.kv_attention(cache, batch, q)
    tail = F.KVCache(*(t[-2:] for t in (k, k, s, s)))
    small = F.KVBatch(torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), batch.seq_len, batch.q_start,
                      num_rows=300)
    want = F.kv_attention(tail, small, q)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int((k[:-2].view(torch.uint8) != 0).sum()) == 0
    ref = R.attention(ref_cache(tail), [[1, 0]], [(0, 300, 300)], R.f64(q), 1 / math.sqrt(d),
                      weight_step=WEIGHT[F8, BF16])
    check_attention(got, ref)


def test_strided_queries_and_odd_alignment():
    rng = np.random.default_rng(17)
    cache = make_cache(rng, 4, 64, 2, 64, BF16)
    for rows in ([3], [140]):
        batch, table, seqs = make_batch(rng, 4, 64, [200], rows)
        wide = randn(rng, rows[0], 4 * 64 + 77)
        q = wide[:, 33:33 + 256].unflatten(1, (4, 64))
        got = F.kv_attention(cache, batch, q)
        want = F.kv_attention(cache, batch, q.contiguous())
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------ streams, graphs, together --

def test_other_stream_and_captured_replay():
    """Calls on a side stream; two captured graphs, replayed with other contents in
    between, each equal to eager calls."""
    rng = np.random.default_rng(18)
    h_kv, d, page = 2, 128, 32
    f = torch.from_numpy((1e4 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()
    caches = [F.KVCache.empty(300, page, h_kv, d, dtype=t) for t in (BF16, F8)]
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150)
    n = torch.tensor([4200, 900], dtype=torch.int32, device="cuda")
    batch = F.KVBatch(table, n, max_len=4800)
    k, v, q = (randn(rng, 2, h, d) for h in (h_kv, h_kv, 8))

    def step(cache):
        qr = F.kv_append(cache, batch, k, v, q=q, inv_freq=f)
        return F.kv_attention(cache, batch, qr, window=3000, sinks=4)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c in caches:
            step(c)
    side.synchronize()
    graphs, outs = [], []
    for c in caches:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c))
        graphs.append(g)
    for i in range(6):
        n += 1
        for x in (k, v, q):
            x.copy_(randn(rng, *x.shape))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [(o.clone(), l.clone()) for o, l in outs]
        for c, (o, l) in zip(caches, got):
            o2, l2 = step(c)  # the same tokens again: the cache is as it was
            torch.cuda.synchronize()
            assert torch.equal(o, o2) and torch.equal(l, l2)
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    o3, l3 = F.kv_attention(caches[0], batch, q, window=3000, sinks=4, stream=s2)
    s2.synchronize()
    o4, l4 = F.kv_attention(caches[0], batch, q, window=3000, sinks=4)
    torch.cuda.synchronize()
    assert torch.equal(o3, o4) and torch.equal(l3, l4)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompt_then_decode_together(dtype):
    """A prompt in two chunks, then decoded tokens, two sequences: append and attention as
    a serving loop calls them, a full and a windowed layer on the same cache."""
    rng = np.random.default_rng(19)
    ct = BF16 if dtype == "bf16" else F8
    h_kv, G, d, page = 2, 4, 128, 64
    cache = F.KVCache.empty(16, page, h_kv, d, dtype=ct)
    table = torch.from_numpy(rng.permutation(16).reshape(2, 8).astype(np.int32)).cuda()
    f = torch.from_numpy((1e4 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()
    n = np.zeros(2, dtype=np.int64)
    for rows in ([200, 130], [150, 1], [1, 1], [1, 1], [4, 0]):
        n += rows
        start = np.concatenate([[0], np.cumsum(rows)])
        batch = F.KVBatch(table, torch.from_numpy(n.astype(np.int32)).cuda(),
                          torch.from_numpy(start.astype(np.int32)).cuda(), num_rows=int(start[-1]),
                          max_rows=max(rows))
        k, v, q = (randn(rng, int(start[-1]), h, d) for h in (h_kv, h_kv, h_kv * G))
        before = ref_cache(cache)
        qr = F.kv_append(cache, batch, k, v, q=q, inv_freq=f)
        full = F.kv_attention(cache, batch, qr)
        win = F.kv_attention(cache, batch, qr, window=100, sinks=4)
        torch.cuda.synchronize()
        t, seqs = table.cpu().numpy(), R.sequences(n, start)
        check_append(before, cache, t, seqs, k, v, f, False)
        for got, w, s in ((full, 0, 0), (win, 100, 4)):
            want = R.attention(ref_cache(cache), t, seqs, R.f64(qr), 1 / math.sqrt(d), w, s, WEIGHT[ct, BF16])
            check_attention(got, want)


def test_one_page_cache_feeds_the_sparse_attention():
    """A cache of one page is the [h_kv][n][d] layout of fathom_sparse_attention: over all
    the tokens that a row sees, both calls give the same attention."""
    rng = np.random.default_rng(20)
    h_kv, G, d, cap = 2, 4, 128, 4096
    cache = F.KVCache.empty(1, cap, h_kv, d)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    n = 3001
    batch = F.KVBatch(table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, n], dtype=torch.int32, device="cuda"), num_rows=n)
    F.kv_append(cache, batch, randn(rng, n, h_kv, d), randn(rng, n, h_kv, d))
    one = F.KVBatch(table, batch.seq_len)
    q = randn(rng, 1, h_kv * G, d, dtype=F32)
    window, sinks = 700, 9
    seen = np.concatenate([np.arange(sinks), np.arange(n - window, n)]).astype(np.int32)
    idx = torch.from_numpy(np.tile(seen, (h_kv * G, 1))).cuda()
    o, l = F.sparse_attention(q[0], cache.k[0], cache.v[0], idx)
    o2, l2 = F.kv_attention(cache, one, q, window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = R.attention(ref_cache(cache), [[0]], [(0, 1, n)], R.f64(q), 1 / math.sqrt(d), window, sinks,
                       WEIGHT[BF16, F32], R.half_step(F32))
    check_attention((o2, l2), want)
    check_attention((o[None], l[None]), want)  # fp32 throughout: within the same bounds


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 96, 160, 256])
def test_units_with_an_unseen_nan_are_done_again(d, dtype):
    """Many rows at the other widths: a NaN token among the rows' own, seen by the later ones
    alone."""
    rng = np.random.default_rng(23)
    ct = BF16 if dtype == "bf16" else F8
    n, m, bad = 300, 170, 222
    cache = make_cache(rng, 6, 64, 2, d, ct)
    batch, table, seqs = make_batch(rng, 6, 64, [n], [m])
    q = randn(rng, m, 4, d)
    ref = list(R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / math.sqrt(d), weight_step=WEIGHT[ct, BF16]))
    at = (table[0][bad // 64], 1, bad % 64)  # of KV head 1: query heads 2 and 3
    if ct == BF16:
        cache.v[at] = math.nan
    else:
        cache.v.view(torch.uint8)[at] = 0x7f
    got = F.kv_attention(cache, batch, q)
    torch.cuda.synchronize()
    late = slice(bad - (n - m), None)
    assert torch.isnan(got[0][late, 2:]).all() and torch.isfinite(got[0][late, :2]).all()
    ref[1][late, 2:] = np.nan  # compare the others
    check_attention(got, ref)


def test_calls_on_two_streams_at_once():
    """Prompts and decoded tokens on two streams without order between them: each call has
    a workspace of its own."""
    rng = np.random.default_rng(24)
    jobs = []
    for ct, lens, rows in ((BF16, [1500, 40], [600, 1]), (F8, [1500, 40], [600, 1]), (F8, [3000, 2000], None),
                           (BF16, [9000], None)):
        pages = sum(-(-x // 64) for x in lens)
        cache = make_cache(rng, pages, 64, 2, 128, ct)
        batch, _, _ = make_batch(rng, pages, 64, lens, rows)
        q = randn(rng, batch.num_rows, 8, 128)
        jobs.append((cache, batch, q, F.kv_attention(cache, batch, q)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        for s, k in zip(streams, (i, i + 1)):
            cache, batch, q, want = jobs[k % len(jobs)]
            got.append((F.kv_attention(cache, batch, q, stream=s), want))
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in got:
        assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_sequences_that_share_pages(dtype):
    """A prefix's pages in two sequences' tables, and one page twice in a table, for
    reading."""
    rng = np.random.default_rng(25)
    ct = BF16 if dtype == "bf16" else F8
    cache = make_cache(rng, 5, 32, 1, 64, ct)
    table = np.array([[0, 1, 2], [0, 1, 3], [4, 4, 0]], dtype=np.int32)
    lens, rows = [90, 80, 96], [20, 1, 40]
    start = np.array([0, 20, 21, 61], dtype=np.int32)
    batch = F.KVBatch(torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                      torch.from_numpy(start).cuda(), num_rows=61, max_rows=40)
    q = randn(rng, 61, 4, 64)
    got = F.kv_attention(cache, batch, q)
    torch.cuda.synchronize()
    want = R.attention(ref_cache(cache), table, R.sequences(lens, start), R.f64(q), 1 / 8, weight_step=WEIGHT[ct, BF16])
    check_attention(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_captured_prompt_chunks_with_one_workspace(dtype):
    """Chunks of two prompts captured on two caches with one workspace between them, replayed
    as the sequences grow, each equal to eager calls with workspaces of their own."""
    rng = np.random.default_rng(26)
    ct = BF16 if dtype == "bf16" else F8
    rows, d = [200, 131], 128
    caches = [make_cache(rng, 128, 64, 2, d, ct) for _ in range(2)]
    table = torch.from_numpy(rng.permutation(128).reshape(2, 64).astype(np.int32)).cuda()
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    batch = F.KVBatch(table, n, torch.tensor([0, 200, 331], dtype=torch.int32).cuda(), num_rows=331,
                      max_rows=200, max_len=4096)
    q = randn(rng, 331, 8, d)
    n += torch.tensor(rows, dtype=torch.int32, device="cuda")
    ws = F.Workspace()
    for c in caches:  # the workspace grows before the capture
        F.kv_attention(c, batch, q, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in caches:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(F.kv_attention(c, batch, q, workspace=ws))
        graphs.append(g)
    for lens in ([200, 131], [201, 1000], [4096, 140], [3000, 0], [777, 4001]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(randn(rng, *q.shape))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [(o.clone(), l.clone()) for o, l in outs]
        for c, (o, l) in zip(caches, got):
            o2, l2 = F.kv_attention(c, batch, q)
            torch.cuda.synchronize()
            assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("m", [1, 3, 90])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_query_that_is_not_finite_spoils_its_own_row(bad, dtype, m):
    """One element of one row's head: that row's head alone may change."""
    rng = np.random.default_rng(27)
    cache = make_cache(rng, 8, 64, 1, 128, BF16 if dtype == "bf16" else F8)
    batch, _, _ = make_batch(rng, 8, 64, [500], [m])
    q = randn(rng, m, 4, 128)
    want = F.kv_attention(cache, batch, q)
    q2 = q.clone()
    q2[m // 2, 1, 77] = bad
    got = F.kv_attention(cache, batch, q2)
    torch.cuda.synchronize()
    assert torch.isnan(got[0][m // 2, 1]).all()
    for a, b in zip(got, want):
        a[m // 2, 1], b[m // 2, 1] = 0, 0
        assert torch.equal(a, b)
