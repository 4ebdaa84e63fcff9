"""fathom_kv_attention on the GPU over calls whose launches are divided, grouped or
bounded in less usual ways, against fp64."""

import math

import numpy as np
import pytest
import torch

import test_gpu_kv as T
from test_gpu_kv import BF16, F32, F8, WEIGHT, _lib, make_batch, make_cache, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def attention64(cache, table, seqs, q, scale, window=0, sinks=0, weight_step=2.0 ** -8, out_step=2.0 ** -8):
    """The formula in fp64 on the GPU, with kv_reference.py's tolerances: (out, lse, tolerance of
    out, tolerance of lse).  weight_step 2^-11 stands for fp16 weights, which have 11 bits down to
    2^-29 of the largest and are off by 2^-40 of it below: 2^-40 sum |v| more."""
    rows, h_q, d = q.shape
    h_kv, page = cache.k.shape[1], cache.page_tokens
    G = h_q // h_kv
    dev = q.device
    out, tol = (torch.zeros((rows, h_q, d), dtype=torch.float64, device=dev) for _ in range(2))
    lse, ltol = (torch.zeros((rows, h_q), dtype=torch.float64, device=dev) for _ in range(2))
    held = torch.zeros(rows, dtype=torch.bool, device=dev)
    q = q.double()
    for s, (row0, m, n) in enumerate(seqs):
        if m == 0:
            continue
        held[row0:row0 + m] = True
        if n == 0:
            lse[row0:row0 + m] = -math.inf
            continue
        j = torch.arange(n, device=dev)
        pg = torch.as_tensor(np.asarray(table[s]), device=dev).long()[j // page]
        sl = j % page
        ok = (pg >= 0) & (pg < cache.k.shape[0])  # tokens whose page exists
        pg = torch.where(ok, pg, 0)
        for g in range(h_kv):
            kv = []
            for name in ("k", "v"):
                x = getattr(cache, name)
                if x.dtype == F8:
                    x = x.view(torch.uint8)[pg, g, sl].view(F8).double()
                    e = getattr(cache, name + "_scale")[pg, g, sl // 16].double().clamp(8, 246)
                    x = x * torch.exp2(e - 127)[:, None]
                else:
                    x = x[pg, g, sl].double()
                kv.append(x)
            k, v = (torch.where(ok[:, None], x, 0.0) for x in kv)
            heads = slice(g * G, (g + 1) * G)
            for r in range(0, m, 256):
                e = min(m, r + 256)
                at = slice(row0 + r, row0 + e)
                p = torch.arange(n - m + r, n - m + e, device=dev)[:, None]
                see = (j <= p) & ok
                if window:
                    see &= (j > p - window) | (j < sinks)
                see = see[:, None, :]
                some = see.any(-1)
                qq = q[at, heads]
                sc = (qq @ k.T * scale).masked_fill(~see, -math.inf)
                lse[at, heads] = torch.logsumexp(sc, -1)
                w = torch.where(some[..., None], torch.softmax(sc, -1), 0.0)
                out[at, heads] = w @ v
                a = w @ v.abs()
                b = (abs(scale) * (qq.abs() @ k.abs().T)).masked_fill(~see, 0.0).amax(-1)
                count = see.sum(-1)
                delta = (d / 16 + 4) * 2.0 ** -22 * b
                adds = count / 16 + 16
                tol[at, heads] = (2 * (delta[..., None] + 2.0 ** -20) + weight_step + adds[..., None] * 2.0 ** -22) * a \
                    + out_step * out[at, heads].abs() + 1e-30
                if weight_step == 2.0 ** -11:
                    tol[at, heads] += 2.0 ** -40 * (see.double() @ v.abs())
                ltol[at, heads] = delta + 2.0 ** -20 + adds * 2.0 ** -23 + 2.0 ** -22 * torch.where(some, lse[at, heads], 0.0).abs().clamp(min=1)
    return out, lse, tol, ltol, held


def check(got, want, what=""):
    out, lse, tol, ltol, held = want
    e = ((got[0].double() - out).abs() / tol.clamp(min=1e-30))[held].max().item()
    assert e <= 1, "%s: out off by %g tolerances" % (what, e)
    nothing = torch.isneginf(lse)
    assert (got[0][nothing & held[:, None]] == 0).all() and torch.isneginf(got[1][nothing & held[:, None]]).all(), what
    lse, mine = torch.where(nothing, 0.0, lse), torch.where(nothing, 0.0, got[1].double())
    e = ((mine - lse).abs() / ltol.clamp(min=1e-30))[held].max().item()
    assert e <= 1, "%s: lse off by %g tolerances" % (what, e)


def test_status_of_a_call_with_more_units_than_processors():
    """A prompt of several hundred units beside sequences that break their bounds: all of these
    are counted, and a good call clears them."""
    rng = np.random.default_rng(50)
    cache = make_cache(rng, 120, 64, 8, 64, BF16)
    table = torch.from_numpy(rng.permutation(120).astype(np.int32)[None].repeat(4, 0)).cuda()
    start = torch.tensor([0, 3000, 3001, 3001, 3002], dtype=torch.int32, device="cuda")
    lens = torch.tensor([7000, -1, 9000, 3], dtype=torch.int32, device="cuda")
    batch = T.F.KVBatch(table, lens, start, num_rows=3002, max_rows=3000)
    q = randn(rng, 3002, 32, 64)
    ws = T.F.Workspace()
    got = T.F.kv_attention(cache, batch, q, workspace=ws)
    with pytest.raises(T.F.FathomError, match="2 faults"):
        T.F.check_device_status(ws)
    want = attention64(cache, table.cpu().numpy(), [(0, 3000, 7000), (0, 0, 0), (0, 0, 0), (3001, 1, 3)], q, 1 / 8)
    check(got, want)
    assert (got[0][3000] == 0).all() and torch.isneginf(got[1][3000]).all()
    lens.copy_(torch.tensor([7000, 1, 0, 3], dtype=torch.int32))
    T.F.kv_attention(cache, batch, q, workspace=ws)
    T.F.check_device_status(ws)


def _size(cache, batch, q, **kw):
    """Bytes of the workspace that the call asks for."""
    ws = T.F.Workspace()
    got = T.F.kv_attention(cache, batch, q, workspace=ws, **kw)
    return got, ws.buf.numel()


DIVIDED = [
    # d, h_kv, G, lens, rows, window, sinks
    (128, 1, 4, [9000], [100], 0, 0),           # fewer units than processors: each is divided
    (64, 2, 4, [7000, 3000], [130, 64], 0, 0),
    (96, 1, 8, [6000], [40], 2500, 300),
    (256, 1, 4, [5000], [70], 0, 0),
    (128, 8, 4, [5200], [1270], 0, 0),          # 160 units on 148 processors: the last 12 are
    (64, 8, 4, [4500], [1265], 3000, 5),
    (256, 8, 4, [2500], [600], 0, 0),           # 152 units
    (160, 8, 2, [4000], [1200], 0, 0),          # 152 units of unequal work: not divided
    (160, 8, 2, [5000], [1200], 0, 0),          # of about equal work (a context of 4 times the rows)
    (128, 1, 4, [60000], None, 0, 0),           # a decoded token: more splits than a cluster has
    (64, 1, 2, [40000, 33, 9000], [1, 2, 3], 0, 0),
    (128, 2, 4, [3000, 40000, 20000], [800, 1, 3], 0, 0),   # both kernels
    (128, 2, 4, [3000, 40000, 20000], [800, 1, 3], 15000, 4),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("d,h_kv,G,lens,rows,window,sinks", DIVIDED)
def test_divided_units(d, h_kv, G, lens, rows, window, sinks, qt, dtype):
    rng = np.random.default_rng(51)
    ct, qt = BF16 if dtype == "bf16" else F8, BF16 if qt == "bf16" else F32
    pages = sum(-(-n // 128) for n in lens)
    cache = make_cache(rng, pages, 128, h_kv, d, ct)
    batch, table, seqs = make_batch(rng, pages, 128, lens, rows)
    q = randn(rng, batch.num_rows, h_kv * G, d, dtype=qt, scale=1.5)
    got, size = _size(cache, batch, q, window=window, sinks=sinks)
    if (ct, qt) == (BF16, BF16) and not window and (lens, d) != ([4000], 160):
        assert size > 2 * 8 * (d + 2) * 4 * G  # divided: there are results to join
    want = attention64(cache, table, seqs, q, 1 / math.sqrt(d), window, sinks, WEIGHT[ct, qt],
                       2.0 ** -8 if qt == BF16 else 2.0 ** -24)
    check(got, want)


WIDENED = [
    # d, h_kv, G, page, lens, rows, window, sinks, max_len
    (128, 2, 4, 64, [9000, 700, 5000], [300, 200, 64], 1000, 0, 1 << 20),
    (64, 1, 8, 48, [4000, 300, 131], [150, 299, 131], 513, 700, 1 << 20),  # more first tokens than a window
    (96, 2, 2, 16, [2500], [1500], 100, 130, 1 << 18),
    (256, 1, 4, 128, [3000, 2000], [400, 300], 640, 5, 1 << 20),
    (128, 1, 4, 32, [6000], [5000], 128, 1, 1 << 16),
    (128, 2, 4, 64, [900, 300, 17, 1500, 64, 2000], [300, 200, 17, 100, 64, 40], 0, 0, 1 << 20),  # two groups of pairs
    (256, 2, 8, 128, [600, 1000, 70], [100, 8, 70], 0, 0, 1 << 20),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,h_kv,G,page,lens,rows,window,sinks,max_len", WIDENED)
def test_bounds_far_above_the_lengths(d, h_kv, G, page, lens, rows, window, sinks, max_len, dtype):
    """What the host sizes by max_len holds whatever the lengths are: over e4m3 the tiles that
    a window sees lie one behind the other in the widened copy, and pairs that do not fit into
    4 GiB come in groups."""
    rng = np.random.default_rng(52)
    ct = BF16 if dtype == "bf16" else F8
    pages = sum(-(-n // page) for n in lens) + 1
    cache = make_cache(rng, pages, page, h_kv, d, ct)
    batch, table, seqs = make_batch(rng, pages, page, lens, rows, max_len=max_len)
    q = randn(rng, batch.num_rows, h_kv * G, d, scale=1.5)
    got = T.F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    want = attention64(cache, table, seqs, q, 1 / math.sqrt(d), window, sinks, WEIGHT[ct, BF16])
    check(got, want)
    exact = T.F.KVBatch(batch.page_table, batch.seq_len, batch.q_start, num_rows=batch.num_rows,
                        max_rows=batch.max_rows, max_len=max(lens))
    check(T.F.kv_attention(cache, exact, q, window=window, sinks=sinks), want)


# -------------------------------------------------------- weights and scales --

FEW = [
    # d, h_kv, G, lens, rows, window, sinks: fewer than 64 columns each
    (128, 2, 4, [700, 1, 33, 2000], None, 0, 0),
    (128, 1, 4, [9000], [15], 0, 0),
    (64, 2, 7, [1500, 400], [9, 3], 200, 5),
    (96, 1, 1, [300, 90], [63, 20], 0, 0),
    (160, 1, 8, [500], [5], 0, 0),
    (256, 1, 2, [800, 60], [31, 2], 100, 3),
    (128, 2, 4, [900, 500, 100], [15, 2, 1], 2, 0),
    (64, 2, 8, [900, 500, 100], [7, 2, 1], 3, 2),
    (128, 8, 1, [700] * 8, None, 33, 0),
]


@pytest.mark.parametrize("d,h_kv,G,lens,rows,window,sinks", FEW)
def test_few_rows_over_e4m3_have_weights_of_11_bits(d, h_kv, G, lens, rows, window, sinks):
    """bf16 queries.  Values of either sign, of which a few keys' nearly cancel: there the output's
    own rounding to bf16 is small, and weights of 8 bits are off by 3 tolerances (windows of 2 to
    33 keys)."""
    rng = np.random.default_rng(53)
    pages = sum(-(-n // 64) for n in lens)
    cache = make_cache(rng, pages, 64, h_kv, d, F8)
    batch, table, seqs = make_batch(rng, pages, 64, lens, rows)
    q = randn(rng, batch.num_rows, h_kv * G, d, scale=1.5)
    got = T.F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    want = attention64(cache, table, seqs, q, 1 / math.sqrt(d), window, sinks, 2.0 ** -11)
    check(got, want)
    # the weights alone: an fp32 row's output is not rounded, and its weights have 21 bits
    got = T.F.kv_attention(cache, batch, q.float(), window=window, sinks=sinks)
    check(got, attention64(cache, table, seqs, q.float(), 1 / math.sqrt(d), window, sinks, 2.0 ** -21, 2.0 ** -24))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.3, -0.01, 2.0, 1e-30])
@pytest.mark.parametrize("d,G,rows", [(64, 4, 150), (96, 2, 100), (128, 8, 40), (256, 4, 90)])
def test_many_rows_with_any_scale(d, G, rows, scale, dtype):
    rng = np.random.default_rng(54)
    ct = BF16 if dtype == "bf16" else F8
    cache = make_cache(rng, 8, 64, 1, d, ct)
    batch, table, seqs = make_batch(rng, 8, 64, [400], [rows])
    q = randn(rng, rows, G, d)
    got = T.F.kv_attention(cache, batch, q, scale, window=150, sinks=4)
    check(got, attention64(cache, table, seqs, q, scale, 150, 4, WEIGHT[ct, BF16]))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 5, 200])
@pytest.mark.parametrize("power", [79, -80])
def test_values_far_from_one(power, rows, qt, dtype):
    """Values just below 2^80, where sums of weights times values may first overflow, and small
    ones: the result scales with them."""
    rng = np.random.default_rng(55)
    ct, qt = BF16 if dtype == "bf16" else F8, BF16 if qt == "bf16" else F32
    cache = make_cache(rng, 80, 64, 1, 64, ct)
    if ct == BF16:
        cache.v.copy_((cache.v.float() / cache.v.float().abs().max() * 2.0 ** power).to(BF16))
    else:  # |code| < 2^9
        cache.v_scale.fill_(127 + power - 9)
    batch, table, seqs = make_batch(rng, 80, 64, [5000], [rows])
    q = randn(rng, rows, 4, 64, dtype=qt)
    got = T.F.kv_attention(cache, batch, q)
    want = attention64(cache, table, seqs, q, 1 / 8, 0, 0, WEIGHT[ct, qt], 2.0 ** -8 if qt == BF16 else 2.0 ** -24)
    check(got, want)


# ------------------------------------------------------------- what is missing --

@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,G,page", [(128, 4, 64), (64, 8, 16), (256, 4, 128), (96, 4, 48)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 20)])
def test_many_rows_with_pages_and_tokens_missing(d, G, page, window, sinks, dtype):
    """Pages outside the pool in the middle and at the end, more rows than tokens, an empty
    sequence with rows; the workspace and the pages that nobody has are full of NaNs."""
    rng = np.random.default_rng(56)
    ct = BF16 if dtype == "bf16" else F8
    lens, rows = [700, 150, 0, 384], [300, 200, 70, 384]
    pages = sum(-(-n // page) for n in lens) + 3
    cache = make_cache(rng, pages, page, 1, d, ct)
    batch, _, _ = make_batch(rng, pages, page, lens, rows)
    table = batch.page_table.cpu().numpy()
    width = table.shape[1]
    free = sorted(set(range(pages)) - set(table[table >= 0].tolist()))
    for at, bad in ((250 // page, -1), (460 // page, pages), (690 // page, 1 << 30)):
        free.append(int(table[0, at]))
        table[0, at] = bad
    free.append(int(table[3, 0]))
    table[3, 0] = -(1 << 31)
    for x in (cache.k, cache.v):
        if ct == BF16:
            x[free] = math.nan
        else:
            x.view(torch.uint8)[free] = 0x7f
    batch.page_table.copy_(torch.from_numpy(table))
    seqs = [(sum(rows[:i]), rows[i], lens[i]) for i in range(4)]
    q = randn(rng, sum(rows), G, d)
    ws = T.F.Workspace()
    ws.get(64 << 20).fill_(255)
    got = T.F.kv_attention(cache, batch, q, window=window, sinks=sinks, workspace=ws)
    assert width == table.shape[1] and ws.buf.numel() == (64 << 20) + 256
    check(got, attention64(cache, table, seqs, q, 1 / math.sqrt(d), window, sinks, WEIGHT[ct, BF16]))
    T.F.check_device_status(ws)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("m,bad,window,sinks", [(6, 196, 0, 0), (200, 120, 0, 0), (150, 60, 50, 3), (150, 2, 50, 3)])
def test_a_key_that_is_not_finite_spoils_the_rows_that_see_it(m, bad, window, sinks, dtype):
    rng = np.random.default_rng(57)
    n, page = 200, 64
    cache = make_cache(rng, 5, page, 2, 128, BF16 if dtype == "bf16" else F8)
    batch, table, _ = make_batch(rng, 5, page, [n], [m])
    q = randn(rng, m, 8, 128)
    want = T.F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    at = (table[0][bad // page], 1, bad % page)  # of KV head 1
    if dtype == "bf16":
        cache.k[at] = math.nan
    else:
        cache.k.view(torch.uint8)[at] = 0x7f
    got = T.F.kv_attention(cache, batch, q, window=window, sinks=sinks)
    p = torch.arange(n - m, n, device="cuda")
    sees = (bad <= p) & ((p - bad < window) | (bad < sinks) if window else torch.ones_like(p, dtype=torch.bool))
    assert sees.any() and torch.isnan(got[0][sees, 4:]).all()
    for g, w in zip(got, want):
        assert torch.equal(g[:, :4], w[:, :4]) and torch.equal(g[~sees], w[~sees])
