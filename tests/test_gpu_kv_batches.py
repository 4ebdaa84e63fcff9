"""The paged cache's calls on the GPU over batches whose row ranges are partly wrong:
sequences that break a bound have no rows, the others are served as ever."""

import math

import numpy as np
import pytest
import torch

import kv_reference as R
import test_gpu_kv as T
from test_gpu_kv import BF16, F8, WEIGHT, _lib, check_append, check_attention, make_cache, randn, ref_cache  # noqa: F401

pytestmark = pytest.mark.gpu
WILD = (-1, -1000, -(1 << 31), (1 << 31) - 1, 1 << 20)


def served(start, lens, num_rows, max_rows):
    """[(row0, rows, len)], rows 0 where the range breaks a bound."""
    start = [int(x) for x in start]
    ok = [0 <= a <= b <= num_rows and b - a <= max_rows for a, b in zip(start, start[1:])]
    return [(a, b - a if o else 0, int(n)) for a, b, n, o in zip(start, start[1:], lens, ok)]


def ranges(rng, seqs, most, bad):
    """q_start of `seqs` sequences with up to `most` rows each, `bad` entries of it wild."""
    start = np.concatenate([[0], np.cumsum(rng.integers(0, most + 1, seqs))])
    num_rows = int(start[-1]) + 3
    if seqs >= 4:  # one long one among them
        start[seqs // 2:] += most * 8
        num_rows += most * 8
    at = rng.choice(seqs + 1, bad, replace=False)
    start[at] = rng.choice(WILD, bad)
    return start.astype(np.int64), num_rows, most * 9


CASES = [("five", [0, 5, -1000, 6, 7], 8, 8), ("wild", [0, 50, 30, 31, -3, 35, 36], 40, 20),
         ("late", [4, 9, 9, 30], 40, 20), ("beyond", [0, 5, 60, 70, 80], 40, 20),
         ("long", [0, 3, 30, 33, 34], 40, 20)]


def _case(name):
    if isinstance(name, int):
        rng = np.random.default_rng(name)
        start, num_rows, max_rows = ranges(rng, name, 6 if name > 100 else 20, max(2, name // 20))
    else:
        _, start, num_rows, max_rows = next(c for c in CASES if c[0] == name)
        rng = np.random.default_rng(40)
    seqs = len(start) - 1
    lens = np.minimum(rng.integers(1, 90, seqs) + (np.diff(start) * (np.abs(np.diff(start)) < 1000)).clip(0), 400)
    page = 16
    width = -(-int(lens.max()) // page)
    pages = int(sum(-(-lens // page))) + 2
    table = np.full((seqs, width), -1, dtype=np.int32)
    order, at = rng.permutation(pages), 0
    for s, n in enumerate(lens):
        w = -(-int(n) // page)
        table[s, :w] = order[at:at + w]
        at += w
    batch = T.F.KVBatch(torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(),
                        torch.from_numpy(np.asarray(start, dtype=np.int64).astype(np.int32)).cuda(),
                        num_rows=num_rows, max_rows=max_rows)
    return rng, batch, table, pages, page, served(start, lens, num_rows, max_rows)


NAMES = [c[0] for c in CASES] + [33, 70, 200, 1100]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", NAMES)
def test_append_serves_the_sequences_that_keep_their_bounds(name, dtype):
    rng, batch, table, pages, page, seqs = _case(name)
    assert any(m for _, m, _ in seqs)
    cache = make_cache(rng, pages, page, 1, 32, BF16 if dtype == "bf16" else F8)
    k, v, q = (randn(rng, batch.num_rows, h, 32) for h in (1, 1, 2))
    qo = torch.full_like(q, 7.0)
    f = torch.full((16,), 0.01, device="cuda")
    before = ref_cache(cache)
    T.F.kv_append(cache, batch, k, v, q=q, inv_freq=f, q_out=qo)
    torch.cuda.synchronize()
    check_append(before, cache, table, seqs, k, v, f, False)
    left = np.ones(batch.num_rows, bool)
    got, x = R.f64(qo), R.f64(q)
    for row0, m, n in seqs:
        rows = slice(row0, row0 + m)
        if m:
            left[rows] = False
            want, mag = R.rotate(x[rows], np.arange(n - m, n), R.f64(f), False)
            assert (np.abs(got[rows] - want) <= R.ROT * mag + 2.0 ** -8 * np.abs(want)).all()
    assert (got[left] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("G", [2, 8])
@pytest.mark.parametrize("name", NAMES)
def test_attention_serves_the_sequences_that_keep_their_bounds(name, G, dtype):
    rng, batch, table, pages, page, seqs = _case(name)
    ct = BF16 if dtype == "bf16" else F8
    cache = make_cache(rng, pages, page, 1, 64, ct)
    q = randn(rng, batch.num_rows, G, 64)
    out = torch.full_like(q, 7.0)
    lse = torch.full((batch.num_rows, G), 7.0, device="cuda")
    ws = T.F.Workspace()
    T.F.kv_attention(cache, batch, q, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    want = R.attention(ref_cache(cache), table, seqs, R.f64(q), 1 / 8, weight_step=WEIGHT[ct, BF16])
    check_attention((out, lse), want, str(name))
    nobody = torch.from_numpy(np.isnan(want[1])).cuda()
    assert (out[nobody] == 7.0).all() and (lse[nobody] == 7.0).all()
    start = batch.q_start.tolist()
    broken = sum(not (0 <= a <= b <= batch.num_rows and b - a <= batch.max_rows)
                 for a, b in zip(start, start[1:]))
    if broken:
        with pytest.raises(T.F.FathomError, match="%d faults" % broken):
            T.F.check_device_status(ws)
    else:
        T.F.check_device_status(ws)
    assert math.isfinite(float(out.float().abs().max()))


def test_status_of_a_call_without_rows():
    """The status is the last call's, also where that had nothing to do."""
    rng = np.random.default_rng(41)
    cache = make_cache(rng, 4, 16, 1, 64, BF16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    ws = T.F.Workspace()

    def call(lens, start, rows):
        batch = T.F.KVBatch(table, i32(*lens), i32(*start), num_rows=rows, max_rows=min(rows, 1))
        out, lse = T.F.kv_attention(cache, batch, randn(rng, rows, 2, 64), workspace=ws)
        assert out.shape == (rows, 2, 64) and lse.shape == (rows, 2)

    ws.buf = torch.full((4096,), 77, dtype=torch.uint8, device="cuda")
    call((3, 4), (0, 0, 0), 0)
    T.F.check_device_status(ws)
    call((3, 99), (0, 1, 2), 2)
    with pytest.raises(T.F.FathomError, match="1 faults"):
        T.F.check_device_status(ws)
    call((3, 4), (0, 0, 0), 0)
    T.F.check_device_status(ws)
    call((-3, 400), (0, 0, 0), 0)
    with pytest.raises(T.F.FathomError, match="2 faults"):
        T.F.check_device_status(ws)
    table = table[:0].contiguous()
    T.F.kv_attention(cache, T.F.KVBatch(table, i32()), randn(rng, 0, 2, 64), workspace=ws)
    T.F.check_device_status(ws)
