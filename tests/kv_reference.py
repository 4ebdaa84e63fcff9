"""Plain fp64 statements of the paged cache's operators, and the tolerances of
their tests.

Tolerances, each from what the kernels round (half a step of a type, relative to
the value: bf16 2^-8, fp16 2^-11, fp32 2^-24, e4m3 2^-4):
  * rotation: the reduced angle is rounded to fp32 (|a| <= pi, so off by
    2^-23), sine and cosine are within 2 steps of fp32, two products and a sum
    follow: each term is within 6 * 2^-23 of its exact value in all, so an element
    is within ROT (|x| + |y|), ROT = 2^-20, before it is rounded to its type;
  * attention: with A = sum_j softmax_j |v_j| per dimension,
      - a score is a sum of d products in d / 16 MMAs, each adding 17 terms cut
        to fp32 (2^-22 of the magnitudes in sum covers that), scaled twice:
        delta = (d / 16 + 4) 2^-22 B, B = max_j scale sum_c |q_c k_jc|; the
        weights and their sum are each off by a factor 1 +- delta (and 2^-20
        for exp2): 2 (delta + 2^-20) A;
      - the weights that meet V are rounded (bf16: 2^-8; fp16, the 8-bit cache:
        2^-11; fp32 queries: split, 2^-21), their sum is not: weight A;
      - V's products are summed over the keys, 16 at a time: (n / 16 + 16) 2^-22 A;
      - out is rounded to its type.
    lse is off by delta, the sum's 2^-20 + (n / 16 + 16) 2^-23, and its own
    rounding 2^-22 max(1, |lse|).
"""

import math

import numpy as np
import torch

ROT = 2.0 ** -20
BLOCK = 16
X_LO, X_HI = 8, 246


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(x):
    return x.detach().cpu().to(torch.float64).numpy()


def bytes_of(x):
    return x.detach().cpu().view(torch.uint8).numpy()


def e4m3_value(codes):
    """uint8 codes -> their fp64 values."""
    t = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn)
    return t.to(torch.float64).numpy()


def e4m3_code(x):
    """fp64 -> nearest e4m3 code (ties to even, saturating), by search in the table."""
    table = e4m3_value(np.arange(127, dtype=np.uint8))  # 0 .. 448, increasing
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - a, a - table[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def sequences(seq_len, q_start, max_len=None):
    """[(row0, rows, len)] of well-formed sequences."""
    n = len(seq_len)
    starts = list(range(n + 1)) if q_start is None else list(q_start)
    return [(int(starts[s]), int(starts[s + 1] - starts[s]), int(seq_len[s])) for s in range(n)]


def rotate(x, pos, inv_freq, interleaved):
    """x [rows, heads, d] fp64 -> (rotated, |x| + |y| of each element's pair)."""
    out, mag = x.copy(), np.abs(x)
    r = 0 if inv_freq is None else len(inv_freq)
    if r == 0:
        return out, mag
    a = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
    i = np.arange(r)
    at, to = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    p, q = x[..., at], x[..., to]
    out[..., at] = p * np.cos(a) - q * np.sin(a)
    out[..., to] = q * np.cos(a) + p * np.sin(a)
    mag[..., at] = mag[..., to] = np.abs(p) + np.abs(q)
    return out, mag


def block_byte(big):
    """The scale's byte for the largest element `big` of a block's new ones."""
    if big == 0:
        return X_LO
    m, e = math.frexp(big)  # big = m 2^e, 1/2 <= m < 1
    return min(max((e - 1 if m == 0.5 else e) - 8 + 127, X_LO), X_HI)


class Cache:
    """A paged cache in numpy: fp64 values (bf16) or codes and scale bytes (e4m3)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self.e4m3 = k.dtype == torch.float8_e4m3fn
        self.k, self.v = (bytes_of(x).copy() if self.e4m3 else f64(x) for x in (k, v))
        self.scales = [x.cpu().numpy().copy() for x in (k_scale, v_scale)] if self.e4m3 else None
        self.page = k.shape[2]

    def value(self, side, page, g, rows):
        x = (self.k, self.v)[side][page, g, rows]
        if not self.e4m3:
            return x
        s = np.repeat(self.scales[side][page, g].astype(int), BLOCK)[rows]
        return e4m3_value(x) * 2.0 ** (np.clip(s, X_LO, X_HI) - 127.0)[:, None]

    def sequence(self, side, table, g, n):
        """[n, d]; tokens whose page is outside the pool are NaN with ok False."""
        d = self.k.shape[-1]
        out, ok = np.full((n, d), np.nan), np.zeros(n, bool)
        for p in range(-(-n // self.page)):
            if p >= len(table) or not 0 <= table[p] < self.k.shape[0]:
                continue
            m = min(self.page, n - p * self.page)
            out[p * self.page:p * self.page + m] = self.value(side, table[p], g, slice(0, m))
            ok[p * self.page:p * self.page + m] = True
        return out, ok

    def append(self, table, seqs, k, v, inv_freq=None, interleaved=False):
        """Writes the rows (bf16: not rounded); returns for each side the places written:
        [(page, slot, values [h_kv, d], pair magnitudes)]."""
        done = ([], [])
        for s, (row0, m, n) in enumerate(seqs):
            pos = np.arange(n - m, n)
            for side, x in ((0, k), (1, v)):
                raw = x[row0:row0 + m]
                val, mag = rotate(raw, pos, inv_freq if side == 0 else None, interleaved)
                for b in range((n - m) // BLOCK, (n - 1) // BLOCK + 1 if m else 0):
                    at = b * BLOCK // self.page
                    if b < 0 or at >= len(table[s]) or not 0 <= table[s][at] < self.k.shape[0]:
                        continue
                    page, slot = table[s][at], b * BLOCK % self.page
                    new = np.nonzero((pos >= b * BLOCK) & (pos < (b + 1) * BLOCK))[0]
                    if len(new) == 0:
                        continue
                    if self.e4m3:
                        self._scale(side, page, slot, pos[new[0]] - b * BLOCK, raw[new])
                    for i in new:
                        at_slot = slot + pos[i] - b * BLOCK
                        done[side].append((page, at_slot, val[i], mag[i]))
                        if self.e4m3:
                            x8 = self.scales[side][page, :, slot // BLOCK].astype(int)
                            (self.k, self.v)[side][page, :, at_slot] = \
                                e4m3_code(val[i] * 2.0 ** (127.0 - x8)[:, None])
                        else:
                            (self.k, self.v)[side][page, :, at_slot] = val[i]
        return done

    def _scale(self, side, page, slot, held, raw):
        codes = (self.k, self.v)[side]
        for g in range(raw.shape[1]):
            x = block_byte(np.abs(raw[:, g][np.isfinite(raw[:, g])]).max(initial=0.0))
            if held:
                was = int(np.clip(self.scales[side][page, g, slot // BLOCK], X_LO, X_HI))
                x = max(x, was)
                if x > was:
                    rows = slice(slot, slot + held)
                    codes[page, g, rows] = e4m3_code(e4m3_value(codes[page, g, rows]) * 2.0 ** (was - x))
            self.scales[side][page, g, slot // BLOCK] = x


def attention(cache, table, seqs, q, scale, window=0, sinks=0, weight_step=2.0 ** -8,
              out_step=2.0 ** -8):
    """(out, lse, tolerance of out, tolerance of lse) for q [rows, h_q, d] fp64; rows that
    no sequence has are NaN."""
    rows, h_q, d = q.shape
    h_kv = cache.k.shape[1]
    out, tol = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse, ltol = np.full((rows, h_q), np.nan), np.zeros((rows, h_q))
    for s, (row0, m, n) in enumerate(seqs):
        if m == 0:
            continue
        for g in range(h_kv):
            k, ok = cache.sequence(0, table[s], g, n)
            v, _ = cache.sequence(1, table[s], g, n)
            j = np.arange(n)
            for i in range(m):
                p = n - m + i
                see = (j <= p) & ok
                if window:
                    see &= (j > p - window) | (j < sinks)
                for h in range(g * (h_q // h_kv), (g + 1) * (h_q // h_kv)):
                    r = row0 + i
                    if not see.any():
                        out[r, h], lse[r, h] = 0.0, -np.inf
                        continue
                    kk, vv = k[see], v[see]
                    sc = scale * (kk @ q[r, h])
                    top = sc.max()
                    w = np.exp(sc - top)
                    lse[r, h] = top + math.log(w.sum())
                    w /= w.sum()
                    out[r, h] = w @ vv
                    a = w @ np.abs(vv)
                    b = abs(scale) * (np.abs(kk) @ np.abs(q[r, h])).max()
                    delta = (d / 16 + 4) * 2.0 ** -22 * b
                    adds = len(sc) / 16 + 16
                    tol[r, h] = (2 * (delta + 2.0 ** -20) + weight_step + adds * 2.0 ** -22) * a \
                        + out_step * np.abs(out[r, h]) + 1e-30
                    ltol[r, h] = delta + 2.0 ** -20 + adds * 2.0 ** -23 \
                        + 2.0 ** -22 * max(1.0, abs(lse[r, h]))
    return out, lse, tol, ltol
