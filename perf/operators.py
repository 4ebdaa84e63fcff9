"""The paged KV cache's operators as they are used in serving: their cases, their plain forms and the library's calls.

  append     new keys and values into a paged cache (bf16, or e4m3 with one power-of-two scale per 16 tokens and
             KV head), keys and queries rotated by their positions on the way
  attention  each new token's attention over its sequence in such a cache, every earlier token visible
  window     the same with a sliding window and a few first tokens that stay visible

`own` false: elementary torch operations in 32 bits (angles in 64); `own` true: the library's calls.
"""

import math
import random

import torch

own = False

BLOCK = 16        # tokens that share a scale in an e4m3 cache
X_LO, X_HI = 8, 246  # the scale's exponent byte x: scale 2^(x - 127)


# ------------------------------------------------------------------ cases --

def listed():
    """seqs sequences of n_lo..n_hi tokens (the first has n_hi), the last rows_lo..rows_hi of each new in this call."""
    def case(name, op, cache, seqs, n_lo, n_hi, rows_lo=1, rows_hi=1, h_q=32, h_kv=8, d=128, page=64, q="bf16",
             window=0, sinks=0, mix=0):
        return dict(name=name, op=op, cache=cache, seqs=seqs, n_lo=n_lo, n_hi=n_hi, rows_lo=rows_lo,
                    rows_hi=rows_hi, h_q=h_q, h_kv=h_kv, d=d, page=page, q=q, window=window, sinks=sinks, mix=mix)
    return [
        # one session's decoded token, late in a 131072-token context: nothing but latency
        case("append_one_bf16", "append", "bf16", 1, 131071, 131071),
        # a decode step of 48 sessions: each token goes into a block that mostly holds older ones
        case("append_step_e4m3", "append", "e4m3", 48, 300, 4096, page=32, mix=1),
        # a continued prompt: 8192 new tokens behind 1000 cached ones
        case("append_prompt_bf16", "append", "bf16", 1, 9192, 9192, 8192, 8192),
        # three prompts of uneven length taken in together
        case("append_prompts_e4m3", "append", "e4m3", 3, 5003, 16384, 5003, 16384, page=128, mix=2),
        # one session's decode step over a short cache: latency
        case("q8_decode_one", "attention", "e4m3", 1, 4099, 4099, mix=3),
        # a decode step of ragged sessions
        case("q8_decode_ragged", "attention", "e4m3", 24, 4096, 65536, mix=4),
        # the 1M-token decode step
        case("q8_decode_1m", "attention", "e4m3", 1, 1 << 20, 1 << 20, page=256, mix=5),
        # a prompt's last chunk: 4096 tokens over a 32768-token cache
        case("q8_chunk", "attention", "e4m3", 1, 32768, 32768, 4096, 4096, mix=6),
        # a windowed layer of one long session, fp32 queries
        case("window_decode_one_f32", "window", "bf16", 1, 131072, 131072, q="f32", window=1024, sinks=4, mix=7),
        # a windowed layer's decode step of 64 sessions, some shorter than the window
        case("window_decode_batch", "window", "bf16", 64, 100, 12000, window=4096, sinks=4, page=16, mix=8),
        # a few drafted tokens a session, narrow heads, e4m3
        case("window_draft_e4m3", "window", "e4m3", 16, 700, 30000, 3, 6, h_q=16, d=64, window=2000, sinks=16, mix=9),
        # a prompt through a windowed layer
        case("window_prompt", "window", "bf16", 1, 8192, 8192, 8192, 8192, window=2048, sinks=4, mix=10),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "window"])
    cache = rng.choice(["bf16", "e4m3"]) if op != "attention" else "e4m3"
    h_q, h_kv = rng.choice([(32, 8), (16, 8), (8, 8), (28, 4), (64, 8), (16, 4)])
    d = rng.choice([64, 128, 128, 128, 256, 96])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    prompt = rng.random() < 0.4
    if prompt:
        seqs = rng.choice([1, 1, 2, 3])
        rows_hi = _spread(rng, 17, 4096)
        n_hi = rows_hi + rng.choice([0, _spread(rng, 1, 16384)])
        n_lo, rows_lo = max(1, n_hi // 2), max(1, rows_hi // 2)
    else:
        seqs = _spread(rng, 1, 64)
        n_hi = _spread(rng, 40, 262144 // seqs)
        n_lo, rows_hi = max(1, n_hi // 8), rng.choice([1, 1, 1, 1, 4])
        rows_lo = 1
    window = sinks = 0
    if op == "window":
        window, sinks = _spread(rng, 16, 8192), rng.choice([0, 1, 4, 16, 100])
    q = rng.choice(["bf16", "bf16", "bf16", "f32"]) if not prompt else "bf16"
    return dict(op=op, cache=cache, seqs=seqs, n_lo=n_lo, n_hi=n_hi, rows_lo=rows_lo, rows_hi=rows_hi, h_q=h_q,
                h_kv=h_kv, d=d, page=page, q=q, window=window, sinks=sinks, mix=rng.randrange(1 << 20))


def _lengths(c):
    """(n_s, m_s) of each sequence: tokens in all, new tokens among them."""
    rng = random.Random(c["mix"])
    ns = [c["n_hi"]] + [rng.randint(c["n_lo"], c["n_hi"]) for _ in range(c["seqs"] - 1)]
    ms = [c["rows_hi"]] + [rng.randint(c["rows_lo"], c["rows_hi"]) for _ in range(c["seqs"] - 1)]
    return ns, [min(n, m) for n, m in zip(ns, ms)]


def _visible(c, n, m):
    """(query-key pairs, distinct keys) that m new tokens behind n - m older ones see."""
    w, s = c["window"], c["sinks"]
    if not w:
        return sum(range(n - m + 1, n + 1)), n
    pairs = sum(p + 1 if p + 1 <= w else w + min(s, p + 1 - w) for p in range(n - m, n))
    first = max(0, n - m - w + 1)  # the first new token's window
    return pairs, n - first + min(s, first)


def work(case):
    c = case
    ns, ms = _lengths(c)
    rows = sum(ms)
    qb = 4 if c["q"] == "f32" else 2
    cb = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        b = 2 * rows * c["h_kv"] * c["d"] * (2 + cb) + 2 * rows * c["h_q"] * c["d"] * qb
        return {"bytes": b, "flops": 3 * rows * (c["h_q"] + c["h_kv"]) * c["d"]}
    seen = [_visible(c, n, m) for n, m in zip(ns, ms)]
    keys, pairs = sum(k for _, k in seen), sum(p for p, _ in seen)
    b = 2 * keys * c["h_kv"] * c["d"] * cb + 2 * rows * c["h_q"] * c["d"] * qb + 4 * rows * c["h_q"]
    if c["cache"] == "e4m3":
        b += 2 * keys * c["h_kv"] // BLOCK
    return {"bytes": b, "flops": 4 * pairs * c["h_q"] * c["d"]}


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    ns, ms = _lengths(c)
    page, h_kv, h_q, d = c["page"], c["h_kv"], c["h_q"], c["d"]
    width = max(-(-n // page) for n in ns)
    pages = sum(-(-n // page) for n in ns)
    # pages handed out in no particular order, as a pool that has been in use has them
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((len(ns), width), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(ns):
        w = -(-n // page)
        table[s, :w] = order[at:at + w]
        at += w

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # keys with a mean and a spread for each channel
    mean = rand(h_kv, 1, d)
    spread = torch.exp(torch.rand((h_kv, 1, d), generator=g, device=dev) * 2 - 1)
    st = {"case": c, "table": table, "seq_len": torch.tensor(ns, dtype=torch.int32, device=dev),
          "q_start": torch.tensor([sum(ms[:i]) for i in range(len(ms) + 1)], dtype=torch.int32, device=dev),
          "max_rows": max(ms), "max_len": max(ns), "rows": sum(ms)}
    for name in ("k", "v"):
        x = torch.empty((pages, h_kv, page, d), dtype=torch.float32, device=dev).normal_(generator=g)
        if name == "k":
            x.mul_(spread).add_(mean)
        if c["cache"] == "bf16":
            st[name] = x.to(torch.bfloat16)
        else:
            b = x.view(pages, h_kv, page // BLOCK, BLOCK, d)
            e = torch.ceil(torch.log2(b.abs().amax((3, 4)) / 256))
            b.mul_(torch.exp2(-e)[..., None, None])
            st[name] = x.to(torch.float8_e4m3fn)
            st[name + "_scale"] = (e + 127).to(torch.uint8)
        del x
    qt = torch.float32 if c["q"] == "f32" else torch.bfloat16
    st["q"] = (rand(st["rows"], h_q, d) * (1.0 if c["op"] == "append" else 2.0)).to(qt)
    if c["op"] == "append":
        st["k_new"] = (rand(st["rows"], h_kv, d) * spread[:, 0] + mean[:, 0]).to(torch.bfloat16)
        st["v_new"] = rand(st["rows"], h_kv, d).to(torch.bfloat16)
        st["inv_freq"] = 1e6 ** (-torch.arange(0, d, 2, device=dev, dtype=torch.float64) / d)
        st["inv_freq"] = st["inv_freq"].to(torch.float32)
    st["scale"] = 1.0 / math.sqrt(d)
    if own:  # the cache's and the step's handles, which a serving loop keeps
        import bit_plane_kv_scan_b200 as F
        st["cache"] = F.KVCache(st["k"], st["v"], st.get("k_scale"), st.get("v_scale"))
        st["batch"] = F.KVBatch(table, st["seq_len"], st["q_start"], num_rows=st["rows"],
                                max_rows=st["max_rows"], max_len=st["max_len"])
    return st


def run(state):
    if own:
        return _own_append(state) if state["case"]["op"] == "append" else _own_attention(state)
    return _append(state) if state["case"]["op"] == "append" else _attention(state)


def _own_append(st):
    import bit_plane_kv_scan_b200 as F
    q = F.kv_append(st["cache"], st["batch"], st["k_new"], st["v_new"], q=st["q"], inv_freq=st["inv_freq"])
    return _written(st, q)


def _own_attention(st):
    import bit_plane_kv_scan_b200 as F
    c = st["case"]
    out, lse = F.kv_attention(st["cache"], st["batch"], st["q"], st["scale"], window=c["window"], sinks=c["sinks"])
    return {"out": out, "lse": lse}


def _written(st, q):
    names = ("k", "v") if st["case"]["cache"] == "bf16" else ("k", "v", "k_scale", "v_scale")
    return {"q": q, **{n: st[n] for n in names}}


# -------------------------------------------------------------- plain forms --

def _rows(st):
    """Of each new token: its sequence and its position."""
    start = st["q_start"].long()
    i = torch.arange(st["rows"], device=start.device)
    seq = torch.searchsorted(start, i, right=True) - 1
    return seq, i - start[seq + 1] + st["seq_len"].long()[seq]


def _rotate(x, cos, sin):
    x = x.float()
    a, b = x.chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)


def _append(st):
    c = st["case"]
    page = c["page"]
    seq, pos = _rows(st)
    where = st["table"].long()[seq, pos // page]
    slot = pos % page
    angle = pos.double()[:, None] * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _rotate(st["q"], cos, sin).to(st["q"].dtype)
    new = {"k": _rotate(st["k_new"], cos, sin), "v": st["v_new"].float()}
    raw = {"k": st["k_new"], "v": st["v_new"]}
    if c["cache"] == "bf16":
        for name in ("k", "v"):
            st[name][where, :, slot] = new[name].to(torch.bfloat16)
        return _written(st, q)
    # the block that a sequence's first new token falls into, and the tokens that it held
    older = (st["seq_len"] - st["q_start"].diff()).long()
    held = torch.where(st["q_start"].diff() > 0, older % BLOCK, 0)
    sp = st["table"].long().gather(1, (older // page).clamp(max=st["table"].shape[1] - 1)[:, None])[:, 0]
    sb = older % page // BLOCK
    blk = where * (page // BLOCK) + slot // BLOCK
    for name in ("k", "v"):
        scale = st[name + "_scale"]  # [pages, h_kv, blocks]
        n_blk = scale.shape[0] * scale.shape[2]
        big = torch.zeros((n_blk, c["h_kv"]), dtype=torch.float32, device=scale.device)
        big.index_reduce_(0, blk, raw[name].float().abs().amax(-1), "amax")
        mant, ex = torch.frexp(big)
        x = torch.where(mant == 0.5, ex - 1, ex) - 8 + 127
        x = torch.where(big == 0, X_LO, x).clamp(X_LO, X_HI)
        x = x.view(scale.shape[0], scale.shape[2], c["h_kv"]).transpose(1, 2)
        old = scale[sp, :, sb].int()  # [seqs, h_kv]
        grown = torch.maximum(old, x[sp, :, sb])
        x[sp, :, sb] = torch.where((held > 0)[:, None], grown, x[sp, :, sb])
        # what the block held moves to its new scale
        tok = torch.arange(BLOCK, device=scale.device)
        codes = st[name].view(torch.uint8).view(scale.shape[0], c["h_kv"], -1, BLOCK, c["d"])
        was = codes[sp, :, sb]  # [seqs, h_kv, BLOCK, d]
        moved = was.view(torch.float8_e4m3fn).float() * torch.exp2((old - grown).float())[..., None, None]
        moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[sp, :, sb] = torch.where((tok < held[:, None])[:, None, :, None], moved, was)
        e = (x[where, :, slot // BLOCK] - 127).float()  # [rows, h_kv]
        put = (new[name] * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn)
        st[name].view(torch.uint8)[where, :, slot] = put.view(torch.uint8)
        scale[where, :, slot // BLOCK] = x[where, :, slot // BLOCK].to(torch.uint8)
    return _written(st, q)


def _sequences(st, name):
    """The cache's rows in order, [seqs, h_kv, tokens, d], in 32 bits."""
    c = st["case"]
    t = st["table"].long()
    x = st[name][t] if c["cache"] == "bf16" else st[name].view(torch.uint8)[t].view(torch.float8_e4m3fn)
    x = x.float()  # [seqs, width, h_kv, page, d]
    if c["cache"] == "e4m3":
        e = torch.exp2(st[name + "_scale"][t].float() - 127)
        x = (x.unflatten(3, (-1, BLOCK)) * e[..., None, None]).flatten(3, 4)
    return x.transpose(1, 2).flatten(2, 3)


def _attention(st):
    c = st["case"]
    seqs, h_kv, d, r = c["seqs"], c["h_kv"], c["d"], st["max_rows"]
    grp = c["h_q"] // h_kv
    seq, pos = _rows(st)
    at = torch.arange(st["rows"], device=pos.device) - st["q_start"].long()[seq]
    # queries by sequence, one behind the other: [seqs, h_kv, grp * r, d]
    q = torch.zeros((seqs, r, h_kv, grp, d), dtype=torch.float32, device=pos.device)
    q[seq, at] = st["q"].float().view(-1, h_kv, grp, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(seqs, h_kv, grp * r, d)
    p = torch.full((seqs, r), -1, device=pos.device)
    p[seq, at] = pos
    k = _sequences(st, "k")
    s = (q @ k.transpose(2, 3)).mul_(st["scale"]).view(seqs, h_kv, grp, r, -1)
    del k
    j = torch.arange(s.shape[-1], device=pos.device)
    see = j <= p[..., None]
    if c["window"]:
        see &= (j < c["sinks"]) | (j > p[..., None] - c["window"])
    s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    out = s.flatten(2, 3) @ _sequences(st, "v") / total.flatten(2, 3).clamp(min=1e-37)
    out = out.view(seqs, h_kv, grp, r, d).permute(0, 3, 1, 2, 4)[seq, at]
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)[seq, at]
    return {"out": out.flatten(1, 2).to(st["q"].dtype), "lse": lse.flatten(1, 2).contiguous()}


# ------------------------------------------------------------------- 64 bits --

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    ns, ms = _lengths(case)
    return _exact_append(st, ns, ms) if case["op"] == "append" else _exact_attention(st, ns, ms)


def _exact_append(st, ns, ms):
    c = st["case"]
    page = c["page"]
    q = torch.empty_like(st["q"], dtype=torch.float64)
    out = {n: st[n].double() for n in ("k", "v")}
    row = 0
    for s, (n, m) in enumerate(zip(ns, ms)):
        p = torch.arange(n - m, n, device=q.device, dtype=torch.float64)
        z = torch.polar(torch.ones((), dtype=torch.float64, device=q.device),
                        p[:, None] * st["inv_freq"].double())[:, None]

        def turn(x):
            w = torch.complex(x[..., :c["d"] // 2].double(), x[..., c["d"] // 2:].double()) * z
            return torch.cat((w.real, w.imag), -1)

        part = slice(row, row + m)
        row += m
        q[part] = turn(st["q"][part])
        first = (n - m) // BLOCK * BLOCK
        j = torch.arange(first, n, device=q.device)
        pg, sl = st["table"][s, j // page].long(), j % page
        for name, raw, val in (("k", st["k_new"][part], turn(st["k_new"][part])),
                               ("v", st["v_new"][part], st["v_new"][part].double())):
            if c["cache"] == "bf16":
                out[name][pg[n - m - first:], :, sl[n - m - first:]] = val
                continue
            held = n - m - first
            for b in range(0, n - first, BLOCK):
                e_page, e_blk = int(pg[b]), int(sl[b]) // BLOCK
                lo, hi = max(b - held, 0), b - held + BLOCK  # the block's new tokens
                a = raw[lo:hi].double().abs().amax((0, 2))
                e = torch.ceil(torch.log2(a) - 8).clamp(X_LO - 127, X_HI - 127)
                if b == 0 and held:
                    old = st[name + "_scale"][e_page, :, e_blk].double() - 127
                    e = torch.maximum(e, old)
                    rows = slice(e_blk * BLOCK, e_blk * BLOCK + held)
                    kept = out[name][e_page, :, rows] * torch.exp2(old - e)[:, None, None]
                    out[name][e_page, :, rows] = kept.to(torch.float8_e4m3fn).double()
                put = val[lo:hi].transpose(0, 1) * torch.exp2(-e)[:, None, None]
                t0 = int(sl[b]) + (held if b == 0 else 0)
                out[name][e_page, :, t0:t0 + put.shape[1]] = put
    if c["cache"] == "e4m3":
        out = {"k": out["k"], "v": out["v"], "k_scale": None, "v_scale": None}
    return {"q": q, **out}


def _exact_attention(st, ns, ms):
    c = st["case"]
    page, grp = c["page"], c["h_q"] // c["h_kv"]
    out = torch.empty_like(st["q"], dtype=torch.float64)
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device=out.device)
    row = 0
    for s, (n, m) in enumerate(zip(ns, ms)):
        j = torch.arange(n, device=out.device)
        pg, sl = st["table"][s, j // page].long(), j % page
        for h in range(c["h_kv"]):
            kv = []
            for name in ("k", "v"):
                x = st[name].view(torch.uint8) if c["cache"] == "e4m3" else st[name]
                x = x[pg, h, sl]
                x = x.view(torch.float8_e4m3fn).double() if c["cache"] == "e4m3" else x.double()
                if c["cache"] == "e4m3":
                    x *= torch.exp2(st[name + "_scale"][pg, h, sl // BLOCK].double() - 127)[:, None]
                kv.append(x)
            heads = slice(h * grp, (h + 1) * grp)
            for r in range(0, m, 512):
                e = min(m, r + 512)
                at = slice(row + r, row + e)
                p = torch.arange(n - m + r, n - m + e, device=out.device)[:, None, None]
                w = st["q"][at, heads].double() @ kv[0].T * st["scale"]
                hide = j > p
                if c["window"]:
                    hide = hide | ((j >= c["sinks"]) & (j <= p - c["window"]))
                w = w.masked_fill(hide, -math.inf)
                lse[at, heads] = torch.logsumexp(w, -1)
                out[at, heads] = torch.softmax(w, -1) @ kv[1]
        row += m
    return {"out": out, "lse": lse}
