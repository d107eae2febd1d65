"""Cases and plain forms of the paged 4-bit serving step: per-head norm with rotation, appending latent rows
to a paged cache of 4-bit codes, and sparse attention over that cache.

A row of the cache is d values: e2m1 codes, two to a byte (the even value in the low nibble), and one power-of-two
exponent for each 32 values.  A sequence's logical row r lives in slot r % page of page block_table[seq][r // page].
"""
import math

import torch

own = False

if torch.cuda.is_available():
    _DEV = torch.device("cuda")
else:
    _DEV = torch.device("cpu")

# magnitudes of the eight e2m1 codes; the sign is the code's fourth bit
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ---------------------------------------------------------------------------------------

def _norm(name, b, s, h, d, rd, gap, weight, ragged):
    return {"name": name, "op": "norm_rotary", "b": b, "s": s, "h": h, "d": d, "rd": rd, "gap": gap,
            "weight": weight, "ragged": ragged}


def _append(name, b, s, d, rd, page, window, base, step, norm, ragged):
    return {"name": name, "op": "append", "b": b, "s": s, "d": d, "rd": rd, "page": page, "window": window,
            "base": base, "step": step, "norm": norm, "ragged": ragged}


def _attn(name, b, m, h, win, comp, topk_comp, neg, page, rd, causal):
    return {"name": name, "op": "attention", "b": b, "m": m, "h": h, "d": 512, "win": win, "comp": comp,
            "topk_comp": topk_comp, "neg": neg, "page": page, "rd": rd, "causal": causal}


def listed():
    return [
        # the queries of one decode step of 64 sequences with 64 heads of 512 (latency counts)
        _norm("norm q decode 64x64", 64, 1, 64, 512, 64, 0, False, False),
        # the queries of a 4096-token prefill chunk: the bandwidth case
        _norm("norm q prefill 4096", 1, 4096, 64, 512, 64, 0, False, False),
        # a padded batch of odd chunks, the rows a slice of a wider projection, with a learned weight
        _norm("norm ragged 7x133 slice", 7, 133, 12, 192, 40, 64, True, True),
        # one decode step of 256 sequences: each new latent row into its ring of 128 slots
        _append("append ring decode 256", 256, 1, 512, 64, 64, 128, 0, 1, True, False),
        # a long prompt's compressed rows, one for each 4 positions, behind the ring's 128 rows
        _append("append prompt 8x4096", 8, 4096, 512, 64, 64, 0, 128, 4, True, False),
        # a padded batch of odd chunks, longer than the ring, pages that are no power of two
        _append("append ragged 33x161", 33, 161, 512, 64, 24, 128, 0, 1, True, True),
        # 64 sequences over a full ring of 128 rows, nothing compressed
        _attn("attn decode window", 64, 1, 64, 128, 0, 0, 0.0, 64, 64, False),
        # 32 sequences: ring and 512 of 4096 compressed rows, some entries unseen
        _attn("attn decode comp", 32, 1, 64, 128, 4096, 512, 0.05, 64, 64, False),
        # 256 sequences, 128 heads: ring and 2048 of 32768 compressed rows
        _attn("attn decode large", 256, 1, 128, 128, 32768, 2048, 0.02, 64, 64, False),
        # one 4096-token prefill chunk: causal windows and up to 512 of 1024 compressed rows
        _attn("attn prefill 4096", 1, 4096, 64, 4096, 1024, 512, 0.0, 64, 64, True),
        # one sequence with a share of 16 heads over a long list: few rows of queries, a long axis
        _attn("attn one seq 16 heads", 1, 1, 16, 128, 8192, 2048, 0.0, 64, 64, False),
        # short speculative steps of a few sequences, odd sizes everywhere
        _attn("attn 5x3 ragged", 5, 3, 40, 57, 731, 299, 0.1, 24, 64, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rotary", "append", "attention", "attention"))
    if op == "norm_rotary":
        d = 8 * _log_int(rng, 4, 128)
        rd = 8 * rng.randint(1, max(1, d // 8))
        h = _log_int(rng, 1, 128)
        b = _log_int(rng, 1, 64)
        s = max(1, min(_log_int(rng, 1, 4096), (64 << 20) // (b * h * d)))
        c = _norm("", b, s, h, d, rd, 8 * rng.randint(0, 16), rng.random() < 0.5, rng.random() < 0.5)
    elif op == "append":
        d = 32 * _log_int(rng, 2, 32)
        rd = 8 * rng.randint(1, max(1, d // 8))
        b = _log_int(rng, 1, 256)
        s = max(1, min(_log_int(rng, 1, 4096), (16 << 20) // (b * d)))
        window = rng.choice((0, _log_int(rng, 8, 512)))
        c = _append("", b, s, d, rd, _log_int(rng, 1, 256), window, rng.randint(0, 200), rng.choice((1, 1, 4)),
                    rng.random() < 0.7, rng.random() < 0.5)
    else:
        b = _log_int(rng, 1, 256)
        m = _log_int(rng, 1, 64)
        h = _log_int(rng, 1, 128)
        win = _log_int(rng, 1, 300)
        comp = _log_int(rng, 1, 16384)
        k = min(comp, _log_int(rng, 1, 2048))
        m = max(1, min(m, (1 << 20) // (b * (win + k)), (48 << 20) // (b * (win + k) * max(h, 16))))
        c = _attn("", b, m, h, win, comp, k, rng.choice((0.0, 0.02, 0.3)), _log_int(rng, 4, 256),
                  rng.choice((0, 8 * rng.randint(1, 64), 64)), False)
    del c["name"]
    return c


# ---- what a program has in hand -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 1009 + 17)
    return g


def _randint(g, lo, hi, shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device=_DEV, dtype=dtype)


def _bf16(g, shape):
    return torch.randn(shape, generator=g, device=_DEV).to(torch.bfloat16)


def _table(positions, rd):
    """(cos, sin) of position * 10000^(-2j/rd), in 64 bits, kept in 32."""
    freq = 10000.0 ** (-torch.arange(0, rd, 2, device=_DEV, dtype=torch.float64) / rd)
    ang = torch.arange(positions, device=_DEV, dtype=torch.float64)[:, None] * freq[None, :]
    return torch.stack((ang.cos(), ang.sin()), dim=-1).float().contiguous()


def _pages(g, b, rows, page):
    """A pool that holds every sequence's rows, its pages in random order."""
    per_seq = -(-rows // page)
    order = torch.randperm(b * per_seq, generator=g, device=_DEV)
    return b * per_seq, order.view(b, per_seq).to(torch.int32).contiguous()


def _filled_cache(g, pages, page, d):
    """A cache of quantised N(0, 1) rows."""
    codes = torch.empty((pages, page, d // 2), dtype=torch.uint8, device=_DEV)
    exps = torch.empty((pages, page, d // 32), dtype=torch.int8, device=_DEV)
    step = max(1, (1 << 19) // page)
    for p in range(0, pages, step):
        n = min(pages, p + step) - p
        c, k = _quantise(torch.randn((n, page, d), generator=g, device=_DEV))
        codes[p:p + n] = c
        exps[p:p + n] = k
    return codes, exps


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "norm_rotary":
        b, t, h, d = c["b"], c["s"], c["h"], c["d"]
        wide = _bf16(g, (b, t, h * d + c["gap"])) * 3.0
        s["x"] = wide[..., :h * d].unflatten(-1, (h, d))
        s["weight"] = 1.0 + 0.1 * torch.randn((d,), generator=g, device=_DEV) if c["weight"] else None
        s["eps"] = 1e-6
        s["first"] = _randint(g, 0, 16384, (b,))
        s["lens"] = _randint(g, 0, t + 1, (b,)) if c["ragged"] else None
        s["table"] = _table(16384 + t, c["rd"])
        s["y"] = torch.zeros((b, t, h, d), dtype=torch.bfloat16, device=_DEV)
    elif c["op"] == "append":
        b, t, d = c["b"], c["s"], c["d"]
        s["x"] = _bf16(g, (b, t, d)) * 2.0
        s["weight"] = 1.0 + 0.1 * torch.randn((d,), generator=g, device=_DEV) if c["norm"] else None
        s["eps"] = 1e-6 if c["norm"] else 0.0
        top = 4096 if c["window"] else 1024
        s["first"] = _randint(g, 0, top, (b,))
        s["lens"] = _randint(g, 0, t + 1, (b,)) if c["ragged"] else None
        s["table"] = _table((top + t) * c["step"], c["rd"])
        rows = c["base"] + (c["window"] if c["window"] else top + t)
        pages, s["block_table"] = _pages(g, b, rows, c["page"])
        s["codes"] = torch.zeros((pages, c["page"], d // 2), dtype=torch.uint8, device=_DEV)
        s["exps"] = torch.zeros((pages, c["page"], d // 32), dtype=torch.int8, device=_DEV)
        s["y"] = torch.zeros((b, t, d), dtype=torch.bfloat16, device=_DEV)
    else:
        b, m, h, d = c["b"], c["m"], c["h"], c["d"]
        pages, s["block_table"] = _pages(g, b, c["win"] + c["comp"], c["page"])
        s["codes"], s["exps"] = _filled_cache(g, pages, c["page"], d)
        s["q"] = _bf16(g, (b, m, h, d))
        s["sink"] = torch.randn((h,), generator=g, device=_DEV)
        s["scale"] = d ** -0.5
        s["idx"] = _index_rows(c, g)
        s["first"] = _randint(g, 0, 16384, (b,))
        s["table"] = _table(16384 + m, c["rd"]) if c["rd"] else None
        s["o"] = torch.empty((b, m, h, d), dtype=torch.bfloat16, device=_DEV)
    return s


def _index_rows(c, g):
    """Window columns, then sorted compressed rows shifted behind the window's, -1 where there is none."""
    n, k = c["b"] * c["m"], c["topk_comp"]
    if c["causal"]:
        q = torch.arange(n, device=_DEV)[:, None]
        w = min(c["win"], 128)
        win = (q - w + 1).clamp(min=0) + torch.arange(w, device=_DEV)[None, :]
        win = torch.where(win <= q, win, -1)
        seen = torch.arange(c["comp"], device=_DEV)[None, :] < q // 4
    else:
        win = torch.arange(c["win"], device=_DEV)[None, :].expand(n, -1)
        seen = None
    cols = [win.to(torch.int32)]
    if k:
        keys = torch.rand((n, c["comp"]), generator=g, device=_DEV)
        if seen is not None:
            keys = torch.where(seen, keys, -1.0)
        val, at = keys.topk(k, dim=-1)
        at = torch.where(val >= 0, at, 1 << 30).sort(dim=-1).values
        at = torch.where(at < (1 << 30), at + c["win"], -1)
        none = int(round(c["neg"] * k))
        if none:
            at.scatter_(1, torch.rand((n, k), generator=g, device=_DEV).topk(none, dim=-1).indices, -1)
        cols.append(at.to(torch.int32))
    return torch.cat(cols, dim=-1).view(c["b"], c["m"], -1).contiguous()


# ---- the plain forms -------------------------------------------------------------------------------

def _rotated(z, cs, inverse=False):
    """The last pairs of z turned by (cos, sin): cs [..., rd / 2, 2] of z's type."""
    rd = 2 * cs.shape[-2]
    a, b = z[..., -rd::2], z[..., -rd + 1::2]
    co, si = cs[..., 0], -cs[..., 1] if inverse else cs[..., 1]
    out = z.clone()
    out[..., -rd::2] = a * co - b * si
    out[..., -rd + 1::2] = a * si + b * co
    return out


def _normed(x, weight, eps):
    z = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + eps)
    return z if weight is None else z * weight.to(z.dtype)


def _quantise(z):
    """Packed e2m1 codes and block exponents of rows z [..., d]: ties to the even code."""
    v = z.unflatten(-1, (-1, 32))
    frac, k = torch.frexp(v.abs().amax(dim=-1).clamp(min=1e-4) / 6.0)
    k = k - (frac == 0.5).to(k.dtype)
    v = torch.ldexp(v, -k[..., None])
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + torch.signbit(v) * 8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), k.to(torch.int8)


def _values(codes, exps):
    """The 32-bit values that packed codes [..., d / 2] and exponents [..., d / 32] stand for."""
    one = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=codes.device)
    at = torch.arange(256, device=codes.device)
    pair = torch.stack((one[at % 16], one[at // 16]), dim=-1)
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * torch.exp2(exps.float())[..., None]).flatten(-2)


def _physical(block_table, rows, page):
    """Slots of logical rows [b, n] (negative ones give slot 0 of the table)."""
    r = rows.clamp(min=0).long()
    return torch.gather(block_table.long(), 1, r // page) * page + r % page


def _plain_norm(s):
    x = s["x"]
    t = torch.arange(x.shape[1], device=x.device)
    pos = s["first"].long()[:, None] + t
    y = _rotated(_normed(x.float(), s["weight"], s["eps"]), s["table"][pos][:, :, None]).to(torch.bfloat16)
    if s["lens"] is not None:
        y = torch.where((t < s["lens"][:, None])[:, :, None, None], y, s["y"])
    return y


def _plain_append(s):
    """In 64 bits: a code next to a border between two values is a decision."""
    c, x = s["case"], s["x"].double()
    t = torch.arange(x.shape[1], device=x.device)
    i = s["first"].long()[:, None] + t
    z = _normed(x, s["weight"], s["eps"]) if s["eps"] > 0 else x
    z = _rotated(z, s["table"][i * c["step"]].double())
    codes, exps = _quantise(z)
    lens = torch.full_like(s["first"], x.shape[1]) if s["lens"] is None else s["lens"]
    live = t < lens[:, None]
    kept = live & (t >= lens[:, None] - c["window"]) if c["window"] else live
    rows = c["base"] + (i % c["window"] if c["window"] else i)
    slot = _physical(s["block_table"], torch.where(kept, rows, 0), c["page"])[kept]
    s["codes"].view(-1, codes.shape[-1])[slot] = codes[kept]
    s["exps"].view(-1, exps.shape[-1])[slot] = exps[kept]
    y = torch.where(live[..., None], _values(codes, exps).to(torch.bfloat16), s["y"])
    return {"y": y, "codes": s["codes"], "exps": s["exps"]}


def _plain_attention(s):
    c, idx = s["case"], s["idx"]
    b, m, h, d = s["q"].shape
    slot = _physical(s["block_table"], idx.flatten(1), c["page"]).view(b * m, -1)
    kv = _values(s["codes"].view(-1, d // 2)[slot], s["exps"].view(-1, d // 32)[slot])
    q = s["q"].float().view(b * m, h, d)
    score = torch.matmul(q, kv.transpose(1, 2)) * s["scale"]
    live = (idx >= 0).view(b * m, 1, -1)
    score = score.masked_fill(~live, -math.inf)
    top = torch.maximum(score.amax(dim=-1, keepdim=True), s["sink"][:, None])
    p = torch.exp(score - top)
    o = torch.matmul(p, kv) / (p.sum(dim=-1, keepdim=True) + torch.exp(s["sink"][:, None] - top))
    o = o.view(b, m, h, d)
    if s["table"] is not None:
        pos = s["first"].long()[:, None] + torch.arange(m, device=idx.device)
        o = _rotated(o, s["table"][pos][:, :, None], inverse=True)
    return o.to(torch.bfloat16)


# ---- one pass --------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "norm_rotary":
            return _plain_norm(s)
        return _plain_append(s) if c["op"] == "append" else _plain_attention(s)
    from sparse_latent_attention_attn_gb300 import dsattn
    if c["op"] == "norm_rotary":
        return dsattn.norm_rotary(s["x"], s["eps"], c["rd"], s["table"], s["first"], weight=s["weight"],
                                  lens=s["lens"], y=s["y"])
    if c["op"] == "append":
        dsattn.kv_append_fp4_paged(s["x"], s["codes"], s["exps"], s["block_table"], s["first"], rd=c["rd"],
                                   table=s["table"], eps=s["eps"], weight=s["weight"], lens=s["lens"],
                                   pos_step=c["step"], base=c["base"], window=c["window"], y=s["y"])
        return {"y": s["y"], "codes": s["codes"], "exps": s["exps"]}
    return dsattn.sparse_attn_fp4_paged(s["q"], s["codes"], s["exps"], s["block_table"], s["sink"], s["idx"],
                                        s["scale"], rd=c["rd"], table=s["table"], first=s["first"], o=s["o"])


# ---- what a pass cannot do without -----------------------------------------------------------------

def _listed_rows(c):
    """Valid entries of all index rows."""
    n = c["b"] * c["m"]
    if c["causal"]:
        w = min(c["win"], 128)
        return sum(min(q + 1, w) + min(q // 4, c["comp"], c["topk_comp"]) for q in range(n))
    return n * (c["win"] + c["topk_comp"] - int(round(c["neg"] * c["topk_comp"])))


def work(case):
    c = case
    part = 0.5 if c.get("ragged") else 1.0
    if c["op"] == "norm_rotary":
        v = c["b"] * c["s"] * c["h"] * c["d"] * part
        return {"bytes": 4 * v + c["b"] * c["s"] * part * c["rd"] * 4, "flops": 5 * v}
    if c["op"] == "append":
        v = c["b"] * c["s"] * c["d"] * part
        kept = min(1.0, c["window"] / max(1, c["s"] * part)) if c["window"] else 1.0
        return {"bytes": v * (2 + 2 + kept * 17 / 32) + c["b"] * c["s"] * part * c["rd"] * 4, "flops": 8 * v}
    n, rows = c["b"] * c["m"], _listed_rows(c)
    held = min(rows, c["b"] * (c["win"] + c["comp"]))
    return {"bytes": held * c["d"] * 17 / 32 + 4 * n * c["h"] * c["d"] + 4 * n * (c["win"] + c["topk_comp"] if not c["causal"] else 128 + c["topk_comp"]),
            "flops": 4.0 * rows * c["h"] * c["d"]}


# ---- the definition, in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm_rotary":
        x = s["x"].double()
        z = x / (x.square().sum(-1, keepdim=True) / c["d"] + s["eps"]).sqrt()
        if s["weight"] is not None:
            z = z * s["weight"].double()
        turn = torch.view_as_complex(s["table"].double())
        at = torch.stack([turn[int(f):int(f) + c["s"]] for f in s["first"]])[:, :, None]
        tail = torch.view_as_complex(z[..., c["d"] - c["rd"]:].unflatten(-1, (-1, 2)).contiguous()) * at
        z[..., c["d"] - c["rd"]:] = torch.view_as_real(tail).flatten(-2)
        if s["lens"] is not None:
            for i, n in enumerate(s["lens"].tolist()):
                z[i, n:] = 0
        return z
    if c["op"] == "append":
        x, d = s["x"].double(), c["d"]
        if c["norm"]:
            x = x / (x.square().sum(-1, keepdim=True) / d + s["eps"]).sqrt() * s["weight"].double()
        turn = torch.view_as_complex(s["table"].double())
        at = torch.stack([turn[int(f) * c["step"]:][:c["s"] * c["step"]:c["step"]] for f in s["first"]])
        tail = torch.view_as_complex(x[..., d - c["rd"]:].unflatten(-1, (-1, 2)).contiguous()) * at
        x[..., d - c["rd"]:] = torch.view_as_real(tail).flatten(-2)
        blocks = x.unflatten(-1, (-1, 32))
        scale = torch.exp2(torch.ceil(torch.log2(blocks.abs().amax(-1, keepdim=True).clamp(min=1e-4) / 6)))
        grid = torch.tensor(_E2M1, dtype=torch.float64, device=_DEV)
        mids = (grid[1:] + grid[:-1]) / 2
        near = torch.bucketize(blocks.abs() / scale, mids)      # a tie goes to the lower of two codes
        tie = (near < 7) & (blocks.abs() / scale == mids[near.clamp(max=6)])
        near = near + (tie & (near % 2 == 1))                   # ... unless the upper one is even
        y = (grid[near] * scale * blocks.sign()).flatten(-2)
        if s["lens"] is not None:
            for i, n in enumerate(s["lens"].tolist()):
                y[i, n:] = 0
        return {"y": y, "codes": None, "exps": None}
    return _exact_attention(s, c)


def _exact_attention(s, c):
    b, m, h, d = s["q"].shape
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=_DEV)
    out = torch.zeros((b, m, h, d), dtype=torch.float64, device=_DEV)
    step = max(1, (1 << 19) // s["idx"].shape[2])
    for i in range(b):
        for t in range(0, m, step):
            idx = s["idx"][i, t:t + step].long()
            page = s["block_table"][i].long()[idx.clamp(min=0) // c["page"]]
            raw = s["codes"][page, idx.clamp(min=0) % c["page"]]
            code = torch.stack((raw & 15, raw >> 4), dim=-1).flatten(-2).long()
            row = grid[code & 7] * (1 - 2 * (code >> 3))
            row = row * torch.exp2(s["exps"][page, idx.clamp(min=0) % c["page"]].double()).repeat_interleave(32, dim=-1)
            logit = torch.einsum("qhd,qkd->qhk", s["q"][i, t:t + step].double(), row) * s["scale"]
            logit[(idx < 0)[:, None].expand_as(logit)] = -math.inf
            sink = s["sink"].double()[None, :, None].expand(logit.shape[0], h, 1)
            share = torch.softmax(torch.cat((logit, sink), dim=-1), dim=-1)[..., :-1]
            o = torch.einsum("qhk,qkd->qhd", share, row)
            if c["rd"]:
                at = torch.view_as_complex(s["table"].double())[int(s["first"][i]) + t:][:o.shape[0], None].conj()
                tail = torch.view_as_complex(o[..., d - c["rd"]:].unflatten(-1, (-1, 2)).contiguous()) * at
                o[..., d - c["rd"]:] = torch.view_as_real(tail).flatten(-2)
            out[i, t:t + step] = o
    return out
