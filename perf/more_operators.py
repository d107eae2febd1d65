"""Cases and plain forms of the paged 8-bit serving step: latent rows appended to a paged cache as e4m3 codes, rows of
a paged cache read back, and the attention of a chunk of new tokens over that cache.

A row of the cache is d values: d e4m3 codes and one power-of-two exponent for each 32 of them (the 4-bit cache: e2m1
codes, two to a byte).  A sequence's logical row r lives in slot r % page of page block_table[seq][r // page].

The attention lists no rows.  The query at position p sees the window's rows, positions p - window + 1 .. p (all
positions up to p for window 0; position i is logical row i % ring, or i without a ring), and the (p + 1) // ratio
compressed rows that stand for whole groups of `ratio` positions (from logical row `base` on; none for ratio 0).
"""
import math

import torch

own = False

if torch.cuda.is_available():
    _DEV = torch.device("cuda")
else:
    _DEV = torch.device("cpu")

_D = 512                                   # width of an attended row
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ---------------------------------------------------------------------------------------

def _append(name, b, s, d, rd, page, window, base, step, norm, ragged):
    return {"name": name, "op": "append", "b": b, "s": s, "d": d, "rd": rd, "page": page, "window": window,
            "base": base, "step": step, "norm": norm, "ragged": ragged}


def _read(name, bits, b, n, d, page, listed, ragged):
    return {"name": name, "op": "read", "bits": bits, "b": b, "n": n, "d": d, "page": page, "listed": listed,
            "ragged": ragged}


def _attn(name, b, m, h, window, ring, ratio, ctx, page, rd, ragged):
    return {"name": name, "op": "attention", "b": b, "m": m, "h": h, "window": window, "ring": ring, "ratio": ratio,
            "ctx": ctx, "page": page, "rd": rd, "ragged": ragged}


def listed():
    return [
        # one decode step of 256 sequences: each new latent row into its ring of 128 slots (latency counts)
        _append("append ring decode 256", 256, 1, 512, 64, 64, 128, 0, 1, True, False),
        # a long prompt's compressed rows, one for each 4 positions, behind the ring's 128 rows
        _append("append prompt 8x4096", 8, 4096, 512, 64, 64, 0, 128, 4, True, False),
        # 16 sequences' rings and compressed rows, back as bf16 rows (a cache handed to another store)
        _read("read fp8 16x4224", 8, 16, 4224, 512, 64, False, False),
        # the listed rows of 64 decoding sequences out of the 4-bit cache, a padded batch
        _read("read fp4 listed 64x640", 4, 64, 640, 512, 64, True, True),
        # one decode step of 64 sequences in a layer without compressed rows: a full ring each
        _attn("attn decode window", 64, 1, 64, 128, 128, 0, 10000, 64, 64, False),
        # one decode step of 32 sequences at position 16383: the ring and all 4096 compressed rows
        _attn("attn decode comp", 32, 1, 64, 128, 128, 4, 16383, 64, 64, False),
        # one decode step of 256 sequences of about 8192 tokens, 128 heads
        _attn("attn decode large", 256, 1, 128, 128, 128, 4, 8191, 64, 64, True),
        # a prompt's first 4096 tokens as one chunk: causal windows and up to 1024 compressed rows
        _attn("attn prefill 4096", 1, 4096, 64, 128, 0, 4, 0, 64, 64, False),
        # four prompts' next chunks of 512 tokens behind some 7680, 128 heads, a padded batch
        _attn("attn chunk 4x512", 4, 512, 128, 128, 640, 4, 7680, 64, 64, True),
        # a layer that attends to every earlier position, a share of 16 heads, 2048 tokens behind 6144
        _attn("attn causal 2048", 1, 2048, 16, 0, 0, 0, 6144, 64, 64, False),
        # one sequence with a share of 16 heads over a long context: few queries, a long axis
        _attn("attn one seq 16 heads", 1, 1, 16, 128, 128, 4, 65535, 64, 64, False),
        # short speculative steps of a few sequences, odd sizes everywhere
        _attn("attn 5x3 ragged", 5, 3, 40, 57, 61, 3, 1001, 24, 40, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "read", "attention", "attention"))
    if op == "append":
        d = 32 * _log_int(rng, 2, 32)
        rd = 8 * rng.randint(1, max(1, d // 8))
        b = _log_int(rng, 1, 256)
        s = max(1, min(_log_int(rng, 1, 4096), (16 << 20) // (b * d)))
        window = rng.choice((0, _log_int(rng, 8, 512)))
        c = _append("", b, s, d, rd, _log_int(rng, 1, 256), window, rng.randint(0, 200), rng.choice((1, 1, 4)),
                    rng.random() < 0.7, rng.random() < 0.5)
    elif op == "read":
        d = 32 * _log_int(rng, 1, 32)
        b = _log_int(rng, 1, 128)
        n = max(1, min(_log_int(rng, 1, 8192), (34 << 20) // (b * d)))
        c = _read("", rng.choice((4, 8)), b, n, d, _log_int(rng, 1, 256), rng.random() < 0.5, rng.random() < 0.5)
    else:
        b = _log_int(rng, 1, 128)
        h = _log_int(rng, 1, 128)
        window = rng.choice((0, _log_int(rng, 1, 600)))
        ratio = rng.choice((0, 2, 4, 8)) if window else 0
        ctx = _log_int(rng, 1, 32768 if ratio else 8192) - 1
        kept = (window if window else ctx) + (ctx // ratio if ratio else 0) + 1
        most = min((1 << 28) // (b * h * kept), math.isqrt((1 << 28) // (b * h)), (1 << 21) // b)
        m = max(1, min(_log_int(rng, 1, 2048), most))
        ring = rng.choice((0, window + m - 1 + rng.randint(0, 70))) if window else 0
        b = max(1, min(b, (1 << 21) // ((ring or ctx + m) + (ctx + m) // (ratio or 1 << 30))))
        c = _attn("", b, m, h, window, ring, ratio, ctx, _log_int(rng, 4, 256), rng.choice((0, 8 * rng.randint(1, 64), 64)),
                  rng.random() < 0.5)
    del c["name"]
    return c


def _base(c):
    """Logical row of the first compressed row: behind the ring, or behind every position."""
    return c["ring"] or c["ctx"] + c["m"]


def _compressed(c):
    return (c["ctx"] + c["m"]) // c["ratio"] if c["ratio"] else 0


# ---- what a program has in hand -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed) * 1009 + 29)
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


def _filled_cache(g, pages, page, d, bits):
    """A cache of quantised N(0, 1) rows."""
    codes = torch.empty((pages, page, d * bits // 8), dtype=torch.uint8, device=_DEV)
    exps = torch.empty((pages, page, d // 32), dtype=torch.int8, device=_DEV)
    step = max(1, (1 << 18) // page)
    for p in range(0, pages, step):
        n = min(pages, p + step) - p
        c, k = (_quantise8 if bits == 8 else _quantise4)(torch.randn((n, page, d), generator=g, device=_DEV))
        codes[p:p + n] = c
        exps[p:p + n] = k
    return codes, exps


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "append":
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
        s["codes"] = torch.zeros((pages, c["page"], d), dtype=torch.uint8, device=_DEV)
        s["exps"] = torch.zeros((pages, c["page"], d // 32), dtype=torch.int8, device=_DEV)
        s["y"] = torch.zeros((b, t, d), dtype=torch.bfloat16, device=_DEV)
    elif c["op"] == "read":
        b, n, d = c["b"], c["n"], c["d"]
        held = 4 * n if c["listed"] else n + 64
        pages, s["block_table"] = _pages(g, b, held, c["page"])
        s["codes"], s["exps"] = _filled_cache(g, pages, c["page"], d, c["bits"])
        s["first"] = None if c["listed"] else _randint(g, 0, 65, (b,))
        s["idx"] = None
        if c["listed"]:                    # ascending rows, some of them none
            at = torch.rand((b, held), generator=g, device=_DEV).topk(n, dim=-1).indices.sort(dim=-1).values
            s["idx"] = torch.where(torch.rand((b, n), generator=g, device=_DEV) < 0.03, -1, at).to(torch.int32)
        s["lens"] = _randint(g, 0, n + 1, (b,)) if c["ragged"] else None
        s["y"] = torch.zeros((b, n, d), dtype=torch.bfloat16, device=_DEV)
    else:
        b, m, h = c["b"], c["m"], c["h"]
        pages, s["block_table"] = _pages(g, b, _base(c) + _compressed(c), c["page"])
        s["codes"], s["exps"] = _filled_cache(g, pages, c["page"], _D, 8)
        s["q"] = _bf16(g, (b, m, h, _D))
        s["sink"] = torch.randn((h,), generator=g, device=_DEV)
        s["scale"] = _D ** -0.5
        s["first"] = torch.full((b,), c["ctx"], dtype=torch.int32, device=_DEV)
        s["lens"] = None
        if c["ragged"]:                    # contexts of three quarters to all of ctx, and padded chunks
            s["first"] -= _randint(g, 0, c["ctx"] // 4 + 1, (b,))
            s["lens"] = _randint(g, (m + 1) // 2, m + 1, (b,))
        s["table"] = _table(c["ctx"] + m, c["rd"]) if c["rd"] else None
        s["o"] = torch.zeros((b, m, h, _D), dtype=torch.bfloat16, device=_DEV)
    return s


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


def _pow2(k):
    """2^k exactly, in 64 bits."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _scaled(z, largest):
    """Blocks of 32 of z over 2^k, and k: the smallest with amax <= largest * 2^k."""
    v = z.unflatten(-1, (-1, 32))
    frac, k = torch.frexp(v.abs().amax(dim=-1).clamp(min=1e-4) / largest)
    k = k - (frac == 0.5).to(k.dtype)
    return v * _pow2(-k[..., None]).to(v.dtype), k


def _quantise8(z):
    """e4m3 codes [..., d] and block exponents of rows z [..., d]: nearest, ties to the even code."""
    v, k = _scaled(z, 448.0)
    step = torch.frexp(v)[1].clamp(min=-5) - 4              # of the values next to v: 2^step
    v = torch.round(v * _pow2(-step).to(v.dtype)) * _pow2(step).to(v.dtype)
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2), k.to(torch.int8)


def _quantise4(z):
    """Packed e2m1 codes and block exponents of rows z [..., d]: ties to the even code."""
    v, k = _scaled(z, 6.0)
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + torch.signbit(v) * 8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), k.to(torch.int8)


def _values(codes, exps):
    """The 32-bit values that codes [..., d] or packed codes [..., d / 2] and exponents [..., d / 32] stand for."""
    if codes.shape[-1] == 32 * exps.shape[-1]:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        one = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=codes.device)
        at = torch.arange(256, device=codes.device)
        v = torch.stack((one[at % 16], one[at // 16]), dim=-1)[codes.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _pow2(exps)[..., None].float()).flatten(-2)


def _physical(block_table, rows, page):
    """Slots of logical rows [b, n] (negative ones give slot 0 of the table)."""
    r = rows.clamp(min=0).long()
    return torch.gather(block_table.long(), 1, r // page) * page + r % page


def _plain_append(s):
    """In 64 bits: a code next to a border between two values is a decision."""
    c, x = s["case"], s["x"].double()
    t = torch.arange(x.shape[1], device=x.device)
    i = s["first"].long()[:, None] + t
    z = _normed(x, s["weight"], s["eps"]) if s["eps"] > 0 else x
    z = _rotated(z, s["table"][i * c["step"]].double())
    codes, exps = _quantise8(z)
    lens = torch.full_like(s["first"], x.shape[1]) if s["lens"] is None else s["lens"]
    live = t < lens[:, None]
    kept = live & (t >= lens[:, None] - c["window"]) if c["window"] else live
    rows = c["base"] + (i % c["window"] if c["window"] else i)
    slot = _physical(s["block_table"], torch.where(kept, rows, 0), c["page"])[kept]
    s["codes"].view(-1, codes.shape[-1])[slot] = codes[kept]
    s["exps"].view(-1, exps.shape[-1])[slot] = exps[kept]
    s["y"].copy_(torch.where(live[..., None], _values(codes, exps).to(torch.bfloat16), s["y"]))


def _plain_read(s):
    c, y = s["case"], s["y"]
    t = torch.arange(c["n"], device=y.device)
    rows = s["idx"] if s["idx"] is not None else s["first"].long()[:, None] + t
    slot = _physical(s["block_table"], rows, c["page"])
    v = _values(s["codes"].flatten(0, 1)[slot], s["exps"].flatten(0, 1)[slot]).to(torch.bfloat16)
    v = torch.where(rows[..., None] >= 0, v, 0)
    return v if s["lens"] is None else torch.where((t < s["lens"][:, None])[..., None], v, y)


def _plain_attention(s):
    c = s["case"]
    b, m, h, d = s["q"].shape
    first = s["first"].long()[:, None]
    pos = first + torch.arange(m, device=_DEV)                       # [b, m]
    if c["window"]:
        i = first + torch.arange(1 - c["window"], m, device=_DEV)    # [b, positions that some query sees]
    else:
        i = torch.arange(c["ctx"] + m, device=_DEV).expand(b, -1)
    live = (i[:, None] <= pos[..., None]) & (i[:, None] >= 0)
    if c["window"]:
        live &= i[:, None] > pos[..., None] - c["window"]
    rows = torch.where(i < 0, 0, i % c["ring"] if c["ring"] else i)
    if c["ratio"]:
        j = torch.arange(_compressed(c), device=_DEV)
        seen = j < ((pos + 1) // c["ratio"])[..., None]
        rows, live = torch.cat((rows, (_base(c) + j).expand(b, -1)), dim=-1), torch.cat((live, seen), dim=-1)
    slot = _physical(s["block_table"], torch.where(live.any(dim=1), rows, 0), c["page"])
    kv = _values(s["codes"].view(-1, d)[slot], s["exps"].view(-1, d // 32)[slot])
    score = torch.matmul(s["q"].float().view(b, m * h, d), kv.transpose(1, 2)).view(b, m, h, -1).mul_(s["scale"])
    score.masked_fill_(~live[:, :, None], -math.inf)
    top = torch.maximum(score.amax(dim=-1, keepdim=True), s["sink"][:, None])
    p = torch.exp(score.sub_(top))
    o = torch.matmul(p.view(b, m * h, -1), kv).view(b, m, h, d)
    o = o / (p.sum(dim=-1, keepdim=True) + torch.exp(s["sink"][:, None] - top))
    if s["table"] is not None:
        o = _rotated(o, s["table"][pos][:, :, None], inverse=True)
    o = o.to(torch.bfloat16)
    if s["lens"] is None:
        return o
    return torch.where((torch.arange(m, device=_DEV) < s["lens"][:, None])[..., None, None], o, s["o"])


# ---- one pass --------------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        from sparse_latent_attention_attn_gb300 import dsattn
        if c["op"] == "append":
            dsattn.kv_append_fp8_paged(s["x"], s["codes"], s["exps"], s["block_table"], s["first"], rd=c["rd"],
                                       table=s["table"], eps=s["eps"], weight=s["weight"], lens=s["lens"],
                                       pos_step=c["step"], base=c["base"], window=c["window"], y=s["y"])
        elif c["op"] == "read":
            read = dsattn.kv_read_fp8_paged if c["bits"] == 8 else dsattn.kv_read_fp4_paged
            return read(s["codes"], s["exps"], s["block_table"], c["n"], first=s["first"], idx=s["idx"], lens=s["lens"],
                        y=s["y"])
        else:
            return dsattn.chunk_attn_fp8_paged(s["q"], s["codes"], s["exps"], s["block_table"], s["first"], s["sink"],
                                               s["scale"], c["window"], ring=c["ring"], ratio=c["ratio"], base=_base(c),
                                               lens=s["lens"], rd=c["rd"], table=s["table"], o=s["o"])
    elif c["op"] == "append":
        _plain_append(s)
    else:
        return _plain_read(s) if c["op"] == "read" else _plain_attention(s)
    return {"y": s["y"], "codes": s["codes"].view(torch.float8_e4m3fn), "exps": s["exps"]}


# ---- what a pass cannot do without -----------------------------------------------------------------

def _tokens(c):
    """Of a sequence, expected."""
    return 0.5 * ((c["m"] + 1) // 2 + c["m"]) if c["ragged"] else c["m"]


def _seen(c):
    """(rows that all queries see, counted for each; rows that some query of a sequence sees), expected values."""
    m = _tokens(c)
    p0 = c["ctx"] * (0.875 if c["ragged"] else 1.0)
    w = c["window"] or 1 << 40
    n = max(1, int(round(m)))
    each = sum(min(p0 + t + 1, w) + ((p0 + t + 1) // c["ratio"] if c["ratio"] else 0) for t in range(n))
    some = min(p0 + m, w + m - 1) + ((p0 + m) // c["ratio"] if c["ratio"] else 0)
    return c["b"] * each, c["b"] * some


def work(case):
    c = case
    part = 0.5 if c["ragged"] else 1.0
    if c["op"] == "append":
        v = c["b"] * c["s"] * c["d"] * part
        kept = min(1.0, c["window"] / max(1, c["s"] * part)) if c["window"] else 1.0
        return {"bytes": v * (2 + 2 + kept * 33 / 32) + c["b"] * c["s"] * part * c["rd"] * 4, "flops": 8 * v}
    if c["op"] == "read":
        v = c["b"] * c["n"] * c["d"] * part
        return {"bytes": v * (2 + c["bits"] / 8 + 1 / 32), "flops": v}
    each, some = _seen(c)
    return {"bytes": some * _D * 33 / 32 + 4 * c["b"] * _tokens(c) * c["h"] * _D,
            "flops": 4.0 * each * c["h"] * _D}


# ---- the definition, in 64 bits --------------------------------------------------------------------

def _turned(z, table, rd, at, back=False):
    """Rows z [n, ..., d] with their last rd values turned as complex numbers by table rows `at` [n]."""
    if not rd:
        return z
    turn = torch.view_as_complex(table.double())[at]
    turn = (turn.conj() if back else turn).reshape(turn.shape[0], *([1] * (z.dim() - 2)), rd // 2)
    tail = torch.view_as_complex(z[..., z.shape[-1] - rd:].unflatten(-1, (-1, 2)).contiguous()) * turn
    return torch.cat((z[..., :z.shape[-1] - rd], torch.view_as_real(tail).flatten(-2)), dim=-1)


def _decoded(s, seq, rows, bits):
    """Logical rows of one sequence in 64 bits, from the codes' bit fields."""
    page = s["codes"].shape[1]
    where = (s["block_table"][seq].long()[rows // page], rows % page)
    raw, k = s["codes"][where].long(), s["exps"][where].long()
    if bits == 4:
        raw = torch.stack((raw & 15, raw >> 4), dim=-1).flatten(-2)
        man, exp, bias, low = raw & 1, (raw >> 1) & 3, 1, 1
    else:
        man, exp, bias, low = raw & 7, (raw >> 3) & 15, 7, 3
    full = (exp > 0).double()
    v = (full + man.double() / (1 << low)) * ((exp.clamp(min=1) - bias + 1023) << 52).view(torch.float64)
    v = torch.where((raw >> (bits - 1)) & 1 == 1, -v, v)
    return v * ((k + 1023) << 52).view(torch.float64).repeat_interleave(32, dim=-1)


def _grid8():
    """The e4m3 values from zero to 448, in order of their codes."""
    code = torch.arange(127, device=_DEV, dtype=torch.float64)
    exp = torch.floor(code / 8).clamp(min=1)
    return (code - 8 * exp + 8) / 8 * ((exp.long() + 1016) << 52).view(torch.float64)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "append":
        x, d = s["x"].double(), c["d"]
        if c["norm"]:
            x = x / (x.square().sum(-1, keepdim=True) / d + s["eps"]).sqrt() * s["weight"].double()
        grid = _grid8()
        mids = (grid[1:] + grid[:-1]) / 2
        for i in range(c["b"]):
            at = (int(s["first"][i]) + torch.arange(c["s"], device=_DEV)) * c["step"]
            z = _turned(x[i], s["table"], c["rd"], at).unflatten(-1, (-1, 32))
            amax = z.abs().amax(-1, keepdim=True).clamp(min=1e-4)
            scale = ((torch.floor(torch.log2(amax)).long() + 1013) << 52).view(torch.float64)
            for _ in range(4):                                       # the smallest power of two with amax <= 448 scale
                scale = torch.where(amax > 448 * scale, 2 * scale, scale)
            near = torch.bucketize(z.abs() / scale, mids)            # a tie goes to the lower of two codes
            tie = (near < 126) & (z.abs() / scale == mids[near.clamp(max=125)])
            near = near + (tie & (near % 2 == 1))                    # ... unless the upper one is even
            x[i] = (grid[near] * scale * z.sign()).flatten(-2)
            if s["lens"] is not None:
                x[i, int(s["lens"][i]):] = 0
        return {"y": x, "codes": None, "exps": None}
    if c["op"] == "read":
        y = torch.zeros((c["b"], c["n"], c["d"]), dtype=torch.float64, device=_DEV)
        for i in range(c["b"]):
            n = c["n"] if s["lens"] is None else int(s["lens"][i])
            rows = s["idx"][i, :n].long() if c["listed"] else int(s["first"][i]) + torch.arange(n, device=_DEV)
            there = rows >= 0
            y[i, :n][there] = _decoded(s, i, rows[there], c["bits"])
        return y
    return _exact_attention(s, c)


def _exact_attention(s, c):
    out = s["o"].double()
    for i in range(c["b"]):
        n, p0 = c["m"] if s["lens"] is None else int(s["lens"][i]), int(s["first"][i])
        step = max(1, (1 << 27) // (c["h"] * (p0 + n)))
        for t in range(0, n, step):
            p = p0 + torch.arange(t, min(n, t + step), device=_DEV)
            lo = max(0, p0 + t - c["window"] + 1) if c["window"] else 0
            near = torch.arange(lo, int(p[-1]) + 1, device=_DEV)
            mask = (near <= p[:, None]) & (near > p[:, None] - (c["window"] or 1 << 40))
            rows = near % c["ring"] if c["ring"] else near
            if c["ratio"]:
                far = torch.arange((int(p[-1]) + 1) // c["ratio"], device=_DEV)
                mask = torch.cat((mask, (far + 1) * c["ratio"] <= p[:, None] + 1), dim=1)
                rows = torch.cat((rows, _base(c) + far))
            kv = _decoded(s, i, rows, 8)
            logit = torch.einsum("qhd,kd->qhk", s["q"][i, t:t + step][:len(p)].double(), kv) * s["scale"]
            logit[~mask[:, None].expand_as(logit)] = -math.inf
            sink = s["sink"].double()[None, :, None].expand(len(p), c["h"], 1)
            share = torch.softmax(torch.cat((logit, sink), dim=-1), dim=-1)[..., :-1]
            o = torch.einsum("qhk,kd->qhd", share, kv)
            out[i, t:t + len(p)] = _turned(o, s["table"], c["rd"], p, back=True)
    return out
