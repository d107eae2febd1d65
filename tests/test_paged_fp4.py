"""The paged 4-bit row store: ds_norm_rotary, ds_kv_append_fp4_paged and ds_sparse_attn_fp4_paged against
plain implementations in 64 bits, their refusals, and a run of them together.

Tolerances.  A bf16 result is off by half a step, 2^-8 of its value; the f32 work before it by less than
2^-20 of the magnitudes it adds up.  A probability, scaled to P = 16 p 2^(e - E) (e the row's largest block
exponent, E the list's), enters the value product as hi - lo, hi in e4m3 and lo in e5m2.  From P >= 2^-6, hi
has four bits, so hi - P is at most 2^-4 of the power of two below P, and three bits of that leave 2^-8 of
P.  Below, hi is a multiple of 2^-9, so hi - P is at most 2^-10, and e5m2's half step of 2^-3 of it (down to
2^-17) leaves 2^-13: 2^-17 of p = 1 at e = E.  With A = sum p |v| / l and F = sum |v| 2^(E - e) / l (l the
denominator relative to the largest probability) an output is off by at most
2^-8 |o| + (2^-8 + 2^-12) A + 2^-17 F; a rotation adds up both values of a pair.  An output below f32's
least normal number, 2^-126, may come as 0 (a sink of 300 makes the exact ones about e^-300).
Codes, exponents and the values they stand for are equal.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---- plain implementations, 64 bits, on the CPU ---------------------------------------------------

def f64(t):
    return t.detach().cpu().double().numpy()


def table_of(positions, rd, scale=1.0):
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rd, 2) / max(rd, 1))[None]
    return torch.from_numpy(scale * np.stack((np.cos(ang), np.sin(ang)), -1)).float().contiguous()


def rotate(z, cs, inverse=False):
    rd = 2 * cs.shape[-2]
    if rd == 0:
        return z
    out = z.copy()
    a, b, c, s = z[..., -rd::2], z[..., -rd + 1::2], cs[..., 0], cs[..., 1] * (-1 if inverse else 1)
    out[..., -rd::2] = a * c - b * s
    out[..., -rd + 1::2] = a * s + b * c
    return out


def normed(x, weight, eps):
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return z if weight is None else z * weight


def quantise(z):
    """codes (0..15) and block exponents, decided value by value against the whole grid."""
    v = z.reshape(z.shape[:-1] + (-1, 32))
    amax = np.maximum(np.abs(v).max(-1), 1e-4)
    k = np.array([next(e for e in range(-20, 130) if a <= 6 * 2.0 ** e) for a in amax.ravel()]).reshape(amax.shape)
    y = np.abs(v) / 2.0 ** k[..., None]
    dist = np.abs(y[..., None] - MAG)
    lower = dist.argmin(-1)                                    # the lower of two that are as near
    upper = np.minimum(lower + 1, 7)
    tie = np.take_along_axis(dist, lower[..., None], -1) == np.take_along_axis(dist, upper[..., None], -1)
    near = np.where(tie[..., 0] & (lower < 7) & (lower % 2 == 1), upper, lower)
    code = near + 8 * np.signbit(v)
    return code.reshape(z.shape).astype(np.uint8), k.astype(np.int8)


def values(code, k):
    v = MAG[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(v.shape[:-1] + (-1, 32)) * 2.0 ** k[..., None].astype(float)).reshape(v.shape)


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[:-1] + (-1,))


def attention(q, rows, live, sink, scale, tops):
    """q [h][d], rows [n][d], live [n], tops [n] the rows' largest exponents -> o, A, F of the header comment."""
    rows, tops = rows[live], tops[live].astype(float)
    if not len(rows):
        return np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    s = scale * q @ rows.T
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    with np.errstate(over="ignore"):
        den = p.sum(-1, keepdims=True) + np.exp(sink[:, None] - top)
    worth = np.abs(rows) * 2.0 ** (tops.max() - tops)[:, None]
    return p @ rows / den, p @ np.abs(rows) / den, worth.sum(0)[None] / den


def pair_sum(a, rd):
    out = a.copy()
    if rd:
        both = a[..., -rd::2] + a[..., -rd + 1::2]
        out[..., -rd::2] = out[..., -rd + 1::2] = both
    return out


# ---- helpers on the GPU -----------------------------------------------------------------------------

@pytest.fixture(scope="module")
def ds():
    from sparse_latent_attention_attn_gb300 import dsattn
    dsattn.device_status()
    return dsattn


def dev(*ts):
    return [t if t is None else t.cuda() for t in ts]


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def random_pool(g, b, rows, page, d, kmin=-3, kmax=3, spare=2):
    """A pool with every sequence's pages in random order among `spare` unused ones."""
    per = -(-rows // page)
    pages = b * per + spare
    bt = torch.randperm(pages, generator=g)[: b * per].view(b, per).to(torch.int32)
    codes = torch.randint(0, 256, (pages, page, d // 2), generator=g, dtype=torch.uint8)
    exps = torch.randint(kmin, kmax + 1, (pages, page, d // 32), generator=g, dtype=torch.int8)
    return codes, exps, bt


def logical_rows(codes, exps, bt, seq, r, page):
    """64-bit rows of logical numbers r (clamped at 0) of one sequence, and their largest exponents."""
    r = np.maximum(r, 0)
    pg = bt.numpy()[seq][r // page]
    k = exps.numpy()[pg, r % page]
    return values(unpack(codes.numpy()[pg, r % page]), k), k.max(-1)


# ---- norm and rotation --------------------------------------------------------------------------------

NORMS = [  # b, s, h, d, rd, gap, weight, ragged
    (1, 1, 1, 8, 8, 0, False, False),
    (1, 1, 4, 64, 16, 0, False, False),
    (3, 5, 3, 40, 8, 24, True, True),
    (2, 3, 5, 128, 128, 8, True, False),
    (2, 7, 9, 192, 40, 64, False, True),
    (64, 1, 64, 512, 64, 0, False, False),
    (2, 33, 17, 512, 0, 0, True, True),
    (2, 3, 2, 1024, 1024, 0, True, False),
    (1, 2, 3, 520, 520, 0, False, False),
]


@gpu
@pytest.mark.parametrize("b,s,h,d,rd,gap,weight,ragged", NORMS)
def test_norm_rotary(ds, b, s, h, d, rd, gap, weight, ragged):
    g = torch.Generator().manual_seed(d + s)
    wide = (torch.randn((b, s, h * d + gap), generator=g) * 3).to(torch.bfloat16)
    w = torch.randn((d,), generator=g) if weight else None
    first = torch.randint(0, 100, (b,), generator=g, dtype=torch.int32)
    lens = torch.randint(0, s + 1, (b,), generator=g, dtype=torch.int32) if ragged else None
    tab = table_of(100 + s, rd, 1.25) if rd else None
    xg = wide.cuda()[..., : h * d].unflatten(-1, (h, d))
    y = torch.full((b, s, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    fg, wg, lg, tg = dev(first, w, lens, tab)
    out = ds.norm_rotary(xg, 1e-5, rd, tg, fg, weight=wg, lens=lg, y=y)
    assert ds.device_status() == 0 and out.data_ptr() == y.data_ptr()
    z = normed(f64(wide[..., : h * d].unflatten(-1, (h, d))), None if w is None else f64(w), 1e-5)
    mag = np.abs(z)
    if rd:
        cs = f64(tab)[first.numpy()[:, None] + np.arange(s)][:, :, None]
        mag = 1.25 * pair_sum(mag, rd)
        z = rotate(z, cs)
    live = np.ones((b, s), bool) if lens is None else np.arange(s) < lens.numpy()[:, None]
    got = f64(y)
    assert (got[~live] == 7).all()
    assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -20 * mag)[live].all()
    # a new output is zero where there is no token; in place gives the same as beside it
    if ragged:
        new = f64(ds.norm_rotary(xg, 1e-5, rd, tg, fg, weight=wg, lens=lg))
        assert (new[~live] == 0).all() and (new[live] == got[live]).all()
    if gap == 0:
        x2 = xg.clone()
        ds.norm_rotary(x2, 1e-5, rd, tg, fg, weight=wg, y=x2)
        assert (f64(x2)[live] == got[live]).all()


@gpu
def test_norm_rotary_positions_outside_the_table(ds):
    x = torch.ones((3, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    tab = table_of(10, 64).cuda()
    y = torch.full_like(x, 5.0)
    ds.norm_rotary(x, 1e-5, 64, tab, ints(0, 9, -1).cuda(), y=y)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    bad = (y == 5.0).all(-1).all(-1).cpu()
    assert bad.tolist() == [[False, False], [False, True], [True, False]]
    assert ds.norm_rotary(x[:0], 1e-5, 64, tab, ints().cuda()).shape == (0, 2, 2, 64)
    assert ds.norm_rotary(x[:, :0], 1e-5, 64, tab, ints(0, 0, 0).cuda()).shape == (3, 0, 2, 64)


@gpu
def test_norm_rotary_zero_and_extreme_rows(ds):
    x = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    x[0, 0, 1] = 1e-30
    x[0, 0, 2] = 1e15
    x[0, 0, 3, 5] = float("nan")
    y = f64(ds.norm_rotary(x.cuda(), 1e-6, 0, None, ints(0).cuda()))[0, 0]
    assert (y[0] == 0).all() and np.isfinite(y[:3]).all() and np.isnan(y[3]).all()
    np.testing.assert_allclose(y[2], 1.0, rtol=2.0 ** -8)


# ---- append ---------------------------------------------------------------------------------------------

APPENDS = [  # b, s, d, rd, page, window, base, step, eps, weight, ragged
    (1, 1, 32, 8, 1, 0, 0, 1, 1e-6, False, False),
    (3, 1, 64, 16, 4, 8, 0, 1, 1e-6, True, False),
    (2, 12, 64, 16, 3, 8, 2, 1, 1e-6, False, False),       # the chunk is longer than the ring
    (4, 9, 128, 64, 5, 0, 11, 4, 1e-6, True, True),
    (5, 7, 512, 64, 16, 128, 0, 1, 1e-6, True, True),
    (2, 40, 512, 64, 64, 16, 3, 1, 0.0, False, True),      # no norm
    (2, 6, 512, 0, 7, 0, 0, 1, 0.0, False, False),         # neither norm nor rotation: ties are real
    (2, 5, 224, 24, 9, 6, 1, 2, 1e-6, True, False),
    (1, 3, 1024, 1024, 2, 0, 0, 1, 1e-6, True, False),
    (64, 64, 512, 64, 24, 0, 5, 1, 1e-6, True, False),     # enough rows that some are near a border
]


def append_reference(x, w, eps, rd, tab, first, lens, step, base, window, codes, exps, bt, y):
    b, s, d = x.shape
    page = codes.shape[1]
    z = f64(x)
    if eps:
        z = normed(z, None if w is None else f64(w), np.float64(np.float32(eps)))
    i = first.numpy()[:, None].astype(np.int64) + np.arange(s)
    if rd:
        z = rotate(z, f64(tab)[i * step])
    code, k = quantise(z)
    codes, exps, y = codes.numpy().copy(), exps.numpy().copy(), f64(y)
    n = np.full(b, s) if lens is None else lens.numpy()
    for bi in range(b):
        for t in range(n[bi]):
            y[bi, t] = values(code[bi, t], k[bi, t])
            if window and t < n[bi] - window:
                continue
            r = base + (i[bi, t] % window if window else i[bi, t])
            pg = bt.numpy()[bi, r // page]
            codes[pg, r % page], exps[pg, r % page] = pack(code[bi, t]), k[bi, t]
    return codes, exps, y


@gpu
@pytest.mark.parametrize("b,s,d,rd,page,window,base,step,eps,weight,ragged", APPENDS)
def test_append(ds, b, s, d, rd, page, window, base, step, eps, weight, ragged):
    g = torch.Generator().manual_seed(d + s)
    wide = (torch.randn((b, s, d + 8), generator=g) * 2).to(torch.bfloat16)
    wide[0, 0, :32] = 0                                        # a block of zeros: the floor's scale
    x = wide[..., :d]
    w = torch.randn((d,), generator=g) if weight else None
    first = torch.randint(0, 50, (b,), generator=g, dtype=torch.int32)
    lens = torch.randint(0, s + 1, (b,), generator=g, dtype=torch.int32) if ragged else None
    tab = table_of((50 + s) * step, rd, 1.25) if rd else None
    codes, exps, bt = random_pool(g, b, base + (window or 50 + s), page, d)
    y = torch.full((b, s, d), 7.0, dtype=torch.bfloat16)
    want = append_reference(x, w, eps, rd, tab, first, lens, step, base, window, codes, exps, bt, y)
    cg, eg, btg, fg, wg, lg, tg, yg = dev(codes, exps, bt, first, w, lens, tab, y)
    args = dict(rd=rd, table=tg, eps=eps, weight=wg, lens=lg, pos_step=step, base=base, window=window)
    ds.kv_append_fp4_paged(wide.cuda()[..., :d], cg, eg, btg, fg, y=yg, **args)
    assert ds.device_status() == 0
    np.testing.assert_array_equal(eg.cpu().numpy(), want[1])
    np.testing.assert_array_equal(cg.cpu().numpy(), want[0])
    np.testing.assert_array_equal(f64(yg), want[2])
    # without y, and with y in place of x
    c2, e2 = dev(codes, exps)
    ds.kv_append_fp4_paged(wide.cuda()[..., :d], c2, e2, btg, fg, **args)
    assert torch.equal(c2, cg) and torch.equal(e2, eg)
    c3, e3, x3 = dev(codes, exps, x.contiguous())
    ds.kv_append_fp4_paged(x3, c3, e3, btg, fg, y=x3, **args)
    assert torch.equal(c3, cg) and torch.equal(e3, eg)
    live = np.ones((b, s), bool) if lens is None else np.arange(s) < lens.numpy()[:, None]
    assert (f64(x3)[live] == want[2][live]).all() and (f64(x3)[~live] == f64(x)[~live]).all()


@gpu
def test_append_ties_and_scales(ds):
    """Every border between two codes at every scale, exactly and one bf16 step to either side."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for k in (-15, -8, 0, 5, 60, 120):
        near = torch.from_numpy(borders * 2.0 ** k).to(torch.bfloat16).view(torch.int16)
        v = torch.cat([(near + j).view(torch.bfloat16) for j in (-1, 0, 1)])
        for top in (6.0, 4.0, 3.0):        # 3 * 2^k is the next smaller scale's largest value
            for edge in (-1, 0, 1):
                t = (torch.tensor([top * 2.0 ** k]).to(torch.bfloat16).view(torch.int16) + edge).view(torch.bfloat16)
                rows.append(torch.cat([t, v, -v])[:32])
    x = torch.stack([torch.nn.functional.pad(r, (0, 32 - len(r))) for r in rows])[None]
    n = x.shape[1]
    codes = torch.zeros((n, 1, 16), dtype=torch.uint8)
    exps = torch.zeros((n, 1, 1), dtype=torch.int8)
    bt = torch.arange(n, dtype=torch.int32)[None]
    y = torch.zeros_like(x)
    want = append_reference(x, None, 0.0, 0, None, ints(0), None, 1, 0, 0, codes, exps, bt, y)
    cg, eg, btg, fg, yg = dev(codes, exps, bt, ints(0), y)
    ds.kv_append_fp4_paged(x.cuda(), cg, eg, btg, fg, y=yg)
    np.testing.assert_array_equal(eg.cpu().numpy(), want[1])
    np.testing.assert_array_equal(cg.cpu().numpy(), want[0])
    np.testing.assert_array_equal(f64(yg), want[2])


@gpu
def test_append_bad_pages_and_positions(ds):
    x = torch.randn((6, 2, 64)).to(torch.bfloat16).cuda()
    codes = torch.full((4, 2, 32), 9, dtype=torch.uint8, device="cuda")
    exps = torch.full((4, 2, 2), 9, dtype=torch.int8, device="cuda")
    bt = torch.tensor([[0], [4], [-1], [1], [2], [3]], dtype=torch.int32, device="cuda")
    tab = table_of(100, 16).cuda()
    y = torch.full_like(x, 5.0)
    # sequence 3 starts past its only page, 4 at a negative row, 5 at the table's end
    ds.kv_append_fp4_paged(x, codes, exps, bt, ints(0, 0, 0, 2, -2, 99).cuda(), rd=16, table=tab, eps=1e-6, y=y)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    touched = [[bool((exps[p, r] != 9).any()) for r in range(2)] for p in range(4)]
    assert touched == [[True, True], [False, False], [False, False], [False, False]]
    assert (codes[1:] == 9).all()
    # the rows themselves are known wherever the position is: y is written, the page is what is missing
    assert [(y[i] != 5.0).any(-1).tolist() for i in range(6)] == [[True, True]] * 4 + [[False, False], [True, False]]


# ---- attention -------------------------------------------------------------------------------------------

ATTNS = [  # b, m, h, rows, topk, neg, page, rd
    (1, 1, 1, 1, 1, 0.0, 1, 0),
    (1, 1, 4, 7, 3, 0.0, 4, 16),
    (2, 1, 64, 128, 128, 0.0, 64, 64),
    (3, 2, 33, 500, 129, 0.3, 24, 64),
    (1, 1, 64, 300, 127, 0.0, 7, 0),
    (2, 3, 65, 400, 200, 0.1, 16, 64),
    (5, 1, 128, 700, 640, 0.05, 64, 64),
    (1, 1, 16, 9000, 2300, 0.02, 64, 512),
    (40, 4, 20, 300, 140, 0.5, 10, 8),
    (1, 2, 100, 3000, 1500, 0.9, 48, 64),
    (300, 1, 5, 40, 33, 0.2, 8, 64),
    (2, 1, 70, 20, 400, 0.0, 6, 64),        # the same row many times
]


def check_attention(ds, q, codes, exps, bt, sink, idx, rd=0, first=None, tab=None, scale=None, sample=None, **more):
    b, m, h, d = q.shape
    page = codes.shape[1]
    scale = d ** -0.5 if scale is None else scale
    qg, cg, eg, btg, sg, ig, fg, tg = dev(q, codes, exps, bt, sink, idx, first, tab)
    o = ds.sparse_attn_fp4_paged(qg, cg, eg, btg, sg, ig, scale, rd=rd, table=tg, first=fg, **more)
    assert ds.device_status() == 0
    got = f64(o)
    assert np.isfinite(got).all()
    toks = [(i, t) for i in range(b) for t in range(m)]
    if sample and len(toks) > sample:
        toks = [toks[j] for j in np.random.RandomState(3).choice(len(toks), sample, replace=False)]
    for i, t in toks:
        ix = idx[i, t].numpy()
        rows, tops = logical_rows(codes, exps, bt, i, ix, page)
        ref, A, F = attention(f64(q[i, t]), rows, ix >= 0, f64(sink), scale, tops)
        if rd:
            ref = rotate(ref, f64(tab)[int(first[i]) + t], inverse=True)
            A, F = pair_sum(A, rd), pair_sum(F, rd)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -17 * F + 2.0 ** -126
        bad = np.abs(got[i, t] - ref) > tol
        assert not bad.any(), (i, t, int(bad.sum()), float(np.abs(got[i, t] - ref)[bad].max()))
    return o


def attention_inputs(seed, b, m, h, rows, topk, neg, page, rd, d=512, qscale=1.0):
    g = torch.Generator().manual_seed(seed)
    codes, exps, bt = random_pool(g, b, rows, page, d)
    q = (torch.randn((b, m, h, d), generator=g) * qscale).to(torch.bfloat16)
    sink = torch.randn((h,), generator=g)
    if topk <= rows:
        idx = torch.stack([torch.randperm(rows, generator=g)[:topk] for _ in range(b * m)]).view(b, m, topk)
    else:
        idx = torch.randint(0, rows, (b, m, topk), generator=g)
    idx = torch.where(torch.rand((b, m, topk), generator=g) < neg, -1, idx).to(torch.int32)
    first = torch.randint(0, 64, (b,), generator=g, dtype=torch.int32) if rd else None
    tab = table_of(64 + m, rd) if rd else None
    return q, codes, exps, bt, sink, idx, rd, first, tab


@gpu
@pytest.mark.parametrize("b,m,h,rows,topk,neg,page,rd", ATTNS)
def test_attention(ds, b, m, h, rows, topk, neg, page, rd):
    x = attention_inputs(b + m + h, b, m, h, rows, topk, neg, page, rd)
    o = check_attention(ds, *x, sample=60)
    # the same call again, into given buffers, gives the same
    need = ds.sparse_attn_fp4_paged_workspace_bytes(b, m, h, 512, topk)
    ws = torch.randint(0, 256, (max(need, 16),), dtype=torch.uint8, device="cuda")
    again = check_attention(ds, *x, sample=1, o=torch.full_like(o, float("nan")), workspace=ws)
    assert torch.equal(again, o)


@gpu
def test_attention_rows_without_entries(ds):
    q, codes, exps, bt, sink, idx, rd, first, tab = attention_inputs(5, 4, 3, 40, 200, 150, 0.1, 16, 64)
    idx[0, 1] = -1
    idx[2] = -1
    idx[3, 2, 1:] = -7
    o = check_attention(ds, q, codes, exps, bt, sink, idx, rd, first, tab)
    assert (o[0, 1] == 0).all() and (o[2] == 0).all()
    # nothing at all to attend to
    idx[:] = -1
    assert (check_attention(ds, q, codes, exps, bt, sink, idx, rd, first, tab) == 0).all()
    none = ds.sparse_attn_fp4_paged(*dev(q, codes, exps, bt, sink, idx[..., :0].contiguous()), 0.1)
    assert (none == 0).all()
    assert ds.sparse_attn_fp4_paged(*dev(q[:0], codes, exps, bt[:0], sink, idx[:0]), 0.1).shape == (0, 3, 40, 512)


@gpu
@pytest.mark.parametrize("h", [3, 64, 128])
def test_attention_peaked_growing_and_flat(ds, h):
    """Scores whose maximum moves through the row, one row far above the rest, and equal scores."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(9, 2, 1, h, 1000, 900, 0.0, 32, 0)
    idx = idx.sort(-1).values
    for qs in (8.0, 40.0):
        check_attention(ds, (q.float() * qs).to(torch.bfloat16), codes, exps, bt, sink, idx)
    check_attention(ds, torch.zeros_like(q), codes, exps, bt, sink, idx)
    up = exps.clone()                                     # rows whose scale grows with their number
    for i in range(2):
        for r in range(1000):
            up[bt[i, r // 32], r % 32] = -6 + r // 100
    check_attention(ds, q, codes, up, bt, sink, idx)
    down = exps.clone()
    for i in range(2):
        for r in range(1000):
            down[bt[i, r // 32], r % 32] = 4 - r // 100
    check_attention(ds, q, codes, down, bt, sink, idx)
    # heads of very different size, and values within a head too
    check_attention(ds, (q * torch.logspace(-4, 1, h)[:, None]).to(torch.bfloat16), codes, exps, bt, sink, idx)
    check_attention(ds, (q * torch.logspace(-6, 0, 512)).to(torch.bfloat16), codes, exps, bt, sink, idx)


@gpu
def test_attention_sinks(ds):
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(11, 2, 2, 30, 300, 200, 0.1, 16, 0)
    check_attention(ds, q, codes, exps, bt, torch.full_like(sink, -math.inf), idx)
    check_attention(ds, q, codes, exps, bt, torch.full_like(sink, 30.0), idx)
    o = check_attention(ds, q, codes, exps, bt, torch.full_like(sink, 300.0), idx)
    assert (o.abs() < 1e-30).all()


@gpu
def test_attention_scale_spread_within_a_row(ds):
    """Blocks of one row 24 octaves apart, rows of zeros, and exponents far from 0."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(13, 2, 1, 24, 300, 200, 0.0, 16, 0)
    wide = exps.clone()
    wide[..., 1::2] = -24
    wide[..., 0::2] = 0
    check_attention(ds, q, codes, wide, bt, sink, idx)
    zero = codes.clone()
    zero[::2] = 0
    check_attention(ds, q, zero, exps, bt, sink, idx)
    zero[:] = 0x88                                         # minus zero
    assert (check_attention(ds, q, zero, exps, bt, sink, idx) == 0).all()
    for k in (-60, 40):
        check_attention(ds, (q.float() * 2.0 ** -k).to(torch.bfloat16), codes, (exps + k), bt, sink, idx)


@gpu
def test_attention_bad_entries(ds):
    q, codes, exps, bt, sink, idx, rd, first, tab = attention_inputs(15, 3, 1, 40, 200, 150, 0.1, 16, 64)
    o = check_attention(ds, q, codes, exps, bt, sink, idx, rd, first, tab)
    bad = torch.cat((idx, torch.full((3, 1, 3), 13 * 16, dtype=torch.int32)), -1)   # past the table's 13 pages
    bad[..., -1] = 2 ** 31 - 1
    args = dev(q, codes, exps, bt, sink)
    got = ds.sparse_attn_fp4_paged(*args, bad.cuda(), 512 ** -0.5, rd=rd, table=tab.cuda(), first=first.cuda())
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    assert (got.float() - o.float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
    hole = bt.clone()
    hole[1, :] = -1
    hole[2, :] = codes.shape[0]
    got = ds.sparse_attn_fp4_paged(args[0], args[1], args[2], hole.cuda(), sink.cuda(), idx.cuda(), 512 ** -0.5)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    assert (got[1:] == 0).all() and (got[0] != 0).any()
    # a position outside the table: that token is not rotated
    far = first.clone()
    far[1] = 1000
    got = ds.sparse_attn_fp4_paged(*args, idx.cuda(), 512 ** -0.5, rd=rd, table=tab.cuda(), first=far.cuda())
    plain = ds.sparse_attn_fp4_paged(*args, idx.cuda(), 512 ** -0.5)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    assert torch.equal(got[1], plain[1]) and torch.equal(got[0], o[0]) and torch.equal(got[2], o[2])


# ---- together ----------------------------------------------------------------------------------------------

@gpu
def test_step_together_and_in_a_graph(ds):
    """A prompt and decode steps of two sequences at positions of their own, through path.decode_step_fp4_paged;
    the last step captured, and replayed for the next position."""
    from sparse_latent_attention_attn_gb300 import path
    g = torch.Generator().manual_seed(3)
    b, h, d, rd, W, page, ratio = 2, 24, 512, 64, 16, 5, 4
    eps, scale = 1e-6, d ** -0.5
    rows = W + 20
    codes, exps, bt = random_pool(g, b, rows, page, d)
    codes.zero_(), exps.zero_()
    tab = table_of(128, rd)
    w = 1 + 0.1 * torch.randn((d,), generator=g)
    sink = torch.randn((h,), generator=g)
    comp = torch.randn((b, 9, d), generator=g).to(torch.bfloat16)
    cg, eg, btg, tg, wg, sg = dev(codes, exps, bt, tab, w, sink)
    ds.kv_append_fp4_paged(comp.cuda(), cg, eg, btg, ints(0, 0).cuda(), rd=rd, table=tg, eps=eps, weight=wg,
                           lens=ints(9, 4).cuda(), pos_step=ratio, base=W)
    ref_c, ref_e, _ = append_reference(comp, w, eps, rd, tab, ints(0, 0), ints(9, 4), ratio, W, 0, codes, exps, bt,
                                       torch.zeros_like(comp))
    ncomp = [9, 4]
    prompt = torch.randn((b, 20, d), generator=g).to(torch.bfloat16)
    n0 = ints(20, 7)
    ds.kv_append_fp4_paged(prompt.cuda(), cg, eg, btg, ints(0, 0).cuda(), rd=rd, table=tg, eps=eps, weight=wg,
                           lens=n0.cuda(), window=W)
    ref_c, ref_e, _ = append_reference(prompt, w, eps, rd, tab, ints(0, 0), n0, 1, 0, W, torch.from_numpy(ref_c),
                                       torch.from_numpy(ref_e), bt, torch.zeros_like(prompt))
    first = n0.clone()
    static = {"q": torch.zeros((b, 1, h, d), dtype=torch.bfloat16, device="cuda"),
              "kv": torch.zeros((b, 1, d), dtype=torch.bfloat16, device="cuda"),
              "first": torch.zeros((b,), dtype=torch.int32, device="cuda"),
              "idx": torch.full((b, 1, W + 10), -1, dtype=torch.int32, device="cuda")}

    def step():
        return path.decode_step_fp4_paged(static["q"], static["kv"], cg, eg, btg, static["first"], sg, static["idx"],
                                          W, scale, rd, tg, eps, kv_weight=wg)

    graph = out = None
    side = torch.cuda.Stream()
    for n in range(4):
        q = torch.randn((b, 1, h, d), generator=g).to(torch.bfloat16)
        kv = torch.randn((b, 1, d), generator=g).to(torch.bfloat16)
        idx = torch.full((b, 1, W + 10), -1, dtype=torch.int32)
        for i in range(b):
            idx[i, 0, :W] = torch.where(torch.arange(W) <= first[i], torch.arange(W), -1)
            idx[i, 0, W:W + ncomp[i]] = W + torch.arange(ncomp[i])
        for k, v in (("q", q), ("kv", kv), ("first", first), ("idx", idx)):
            static[k].copy_(v)
        torch.cuda.synchronize()
        if n < 2:
            with torch.cuda.stream(side):
                got = step()
            side.synchronize()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out = step()
            graph.replay()
            torch.cuda.synchronize()
            got = out
        ref_c, ref_e, _ = append_reference(kv, w, eps, rd, tab, first, None, 1, 0, W, torch.from_numpy(ref_c),
                                           torch.from_numpy(ref_e), bt, torch.zeros_like(kv))
        np.testing.assert_array_equal(cg.cpu().numpy(), ref_c)
        np.testing.assert_array_equal(eg.cpu().numpy(), ref_e)
        for i in range(b):
            zq = rotate(normed(f64(q[i, 0]), None, eps), f64(tab)[int(first[i])][None])
            zq = f64(torch.from_numpy(zq).to(torch.bfloat16))
            ix = idx[i, 0].numpy()
            rr, tops = logical_rows(torch.from_numpy(ref_c), torch.from_numpy(ref_e), bt, i, ix, page)
            ref, A, F = attention(zq, rr, ix >= 0, f64(sink), scale, tops)
            ref = rotate(ref, f64(tab)[int(first[i])][None], inverse=True)
            A, F = pair_sum(A, rd), pair_sum(F, rd)
            # beside the attention's own: q may be one bf16 step off where the norm's f32 falls on the other
            # side of a border; its effect is far below a step of all 512 products together
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * A + 2.0 ** -17 * F
            assert (np.abs(f64(got[i, 0]) - ref) <= tol).all()
        first += 1
    assert ds.device_status() == 0


# ---- the edges of what the documentation allows ---------------------------------------------------------------

@gpu
@pytest.mark.parametrize("b,s,h,d,rd", [(19, 33, 64, 512, 64), (31, 57, 89, 40, 16), (23, 45, 76, 128, 128),
                                        (3, 21000, 1, 512, 512)])
def test_norm_rotary_many_rows(ds, b, s, h, d, rd):
    """Batches long enough for several rows a warp (rows of one warp then belong to different tokens and
    sequences): against the formula, and the same as one sequence at a time."""
    g = torch.Generator().manual_seed(d)
    wide = torch.randn((b, s, h * d + 8), generator=g).to(torch.bfloat16)
    w = torch.randn((d,), generator=g)
    first = torch.randint(0, 100, (b,), generator=g, dtype=torch.int32)
    lens = torch.randint(0, s + 1, (b,), generator=g, dtype=torch.int32)
    lens[0], lens[-1] = s + 5, -3                          # more than there are: all of them; fewer than none: none
    tab = table_of(100 + s, rd)
    xg, fg, wg, lg, tg = dev(wide, first, w, lens, tab)
    xg = xg[..., : h * d].unflatten(-1, (h, d))
    y = torch.full((b, s, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ds.norm_rotary(xg, 1e-5, rd, tg, fg, weight=wg, lens=lg, y=y)
    one = torch.full_like(y, 7.0)
    step = max(1, 20000 // h)                              # short enough for one row a warp
    for i in range(b):
        for t in range(0, s, step):
            n = min(step, s - t)
            o = one[i, t:t + n][None].clone()
            ds.norm_rotary(xg[i:i + 1, t:t + n], 1e-5, rd, tg, fg[i:i + 1] + t, weight=wg, lens=lg[i:i + 1] - t, y=o)
            one[i, t:t + n] = o[0]
    assert ds.device_status() == 0
    assert torch.equal(y, one)
    assert (y[-1] == 7).all() and (y[0] != 7).any(-1).all()
    for i in np.random.RandomState(1).choice(b - 1, min(b - 1, 3), replace=False):
        n = min(max(int(lens[i]), 0), s, 2000)
        z = normed(f64(wide[i, :n, : h * d].unflatten(-1, (h, d))), f64(w), 1e-5)
        mag = pair_sum(np.abs(z), rd)
        z = rotate(z, f64(tab)[int(first[i]) + np.arange(n)][:, None])
        assert (np.abs(f64(y[i, :n]) - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -20 * mag).all()


@gpu
def test_append_signs_of_zero(ds):
    """Minus zero stays minus zero in its code, with and without norm and rotation by nothing."""
    x = torch.randn((1, 6, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0, :, ::3] = -0.0
    x[0, :, 1::3] = 0.0
    x[0, 5] = -0.0
    codes = torch.zeros((6, 1, 32), dtype=torch.uint8)
    exps = torch.zeros((6, 1, 2), dtype=torch.int8)
    bt = torch.arange(6, dtype=torch.int32)[None]
    for eps in (0.0, 1e-6):
        want = append_reference(x, None, eps, 0, None, ints(0), None, 1, 0, 0, codes, exps, bt, torch.zeros_like(x))
        cg, eg, btg, fg = dev(codes, exps, bt, ints(0))
        ds.kv_append_fp4_paged(x.cuda(), cg, eg, btg, fg, eps=eps)
        np.testing.assert_array_equal(eg.cpu().numpy(), want[1])
        np.testing.assert_array_equal(cg.cpu().numpy(), want[0])


@gpu
def test_append_lengths_and_last_positions(ds):
    """Lengths below none and above all, rows at the largest number, and the position after it."""
    x = torch.randn((4, 3, 32), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    codes = torch.full((4, 8, 16), 9, dtype=torch.uint8, device="cuda")
    exps = torch.full((4, 8, 1), 99, dtype=torch.int8, device="cuda")
    bt = torch.arange(4, dtype=torch.int32, device="cuda")[:, None].contiguous()
    last = 2 ** 31 - 1
    y = torch.full_like(x, 5.0).cuda()
    ds.kv_append_fp4_paged(x.cuda(), codes, exps, bt, ints(0, 0, last, last - 1).cuda(), window=8, y=y,
                           lens=ints(-1, 7, 1, 3).cuda())
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX       # sequence 3 has a third token
    want = [[], [0, 1, 2], [7], [6, 7]]
    for i in range(4):
        assert [r for r in range(8) if bool((exps[i, r] != 99).all())] == want[i]
    assert (y != 5.0).any(-1).cpu().tolist() == [[False] * 3, [True] * 3, [True, False, False], [True, True, False]]


@gpu
def test_store_without_pages(ds):
    """No pages at all, and a table without columns: every row is without a page."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(17, 2, 2, 70, 50, 30, 0.5, 16, 0)
    x = torch.randn((2, 3, 512)).to(torch.bfloat16).cuda()
    qg, cg, eg, btg, sg, ig = dev(q, codes, exps, bt, sink, idx)
    for c, e, t in ((cg[:0], eg[:0], btg), (cg, eg, btg[:, :0].contiguous()), (cg[:0], eg[:0], btg[:, :0].contiguous())):
        o = ds.sparse_attn_fp4_paged(qg, c, e, t, sg, ig, 0.1)
        assert ds.device_status() == ds.DS_DEV_BAD_INDEX and (o == 0).all()
        assert (ds.sparse_attn_fp4_paged(qg, c, e, t, sg, torch.full_like(ig, -1), 0.1) == 0).all()
        assert ds.device_status() == 0
        y = torch.zeros_like(x)
        ds.kv_append_fp4_paged(x, c, e, t, ints(0, 0).cuda(), y=y)
        assert ds.device_status() == ds.DS_DEV_BAD_INDEX and (y != 0).any(-1).all()
    assert torch.equal(cg.cpu(), codes) and torch.equal(eg.cpu(), exps)


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.05, 3e-5])
def test_attention_scales(ds, scale):
    q, codes, exps, bt, sink, idx, rd, first, tab = attention_inputs(19, 2, 2, 70, 300, 200, 0.1, 16, 64)
    check_attention(ds, q, codes, exps, bt, sink, idx, rd, first, tab, scale=scale)


@gpu
@pytest.mark.parametrize("topk", [1, 32, 127, 128, 129, 255, 256, 257, 512])
def test_attention_lengths_around_a_tile(ds, topk):
    """Rows that leave every count of a last tile, in units of a range of their own and in shared ones."""
    for b, m, h in ((1, 1, 64), (160, 1, 3), (2, 3, 128)):
        x = attention_inputs(topk + b, b, m, h, 600, topk, 0.0, 16, 64)
        check_attention(ds, *x, sample=12)


@gpu
def test_attention_and_append_in_a_large_pool(ds):
    """Pages whose codes lie more than 2^31 and 2^32 bytes into the pool."""
    page, d = 64, 512
    pages = 2 ** 32 // (page * d // 2) + 40                   # 4.3 GB of codes
    q, codes, exps, bt, sink, idx, rd, first, tab = attention_inputs(21, 2, 1, 64, 8 * page, 300, 0.1, page, 64)
    n = codes.shape[0]
    where = torch.tensor([0, 3, pages // 2 - 5, pages // 2 + 7] + list(range(pages - n + 4, pages)))
    big = torch.zeros((pages, page, d // 2), dtype=torch.uint8, device="cuda")
    bige = torch.zeros((pages, page, d // 32), dtype=torch.int8, device="cuda")
    for i, j in enumerate(where.tolist()):
        big[j], bige[j] = codes[i].cuda(), exps[i].cuda()
    far = where[bt.long()].to(torch.int32)
    o = check_attention(ds, q, codes, exps, bt, sink, idx, rd, first, tab)
    got = ds.sparse_attn_fp4_paged(*dev(q), big, bige, *dev(far, sink, idx), d ** -0.5, rd=rd, table=tab.cuda(),
                                   first=first.cuda())
    assert torch.equal(got, o)
    x = torch.randn((2, 70, d)).to(torch.bfloat16).cuda()
    small, smalle = dev(codes, exps)
    for c, e, t in ((small, smalle, bt), (big, bige, far)):
        ds.kv_append_fp4_paged(x, c, e, t.cuda(), ints(5, 400).cuda(), rd=0, eps=1e-6)
    assert ds.device_status() == 0
    for i, j in enumerate(where.tolist()):
        assert torch.equal(big[j], small[i]) and torch.equal(bige[j], smalle[i])


@gpu
def test_attention_calls_at_once_and_captured(ds):
    """Two calls at once on streams of their own, then two graphs replayed at once and over again, each with
    its workspace: the same as one after the other."""
    shapes = ((4, 1, 128, 700), (1, 1, 16, 2300))             # both cut units, and need a workspace
    x = [attention_inputs(23 + b, b, m, h, 3000, topk, 0.1, 64, 64) for b, m, h, topk in shapes]
    want = [check_attention(ds, *v, sample=2) for v in x]
    args = [dev(*v[:6]) + [512 ** -0.5] for v in x]
    more = [dict(rd=v[6], first=v[7].cuda(), table=v[8].cuda()) for v in x]
    for k, (b, m, h, topk) in enumerate(shapes):
        need = ds.sparse_attn_fp4_paged_workspace_bytes(b, m, h, 512, topk)
        assert need > 0
        more[k]["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        more[k]["o"] = torch.empty_like(want[k])
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, st in enumerate(streams):
            more[k]["o"].zero_()
        torch.cuda.synchronize()
        for k, st in enumerate(streams):
            ds.sparse_attn_fp4_paged(*args[k], **more[k], stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(more[k]["o"], want[k]) for k in range(2))
    # without a workspace given, and on a stream given by a context
    for k, st in enumerate(streams):
        own = {n: v for n, v in more[k].items() if n not in ("o", "workspace")}
        with torch.cuda.stream(st):
            a = ds.sparse_attn_fp4_paged(*args[k], **own)
        b = ds.sparse_attn_fp4_paged(*args[k], **own, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(a, want[k]) and torch.equal(b, want[k])
    graphs, outs = [], []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        own = {n: v for n, v in more[k].items() if n != ("o" if k else "workspace")}
        with torch.cuda.graph(graphs[k]):
            outs.append(ds.sparse_attn_fp4_paged(*args[k], **own))
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(outs[k], want[k]) for k in range(2))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
    assert ds.device_status() == 0


@gpu
def test_attention_workspace_refused(ds):
    b, m, h, topk = 4, 1, 64, 700
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(29, b, m, h, 1000, topk, 0.0, 64, 0)
    args = dev(q, codes, exps, bt, sink, idx)
    need = ds.sparse_attn_fp4_paged_workspace_bytes(b, m, h, 512, topk)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    o = torch.full_like(args[0], 3.0)
    for bad in (ws[:need - 1], ws[16:16 + need], ws[:0]):
        with pytest.raises(ds.DsError):
            ds.sparse_attn_fp4_paged(*args, 0.1, o=o, workspace=bad)
    assert ds.device_status() == 0 and (o == 3).all()


@gpu
@pytest.mark.parametrize("b,h,topk", [(4, 64, 700), (4, 128, 700), (1, 5, 1), (200, 64, 300)])
def test_attention_wait_that_runs_out(ds, b, h, topk):
    """With the hook on, the row warps withhold the first tile: the call ends, says so, and the next is clean."""
    x = attention_inputs(31 + b, b, 1, h, 2000, topk, 0.0, 64, 64)
    args, more = dev(*x[:6]) + [512 ** -0.5], dict(rd=x[6], first=x[7].cuda(), table=x[8].cuda())
    assert ds.device_status() == 0
    ds.test_set_stall(True)
    try:
        ds.sparse_attn_fp4_paged(*args, **more)
        bits = ds.device_status()
    finally:
        ds.test_set_stall(False)
    assert bits == ds.DS_DEV_TIMEOUT
    check_attention(ds, *x, sample=4)


@gpu
def test_bindings_refuse_what_does_not_fit(ds):
    """Each argument in turn with another type, shape, layout or place: refused before anything runs."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    i32, f32, u8, i8 = torch.int32, torch.float32, torch.uint8, torch.int8
    norm = dict(x=z(2, 3, 4, 64), eps=1e-6, rd=16, table=z(9, 8, 2, dt=f32), first=z(2, dt=i32), weight=z(64, dt=f32),
                lens=z(2, dt=i32), y=z(2, 3, 4, 64))
    app = dict(x=z(2, 3, 64), codes=z(5, 4, 32, dt=u8), exps=z(5, 4, 2, dt=i8), block_table=z(2, 3, dt=i32),
               first=z(2, dt=i32), rd=16, table=z(9, 8, 2, dt=f32), eps=1e-6, weight=z(64, dt=f32), lens=z(2, dt=i32),
               y=z(2, 3, 64))
    attn = dict(q=z(2, 1, 4, 512), codes=z(5, 4, 256, dt=u8), exps=z(5, 4, 16, dt=i8), block_table=z(2, 3, dt=i32),
                sink=z(4, dt=f32), idx=z(2, 1, 7, dt=i32), scale=0.1, rd=16, table=z(9, 8, 2, dt=f32), first=z(2, dt=i32),
                o=z(2, 1, 4, 512))
    for f, args in ((ds.norm_rotary, norm), (ds.kv_append_fp4_paged, app), (ds.sparse_attn_fp4_paged, attn)):
        f(**args)
        for name, t in args.items():
            if not isinstance(t, torch.Tensor):
                continue
            wide = torch.zeros(t.shape + (2,), dtype=t.dtype, device="cuda")[..., 0]
            bad = [t.to(torch.int64), t.cpu(), wide, t.unsqueeze(0)]
            if (f, name) not in ((ds.norm_rotary, "table"), (ds.kv_append_fp4_paged, "table"), (ds.sparse_attn_fp4_paged, "table"),
                                 (ds.kv_append_fp4_paged, "exps")):
                bad.append(torch.zeros(t.shape[:-1] + (t.shape[-1] + 1,), dtype=t.dtype, device="cuda"))
            for v in bad:
                if (name, f) in (("idx", ds.sparse_attn_fp4_paged), ("block_table", ds.kv_append_fp4_paged),
                                 ("block_table", ds.sparse_attn_fp4_paged)) and v.shape[:-1] == t.shape[:-1] \
                        and v.dtype == t.dtype and v.is_cuda and v.is_contiguous():
                    continue                               # another number of columns is another valid call
                with pytest.raises((TypeError, ValueError, RuntimeError)):
                    f(**{**args, name: v})
    assert ds.device_status() == 0


# ---- refusals, no GPU needed ---------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    from sparse_latent_attention_attn_gb300 import build
    build.build()
    from sparse_latent_attention_attn_gb300 import dsattn
    return dsattn._lib


FAKE = 4096   # never dereferenced: every call below fails its checks first


def call(fn, base, /, **change):
    args = {**base, **change}
    return fn(*args.values())


def test_norm_rotary_refusals(lib):
    base = dict(x=FAKE, xb=512, xt=512, y=FAKE, b=2, s=1, h=8, d=64, w=None, eps=1e-6, rd=16, table=FAKE, rows=10,
                first=FAKE, lens=None, stream=None)
    f = lib.ds_norm_rotary
    for bad in (dict(b=-1), dict(s=-1), dict(h=0), dict(d=0), dict(d=60), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(rd=12), dict(rd=-8), dict(rd=72), dict(table=None), dict(table=FAKE + 4),
                dict(rows=-1), dict(x=None), dict(x=FAKE + 8), dict(y=None), dict(y=FAKE + 2), dict(first=None),
                dict(first=FAKE + 2), dict(lens=FAKE + 1), dict(w=FAKE + 2), dict(xb=511), dict(xb=504), dict(xb=-512),
                dict(s=2, xt=504)):
        assert call(f, base, **bad) == -1, bad
    assert call(f, base, d=1032, xb=8 * 1032) == -2
    assert call(f, base, b=1 << 20, s=1 << 10, h=2) == -2
    assert call(f, base, b=0, x=None, y=None, first=None) == 0
    assert call(f, base, s=0, x=None, y=None, first=None) == 0


def test_append_refusals(lib):
    base = dict(x=FAKE, xb=64, xt=64, y=None, b=2, s=1, d=64, w=None, eps=1e-6, rd=16, table=FAKE, rows=10, first=FAKE,
                lens=None, step=1, base=0, window=8, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, stream=None)
    f = lib.ds_kv_append_fp4_paged
    for bad in (dict(b=-1), dict(s=-1), dict(d=0), dict(d=48), dict(eps=-1.0), dict(eps=float("nan")), dict(step=0),
                dict(base=-1), dict(window=-1), dict(rd=12), dict(rd=72), dict(table=None), dict(table=FAKE + 4),
                dict(pages=-1), dict(page=0), dict(mp=-1), dict(x=None), dict(x=FAKE + 8), dict(y=FAKE + 8),
                dict(first=None), dict(lens=FAKE + 2), dict(w=FAKE + 2), dict(codes=None), dict(codes=FAKE + 4),
                dict(exps=None), dict(bt=None), dict(bt=FAKE + 2), dict(xb=60), dict(xb=56), dict(s=2, xb=128, xt=56)):
        assert call(f, base, **bad) == -1, bad
    assert call(f, base, d=1056, xb=1056, xt=1056) == -2
    assert call(f, base, pages=1 << 27) == -2
    assert call(f, base, b=1 << 16, s=1 << 16) == -2
    assert call(f, base, b=0, x=None, codes=None, exps=None, bt=None, first=None) == 0


def test_attention_refusals(lib):
    base = dict(q=FAKE, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, sink=FAKE, idx=FAKE, topk=4, scale=0.1,
                o=FAKE, b=1, m=1, h=4, d=512, ws=None, wsb=0, rd=0, table=None, rows=0, first=None, stream=None)
    f = lib.ds_sparse_attn_fp4_paged
    for bad in (dict(b=-1), dict(m=-1), dict(h=0), dict(topk=-1), dict(pages=-1), dict(page=0), dict(mp=-1),
                dict(q=None), dict(q=FAKE + 8), dict(o=None), dict(o=FAKE + 8), dict(sink=None), dict(sink=FAKE + 2),
                dict(idx=None), dict(idx=FAKE + 2), dict(codes=None), dict(codes=FAKE + 8), dict(exps=None),
                dict(exps=FAKE + 8), dict(bt=None), dict(bt=FAKE + 1), dict(rd=12, table=FAKE, rows=9, first=FAKE),
                dict(rd=520, table=FAKE, rows=9, first=FAKE), dict(rd=16, rows=9, first=FAKE),
                dict(rd=16, table=FAKE + 4, rows=9, first=FAKE), dict(rd=16, table=FAKE, rows=9),
                dict(rd=16, table=FAKE, rows=9, first=FAKE + 2)):
        assert call(f, base, **bad) == -1, bad
    for bad in (dict(d=256), dict(h=129), dict(pages=1 << 27)):
        assert call(f, base, **bad) == -2, bad
    assert call(f, base, b=0, q=None, o=None, sink=None) == 0
    w = lib.ds_sparse_attn_fp4_paged_workspace_bytes
    assert w(1, 1, 4, 256, 8) == 0 and w(1, 1, 129, 512, 8) == 0 and w(-1, 1, 4, 512, 8) == 0


def test_refusals_of_work_that_cannot_be_numbered_and_of_missing_stores(lib):
    base = dict(q=FAKE, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, sink=FAKE, idx=FAKE, topk=4, scale=0.1,
                o=FAKE, b=1, m=1, h=4, d=512, ws=None, wsb=0, rd=0, table=None, rows=0, first=None, stream=None)
    f = lib.ds_sparse_attn_fp4_paged
    assert call(f, base, b=1 << 15, m=1 << 15) == -2
    assert call(f, base, b=1 << 14, m=1 << 15, topk=(1 << 31) - 1) == -2
    assert call(f, base, pages=0, bt=None) == -1 and call(f, base, mp=0, codes=None) == -1
    assert lib.ds_sparse_attn_fp4_paged_workspace_bytes(1 << 15, 1 << 15, 4, 512, 8) == 0


def test_bindings_refuse_cpu_tensors_and_shapes(lib):
    from sparse_latent_attention_attn_gb300 import dsattn
    x = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dsattn.norm_rotary(x, 1e-6, 0, None, ints(0))
    with pytest.raises(TypeError):
        dsattn.norm_rotary(x.float(), 1e-6, 0, None, ints(0))
    with pytest.raises(ValueError, match="CUDA"):
        dsattn.kv_append_fp4_paged(x[:, 0], torch.zeros((1, 1, 32), dtype=torch.uint8),
                                   torch.zeros((1, 1, 2), dtype=torch.int8), ints(0).view(1, 1), ints(0))
    with pytest.raises(ValueError, match="CUDA"):
        dsattn.sparse_attn_fp4_paged(x, torch.zeros((1, 1, 32), dtype=torch.uint8),
                                     torch.zeros((1, 1, 2), dtype=torch.int8), ints(0).view(1, 1), torch.zeros(2),
                                     torch.zeros((1, 1, 1), dtype=torch.int32), 0.1)


def test_the_plain_quantiser():
    """The tests' own quantiser: ties to even, the smallest scale that holds the block."""
    z = np.zeros((1, 32))
    z[0, :8] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    z[0, 8:] = -0.3
    code, k = quantise(z)
    assert k.tolist() == [[0]] and code[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 6] and (code[0, 8:] == 9).all()
    assert quantise(np.full((1, 32), 6.01))[1].tolist() == [[1]] and quantise(np.full((1, 32), 3.0))[1].tolist() == [[-1]]
    assert quantise(np.zeros((1, 32)))[1].tolist() == [[-15]]


# ---- rows of very different scale: a row's weight is its probability times its scale -------------------------

def attention_by_weight(q, rows, live, sink, scale, tops):
    """As attention(), F relative to each head's largest p 2^e (e the row's largest exponent, -96 at least): a
    probability is held to 2^-8 of itself or to 2^-17 of that, whatever exponents other rows have."""
    rows, e = rows[live], np.maximum(tops[live], -96).astype(float)
    s = scale * q @ rows.T
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    with np.errstate(over="ignore"):
        den = p.sum(-1, keepdims=True) + np.exp(sink[:, None] - top)
    worth = (np.exp((s - top) + e * math.log(2))).max(-1, keepdims=True) * (np.abs(rows) * 2.0 ** -e[:, None]).sum(0)[None]
    return p @ rows / den, p @ np.abs(rows) / den, worth / den


def check_by_weight(ds, q, codes, exps, bt, sink, idx, scale=512 ** -0.5, status=0, read=None):
    """Every element against 64 bits; `read`: the exponents as the documentation says they are read."""
    b, m = q.shape[:2]
    o = ds.sparse_attn_fp4_paged(*dev(q, codes, exps, bt, sink, idx), scale)
    assert ds.device_status() == status
    got = f64(o)
    for i in range(b):
        for t in range(m):
            ix = idx[i, t].numpy()
            rows, tops = logical_rows(codes, exps if read is None else read, bt, i, ix, codes.shape[1])
            ref, A, F = attention_by_weight(f64(q[i, t]), rows, ix >= 0, f64(sink), scale, tops)
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -17 * F + 2.0 ** -126
            assert (np.abs(got[i, t] - ref) <= tol).all(), (i, t, float((np.abs(got[i, t] - ref) / tol).max()))
    return o


@gpu
@pytest.mark.parametrize("octaves", [8, 12, 16, 20, 30, 40])
@pytest.mark.parametrize("b,h,topk", [(2, 24, 200), (1, 16, 1500), (1, 70, 90)])
def test_attention_large_row_without_weight(ds, b, h, topk, octaves):
    """One row `octaves` above the others: without probability in the even heads, whose output is the other
    rows' as if it were not listed, and with all of it in the odd ones."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(41 + octaves, b, 1, h, 2000, topk, 0.0, 16, 0)
    sign = torch.where(torch.rand(512, generator=torch.Generator().manual_seed(octaves)) < 0.5, -1.0, 1.0)
    code = torch.where(sign < 0, 10, 2).to(torch.uint8)            # -1 and 1
    exps.clamp_(max=0)
    for i in range(b):
        for at in (0, topk // 2, topk - 1):
            r = int(idx[i, 0, at])
            codes[bt[i, r // 16], r % 16] = code[0::2] | code[1::2] << 4
            exps[bt[i, r // 16], r % 16] = octaves
    half = torch.where(torch.arange(h) % 2 == 0, -1.0, 1.0)[:, None]
    q = (q.float() + 0.5 * half * sign).to(torch.bfloat16)
    o = check_by_weight(ds, q, codes, exps, bt, sink, idx)
    # without the large rows at all: the even heads' sums are the same but for their order
    rest = torch.ones(topk, dtype=torch.bool)
    rest[[0, topk // 2, topk - 1]] = False
    few = check_by_weight(ds, q, codes, exps, bt, sink, idx[..., rest].contiguous())
    worst = (o - few).float().abs()[:, :, 0::2].amax() / few.float().abs()[:, :, 0::2].amax()
    assert worst <= 2.0 ** -6


@gpu
@pytest.mark.parametrize("b,h,topk", [(2, 24, 200), (1, 70, 900)])
@pytest.mark.parametrize("k", [97, 60, 20, -20, -60, -93, -119])
def test_attention_exponent_range(ds, b, h, topk, k):
    """All rows near one end of the exponents that are read as they are."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(43, b, 1, h, 1000, topk, 0.1, 16, 0)
    q = (q.float() * 2.0 ** -k).to(torch.bfloat16)
    check_by_weight(ds, q, codes, exps + k, bt, sink, idx)
    # exponents of a block apart too: 26 below the row's largest still count
    wide = exps + k
    wide[..., 1::2] = max(k, -96) - 23
    check_by_weight(ds, q, codes, wide, bt, sink, idx)


@gpu
@pytest.mark.parametrize("b,h,topk", [(2, 24, 200), (1, 70, 900)])
@pytest.mark.parametrize("hi,lo", [(100, 4), (48, -48), (81, -15), (0, -96)])
def test_attention_both_ends_of_the_exponents(ds, b, h, topk, hi, lo):
    """Rows 96 octaves above others: with the scores of order one, and with the large rows far below."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(45, b, 1, h, 1000, topk, 0.0, 16, 0)
    odd = torch.zeros((b, 1000), dtype=torch.bool)
    for i in range(b):
        odd[i, idx[i, 0, 1::2].long()] = True
    sign = torch.where(torch.rand(512, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0)
    code = torch.where(sign < 0, 10, 2).to(torch.uint8)
    for i in range(b):
        for r in range(1000):
            exps[bt[i, r // 16], r % 16] = hi if odd[i, r] else lo
    check_by_weight(ds, q, codes, exps, bt, sink, idx, scale=2.0 ** -hi * 512 ** -0.5)
    for i in range(b):
        for r in torch.nonzero(odd[i])[:, 0].tolist():
            codes[bt[i, r // 16], r % 16] = code[0::2] | code[1::2] << 4
    low = (q.float() - 20 * sign).to(torch.bfloat16)               # their scores: about -512
    o = check_by_weight(ds, low, codes, exps, bt, torch.full_like(sink, -math.inf), idx, scale=2.0 ** -hi * 0.05)
    assert (o.abs() < 2.0 ** (lo + 4)).all() and (o != 0).any(-1).all()


@gpu
@pytest.mark.parametrize("b,h,topk", [(2, 24, 200), (1, 70, 900)])
def test_attention_exponents_outside_the_range(ds, b, h, topk):
    """Above 100: read as 100, and said so; below -122: zeros."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(47, b, 1, h, 1000, topk, 0.1, 16, 0)
    q = (q.float() * 2.0 ** -100).to(torch.bfloat16)
    for lo, hi in ((101, 127), (90, 110), (110, 121)):
        high = torch.randint(lo, hi + 1, exps.shape, generator=torch.Generator().manual_seed(lo), dtype=torch.int8)
        check_by_weight(ds, q, codes, high, bt, sink, idx, status=ds.DS_DEV_BAD_VALUE, read=high.clamp(max=100))
    # one block of one listed row is enough; of a row that is not listed, none counts
    one = torch.zeros_like(exps)
    r = int(idx[0, 0][idx[0, 0] >= 0][5])
    unlisted = next(x for x in range(1000) if x not in idx[0, 0].tolist())
    one[bt[0, unlisted // 16], unlisted % 16] = 120
    check_by_weight(ds, q, codes, one, bt, sink, idx)
    one[bt[0, r // 16], r % 16, 7] = 101
    check_by_weight(ds, q, codes, one, bt, sink, idx, status=ds.DS_DEV_BAD_VALUE, read=one.clamp(max=100))
    for lo, hi in ((-128, -123), (-128, -128), (-125, -124)):
        tiny = torch.randint(lo, hi + 1, exps.shape, generator=torch.Generator().manual_seed(hi + 200), dtype=torch.int8)
        assert (check_by_weight(ds, q, codes, tiny, bt, sink, idx, read=torch.zeros_like(tiny) - 128) == 0).all()


@gpu
def test_attention_tiny_scales_of_queries(ds):
    """Queries and scales whose product lies below the normal f32 numbers: scores of 0, not of a clamped scale."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(49, 2, 1, 24, 300, 200, 0.0, 16, 0)
    for qs, scale in ((2.0 ** -126, 1e-3), (2.0 ** -130, 1.0), (1.0, 0.0), (0.0, 1.0), (2.0 ** -120, -1e-5)):
        check_by_weight(ds, (q.float() * qs).to(torch.bfloat16), codes, exps + 44, bt, sink, idx, scale=scale)


# ---- padded batches -----------------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("b,m,h,topk", [(4, 5, 40, 150), (3, 2, 128, 700), (60, 4, 5, 33), (5, 1, 70, 0)])
def test_attention_of_a_padded_batch(ds, b, m, h, topk):
    """Tokens behind their sequence's last one: their q, positions and index rows do not matter, and o is left as
    it was; the others are those of the call without lengths."""
    g = torch.Generator().manual_seed(51)
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(51, b, m, h, 900, topk, 0.1, 16, 64)
    lens = torch.randint(0, m + 1, (b,), generator=g, dtype=torch.int32)
    lens[0], lens[1], lens[2] = 0, m + 3, -1
    live = torch.arange(m) < lens[:, None]
    tab = table_of(64 + m, 64)
    first = torch.where(lens > 0, 64 + m - lens.clamp(0, m), -9).to(torch.int32)     # padding: behind the table
    args = dev(q, codes, exps, bt, sink, idx)
    want = ds.sparse_attn_fp4_paged(*args, 512 ** -0.5)
    assert ds.device_status() == 0
    bad_q, bad_idx = q.clone(), idx.clone()
    bad_q[~live] = float("nan")
    bad_idx[~live] = 2 ** 31 - 1
    o = torch.full_like(args[0], 7.0)
    ds.sparse_attn_fp4_paged(bad_q.cuda(), *args[1:5], bad_idx.cuda(), 512 ** -0.5, lens=lens.cuda(), o=o)
    assert ds.device_status() == 0
    assert torch.equal(o.cpu()[live], want.cpu()[live]) and (o.cpu()[~live] == 7).all()
    more = dict(rd=64, table=tab.cuda(), first=first.cuda())
    turned = ds.sparse_attn_fp4_paged(bad_q.cuda(), *args[1:5], bad_idx.cuda(), 512 ** -0.5, lens=lens.cuda(), **more)
    assert ds.device_status() == 0 and (turned.cpu()[~live] == 0).all()
    for i in range(b):
        n = min(max(int(lens[i]), 0), m)
        for t in range(n):
            ix = idx[i, t].numpy()
            if topk == 0:
                assert (turned[i, t] == 0).all()
                continue
            rows, tops = logical_rows(codes, exps, bt, i, ix, 16)
            ref, A, F = attention_by_weight(f64(q[i, t]), rows, ix >= 0, f64(sink), 512 ** -0.5, tops)
            ref, A, F = rotate(ref, f64(tab)[int(first[i]) + t], inverse=True), pair_sum(A, 64), pair_sum(F, 64)
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -17 * F
            assert (np.abs(f64(turned[i, t]) - ref) <= tol).all()
    with pytest.raises((TypeError, ValueError)):
        ds.sparse_attn_fp4_paged(*args, 0.1, lens=lens.cuda().long())
    with pytest.raises((TypeError, ValueError)):
        ds.sparse_attn_fp4_paged(*args, 0.1, lens=lens[:-1].cuda())


@gpu
def test_step_of_several_tokens_in_a_padded_batch(ds):
    """Three tokens a step, some sequences with fewer or none (their pages and position then do not matter, and the
    padding lies behind the table), a ring that is full and holds the step's tokens beside the window: every
    token against 64 bits."""
    from sparse_latent_attention_attn_gb300 import path
    g = torch.Generator().manual_seed(8)
    b, s, h, d, rd, window, page, eps = 5, 3, 20, 512, 64, 12, 5, 1e-6
    ring = window + s - 1                                  # slots: the window of the first token and the later ones
    codes, exps, bt = random_pool(g, b, ring, page, d)
    tab = table_of(60, rd)
    w = 1 + 0.1 * torch.randn((d,), generator=g)
    sink = torch.randn((h,), generator=g)
    q = torch.randn((b, s, h, d), generator=g).to(torch.bfloat16)
    kv = torch.randn((b, s, d), generator=g).to(torch.bfloat16)
    first, lens = ints(40, 57, 3, 59, -5), ints(3, 3, 2, 1, 0)
    bt[4] = -1
    live = torch.arange(s) < lens[:, None]
    idx = torch.full((b, s, window), 2 ** 31 - 1, dtype=torch.int32)
    for i in range(b):
        for t in range(int(lens[i])):
            pos = torch.arange(int(first[i]) + t - window + 1, int(first[i]) + t + 1)
            idx[i, t] = torch.where(pos >= 0, pos % ring, -1)
    q[~live], kv[~live] = float("nan"), float("nan")
    qg, kg, cg, eg, btg, fg, sg, ig, tg, wg, lg = dev(q, kv, codes, exps, bt, first, sink, idx, tab, w, lens)
    o = torch.full_like(qg, 7.0)
    for given in (o, None):
        got = path.decode_step_fp4_paged(qg, kg, cg, eg, btg, fg, sg, ig, ring, d ** -0.5, rd, tg, eps, kv_weight=wg,
                                         lens=lg, o=given)
        assert ds.device_status() == 0
        assert (got.cpu()[~live] == (0 if given is None else 7)).all()
    assert torch.equal(got.cpu()[live], o.cpu()[live])
    zero = torch.where(live[..., None], kv, 0)
    ref_c, ref_e, _ = append_reference(zero, w, eps, rd, table_of(70, rd), first.clamp(min=0), lens, 1, 0, ring, codes, exps,
                                       bt, torch.zeros_like(kv))
    np.testing.assert_array_equal(cg.cpu().numpy(), ref_c)
    np.testing.assert_array_equal(eg.cpu().numpy(), ref_e)
    for i in range(b):
        for t in range(int(lens[i])):
            cs = f64(tab)[int(first[i]) + t][None]
            zq = f64(torch.from_numpy(rotate(normed(f64(q[i, t]), None, eps), cs)).to(torch.bfloat16))
            rr, tops = logical_rows(torch.from_numpy(ref_c), torch.from_numpy(ref_e), bt, i, idx[i, t].numpy(), page)
            ref, A, F = attention_by_weight(zq, rr, idx[i, t].numpy() >= 0, f64(sink), d ** -0.5, tops)
            ref = rotate(ref, cs, inverse=True)
            A, F = pair_sum(A, rd), pair_sum(F, rd)
            # q may be one bf16 step off where the norm's f32 falls on the other side of a border
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * A + 2.0 ** -17 * F
            assert (np.abs(f64(got[i, t]) - ref) <= tol).all()


def test_attention_of_a_padded_batch_refusals(lib):
    base = dict(q=FAKE, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, sink=FAKE, idx=FAKE, topk=4, scale=0.1,
                o=FAKE, b=1, m=1, h=4, d=512, ws=None, wsb=0, rd=0, table=None, rows=0, first=None, lens=FAKE, stream=None)
    f = lib.ds_sparse_attn_fp4_paged_ragged
    for bad in (dict(lens=FAKE + 2), dict(lens=FAKE + 1, topk=0), dict(q=None), dict(o=FAKE + 8), dict(h=0), dict(rd=16, rows=9)):
        assert call(f, base, **bad) == -1, bad
    assert call(f, base, h=129) == -2 and call(f, base, b=0, q=None, o=None, sink=None) == 0


def test_refusal_of_lists_too_long_to_count(lib):
    base = dict(q=FAKE, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, sink=FAKE, idx=FAKE, topk=4, scale=0.1,
                o=FAKE, b=1, m=1, h=4, d=512, ws=None, wsb=0, rd=0, table=None, rows=0, first=None, stream=None)
    for topk in (2 ** 31 - 1, 2 ** 31 - 256):
        assert call(lib.ds_sparse_attn_fp4_paged, base, topk=topk) == -2
        assert lib.ds_sparse_attn_fp4_paged_workspace_bytes(1, 1, 4, 512, topk) == 0


def test_append_refuses_an_eps_that_is_next_to_nothing(lib):
    base = dict(x=FAKE, xb=64, xt=64, y=None, b=2, s=1, d=64, w=None, eps=1e-6, rd=0, table=None, rows=0, first=FAKE,
                lens=None, step=1, base=0, window=8, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, stream=None)
    for eps in (1e-40, 7.8e-31, -1e-40, float("nan")):
        assert call(lib.ds_kv_append_fp4_paged, base, eps=eps) == -1
    assert call(lib.ds_kv_append_fp4_paged, base, eps=2.0 ** -100, b=0) == 0


@gpu
def test_append_binding_refuses_an_eps_that_rounds_to_none(ds):
    x = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((1, 4, 32), 9, dtype=torch.uint8, device="cuda")
    exps = torch.full((1, 4, 2), 9, dtype=torch.int8, device="cuda")
    for eps in (1e-50, 1e-40):
        with pytest.raises(ds.DsError):
            ds.kv_append_fp4_paged(x, codes, exps, ints(0).view(1, 1).cuda(), ints(0).cuda(), eps=eps)
    torch.cuda.synchronize()
    assert (codes == 9).all() and (exps == 9).all()


@gpu
def test_bindings_refuse_numbers_beyond_an_int(ds):
    """Numbers whose low 32 bits would be another valid call."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    wide = 1 << 32
    app = dict(x=z(1, 1, 64), codes=z(1, 8, 32, dt=torch.uint8), exps=z(1, 8, 2, dt=torch.int8),
               block_table=z(1, 1, dt=torch.int32), first=z(1, dt=torch.int32))
    pool = dict(codes=z(0, wide + 8, 32, dt=torch.uint8), exps=z(0, wide + 8, 2, dt=torch.int8))
    app["codes"].fill_(9)
    for bad in (dict(base=wide), dict(window=wide + 8), dict(pos_step=wide + 1), dict(base=-wide), dict(base=2 ** 31), pool):
        with pytest.raises(ds.DsError):
            ds.kv_append_fp4_paged(**{**app, **bad})
    assert ds.device_status() == 0 and (app["codes"] == 9).all()
    with pytest.raises(ds.DsError):                        # in an int, and refused for what it is
        ds.kv_append_fp4_paged(**app, base=-1)
    attn = dict(q=z(1, 1, 4, 512), codes=z(0, wide + 16, 256, dt=torch.uint8), exps=z(0, wide + 16, 16, dt=torch.int8),
                block_table=z(1, 1, dt=torch.int32), sink=z(4, dt=torch.float32), idx=z(1, 1, 3, dt=torch.int32), scale=0.1)
    with pytest.raises(ds.DsError):
        ds.sparse_attn_fp4_paged(**attn)
    with pytest.raises((ds.DsError, ValueError)):
        ds.norm_rotary(z(1, 1, 4, 64), 1e-6, wide, z(4, 0, 2, dt=torch.float32), z(1, dt=torch.int32))
    assert ds.device_status() == 0


@gpu
def test_attention_asks_anew_for_a_workspace_after_a_failure(ds, monkeypatch):
    """The size of a shape's workspace is kept, but not that of a query that failed (0)."""
    x = attention_inputs(53, 1, 1, 16, 3000, 2300, 0.1, 64, 0)
    args = dev(*x[:6]) + [512 ** -0.5]
    assert ds.sparse_attn_fp4_paged_workspace_bytes(1, 1, 16, 512, 2300) > 0
    ds._fp4_workspace_bytes.cache_clear()
    with monkeypatch.context() as mp:
        mp.setattr(ds, "sparse_attn_fp4_paged_workspace_bytes", lambda *a: 0)
        with pytest.raises(ds.DsError):
            ds.sparse_attn_fp4_paged(*args)
    check_attention(ds, *x)


IMPORT_WITHOUT = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from sparse_latent_attention_attn_gb300 import dsattn
assert dsattn._device is torch.cuda.current_device
"""


def test_import_without_the_private_functions_of_torch(lib):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", IMPORT_WITHOUT], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@gpu
@pytest.mark.parametrize("b,m,h,topk", [(2, 1, 40, 150), (1, 1, 70, 2300), (200, 1, 100, 130), (1, 1, 3, 1)])
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_attention_of_queries_that_are_not_finite(ds, b, m, h, topk, what):
    """One such value makes its head's output NaN, in units whole and cut; the other heads are as without it."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(55, b, m, h, 3000, topk, 0.1, 16, 0)
    idx[0, 0, 0] = 7
    args = dev(q, codes, exps, bt, sink, idx)
    want = ds.sparse_attn_fp4_paged(*args, 512 ** -0.5)
    hit = torch.zeros((b, m, h), dtype=torch.bool)
    hit[0, 0, h // 2] = hit[-1, -1, 0] = True
    bad = q.clone()
    bad[0, 0, h // 2, 77] = what
    bad[-1, -1, 0, 0] = what
    got = ds.sparse_attn_fp4_paged(bad.cuda(), *args[1:], 512 ** -0.5)
    assert ds.device_status() == 0
    none = (idx < 0).all(-1)[..., None] & hit              # without rows: 0, whatever q is
    assert got.cpu()[hit & ~none].isnan().all() and (got.cpu()[none] == 0).all()
    assert torch.equal(got.cpu()[~hit], want.cpu()[~hit])


@gpu
@pytest.mark.parametrize("d,rd", [(1024, 1024), (544, 64), (992, 480)])
def test_append_many_wide_rows(ds, d, rd):
    """Rows above 512 values, enough of them that many values lie next to a border between two codes."""
    g = torch.Generator().manual_seed(d)
    b, s = 3, 700
    x = (torch.randn((b, s, d), generator=g) * 2).to(torch.bfloat16)
    w = torch.randn((d,), generator=g)
    first, tab = ints(0, 300, 77), table_of(1000, rd, 1.25)
    codes, exps, bt = random_pool(g, b, 1000, 48, d)
    y = torch.zeros((b, s, d), dtype=torch.bfloat16)
    want = append_reference(x, w, 1e-6, rd, tab, first, None, 1, 0, 0, codes, exps, bt, y)
    xg, cg, eg, btg, fg, wg, tg, yg = dev(x, codes, exps, bt, first, w, tab, y)
    ds.kv_append_fp4_paged(xg, cg, eg, btg, fg, rd=rd, table=tg, eps=1e-6, weight=wg, y=yg)
    assert ds.device_status() == 0
    np.testing.assert_array_equal(eg.cpu().numpy(), want[1])
    np.testing.assert_array_equal(cg.cpu().numpy(), want[0])
    np.testing.assert_array_equal(f64(yg), want[2])


@gpu
@pytest.mark.parametrize("rd", [0, 8])
def test_append_of_the_largest_values(ds, rd):
    """Values up to bf16's largest: below 3.5 * 2^126 y is finite, from there on the code stands for 2^128."""
    top = torch.tensor([3.5 * 2.0 ** 126, float(torch.finfo(torch.bfloat16).max)]).to(torch.bfloat16)
    x = torch.randn((1, 4, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    x[0, 0, 3] = (top[:1].view(torch.int16) - 1).view(torch.bfloat16)[0]
    x[0, 1, 40], x[0, 1, 5] = top[0], -top[1]
    x[0, 2, 20] = -3 * 2.0 ** 125
    x[0, 3] = x[0, 3].float() * 2.0 ** 124
    codes = torch.zeros((4, 1, 32), dtype=torch.uint8)
    exps = torch.zeros((4, 1, 2), dtype=torch.int8)
    bt = torch.arange(4, dtype=torch.int32)[None]
    tab = table_of(4, rd) if rd else None
    y = torch.zeros_like(x)
    want = append_reference(x, None, 0.0, rd, tab, ints(0), None, 1, 0, 0, codes, exps, bt, y)
    cg, eg, btg, fg, yg, tg = dev(codes, exps, bt, ints(0), y, tab)
    ds.kv_append_fp4_paged(x.cuda(), cg, eg, btg, fg, rd=rd, table=tg, y=yg)
    np.testing.assert_array_equal(eg.cpu().numpy(), want[1])
    np.testing.assert_array_equal(cg.cpu().numpy(), want[0])
    stored = np.where(np.abs(want[2]) == 2.0 ** 128, np.copysign(math.inf, want[2]), want[2])
    np.testing.assert_array_equal(f64(yg), stored)
    assert int(exps.new_tensor(want[1]).max()) == 126 and np.isinf(stored).sum() == 2 and np.isfinite(stored[0, 0]).all()


def test_step_refuses_more_tokens_than_the_ring_holds(lib):
    from sparse_latent_attention_attn_gb300 import path
    q = torch.zeros((1, 5, 2, 512), dtype=torch.bfloat16)
    store = (torch.zeros((1, 16, 256), dtype=torch.uint8), torch.zeros((1, 16, 16), dtype=torch.int8), ints(0).view(1, 1))
    with pytest.raises(ValueError, match="ring"):
        path.decode_step_fp4_paged(q, q[:, :, 0], *store, ints(0), torch.zeros(2), torch.zeros((1, 5, 4), dtype=torch.int32), 4,
                                   0.1, 0, None, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):          # five slots are enough: refused for the CPU tensors only
        path.decode_step_fp4_paged(q, q[:, :, 0], *store, ints(0), torch.zeros(2), torch.zeros((1, 5, 4), dtype=torch.int32), 5,
                                   0.1, 0, None, 1e-6)


@gpu
def test_step_of_several_tokens_without_a_ring(ds):
    """window = 0: rows are positions; three tokens a step, the same as three steps of one."""
    from sparse_latent_attention_attn_gb300 import path
    g = torch.Generator().manual_seed(12)
    b, s, h, d, rd, page, eps = 2, 3, 9, 512, 64, 7, 1e-6
    codes, exps, bt = random_pool(g, b, 40, page, d)
    tab, sink = table_of(60, rd), torch.randn((h,), generator=g)
    q = torch.randn((b, s, h, d), generator=g).to(torch.bfloat16)
    kv = torch.randn((b, s, d), generator=g).to(torch.bfloat16)
    first = ints(30, 5)
    idx = torch.arange(40, dtype=torch.int32).expand(b, s, 40).clone()
    idx[idx > (first[:, None] + torch.arange(s))[..., None]] = -1
    qg, kg, btg, fg, sg, ig, tg = dev(q, kv, bt, first, sink, idx, tab)
    c1, e1 = dev(codes, exps)
    whole = path.decode_step_fp4_paged(qg, kg, c1, e1, btg, fg, sg, ig, 0, d ** -0.5, rd, tg, eps)
    c2, e2 = dev(codes, exps)
    for t in range(s):
        one = path.decode_step_fp4_paged(qg[:, t:t + 1].contiguous(), kg[:, t:t + 1].contiguous(), c2, e2, btg, fg + t, sg,
                                         ig[:, t:t + 1].contiguous(), 0, d ** -0.5, rd, tg, eps)
        assert torch.equal(one, whole[:, t:t + 1])
    assert torch.equal(c1, c2) and torch.equal(e1, e2) and ds.device_status() == 0


# ---- with the library's other calls --------------------------------------------------------------------------

def against_64_bits(got, q, codes, exps, bt, seq, ix, page, sink, scale, tab, pos, rd):
    rows, tops = logical_rows(codes, exps, bt, seq, ix, page)
    ref, A, F = attention_by_weight(f64(q), rows, ix >= 0, f64(sink), scale, tops)
    ref, A, F = rotate(ref, f64(tab)[pos][None], inverse=True), pair_sum(A, rd), pair_sum(F, rd)
    assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -17 * F).all()


@gpu
def test_index_rows_of_the_library_for_sequences_at_their_own_positions(ds):
    """Window rows by ds_window_topk_idxs and compressed ones by ds_indexer_topk, a call for each sequence."""
    g = torch.Generator().manual_seed(61)
    b, h, d, rd, W, page, ratio, topk = 3, 12, 512, 64, 32, 8, 4, 40
    start = [300, 17, 131]
    codes, exps, bt = random_pool(g, b, W + 80, page, d)
    q, sink, tab = torch.randn((b, 1, h, d), generator=g).to(torch.bfloat16), torch.randn((h,), generator=g), table_of(400, rd)
    iq, ik = torch.randn((b, 1, 64, 128), generator=g).to(torch.bfloat16), torch.randn((b, 80, 128), generator=g).to(torch.bfloat16)
    iw = torch.rand((b, 1, 64), generator=g)
    idx = torch.full((b, 1, W + topk), -1, dtype=torch.int32, device="cuda")
    for i in range(b):
        assert ds.window_topk_idxs(idx[i], 1, 1, start[i], W) == W
        comp = ds.indexer_topk(*dev(iq[i:i + 1], ik[i:i + 1], iw[i:i + 1]), start[i], ratio, topk, offset=W)
        idx[i, 0, W:W + comp.shape[-1]] = comp[0, 0]
    ix = idx.cpu()
    for i in range(b):
        ring = sorted(v for v in ix[i, 0, :W].tolist() if v >= 0)
        assert ring == sorted({p % W for p in range(max(0, start[i] - W + 1), start[i] + 1)})
        comp = [v for v in ix[i, 0, W:].tolist() if v >= 0]
        assert len(comp) == min(topk, (start[i] + 1) // ratio) and all(W <= v < W + (start[i] + 1) // ratio for v in comp)
    o = ds.sparse_attn_fp4_paged(*dev(q, codes, exps, bt, sink), idx, d ** -0.5, rd=rd, table=tab.cuda(), first=ints(*start).cuda())
    assert ds.device_status() == 0
    for i in range(b):
        against_64_bits(o[i, 0], q[i, 0], codes, exps, bt, i, ix[i, 0].numpy(), page, sink, d ** -0.5, tab, start[i], rd)


@gpu
def test_prompt_and_decode_share_one_store(ds):
    """A prompt through a block table of its own, the compressed rows' pages shared with the decode table; then a
    decode step over ring and compressed rows."""
    from sparse_latent_attention_attn_gb300 import path
    g = torch.Generator().manual_seed(63)
    n, W, page, ratio, h, d, rd, eps = 40, 16, 8, 4, 10, 512, 64, 1e-6
    ncomp, scale = n // ratio, d ** -0.5
    order = torch.randperm(20, generator=g).to(torch.int32)
    chunk, comp, ring = order[:n // page], order[5:8], order[8:8 + W // page]
    prompt_bt, decode_bt = torch.cat((chunk, comp))[None].contiguous(), torch.cat((ring, comp))[None].contiguous()
    codes = torch.zeros((20, page, d // 2), dtype=torch.uint8, device="cuda")
    exps = torch.zeros((20, page, d // 32), dtype=torch.int8, device="cuda")
    tab, sink, w = table_of(64, rd), torch.randn((h,), generator=g), 1 + 0.1 * torch.randn((d,), generator=g)
    kv = torch.randn((1, n, d), generator=g).to(torch.bfloat16)
    ckv = torch.randn((1, ncomp, d), generator=g).to(torch.bfloat16)
    q = torch.randn((1, n, h, d), generator=g).to(torch.bfloat16)
    kvg, cg, qg, tg, sg, wg, pt, dt = dev(kv, ckv, q, tab, sink, w, prompt_bt, decode_bt)
    zero = ints(0).cuda()
    more = dict(rd=rd, table=tg, eps=eps, weight=wg)
    ds.kv_append_fp4_paged(kvg, codes, exps, pt, zero, **more)
    ds.kv_append_fp4_paged(kvg, codes, exps, dt, zero, window=W, **more)
    ds.kv_append_fp4_paged(cg, codes, exps, dt, zero, pos_step=ratio, base=W, **more)
    idx = torch.full((1, n, W + ncomp), -1, dtype=torch.int32, device="cuda")
    assert ds.window_topk_idxs(idx, 1, n, 0, W) == W
    seen = torch.arange(n, device="cuda")[:, None] + 1
    j = torch.arange(ncomp, device="cuda")
    idx[0, :, W:] = torch.where((j + 1) * ratio <= seen, n + j, -1).to(torch.int32)
    qn = ds.norm_rotary(qg, eps, rd, tg, zero)
    o = ds.sparse_attn_fp4_paged(qn, codes, exps, pt, sg, idx, scale, rd=rd, table=tg, first=zero)
    assert ds.device_status() == 0
    hc, he, ix = codes.cpu(), exps.cpu(), idx.cpu()
    ref = append_reference(kv, w, eps, rd, tab, ints(0), None, 1, 0, 0, torch.zeros_like(hc), torch.zeros_like(he), prompt_bt,
                           torch.zeros_like(kv))
    assert (hc.numpy()[chunk.numpy()] == ref[0][chunk.numpy()]).all()
    for t in range(n):
        against_64_bits(o[0, t], qn[0, t].cpu(), hc, he, prompt_bt, 0, ix[0, t].numpy(), page, sink, scale, tab, t, rd)
    # the chunk's own pages are free now: other rows may take them
    codes[chunk.long().cuda()] = 255
    exps[chunk.long().cuda()] = 40
    nq, nkv = torch.randn((1, 1, h, d), generator=g).to(torch.bfloat16), torch.randn((1, 1, d), generator=g).to(torch.bfloat16)
    step = torch.full((1, 1, W + ncomp), -1, dtype=torch.int32, device="cuda")
    ds.window_topk_idxs(step, 1, 1, n, W)
    step[0, 0, W:] = W + j
    at = ints(n).cuda()
    o = path.decode_step_fp4_paged(nq.cuda(), nkv.cuda(), codes, exps, dt, at, sg, step, W, scale, rd, tg, eps, kv_weight=wg)
    assert ds.device_status() == 0
    qd = ds.norm_rotary(nq.cuda(), eps, rd, tg, at).cpu()
    hc, he = codes.cpu(), exps.cpu()
    rows = logical_rows(hc, he, decode_bt, 0, np.arange(W), page)[0]
    for p in range(n - W + 1, n):                          # the ring holds the prompt's last rows
        one = append_reference(kv[:, p:p + 1], w, eps, rd, tab, ints(p), None, 1, 0, W, hc, he, decode_bt, torch.zeros_like(nkv))
        np.testing.assert_array_equal(rows[p % W], one[2][0, 0])
    against_64_bits(o[0, 0], qd[0, 0], hc, he, decode_bt, 0, step.cpu()[0, 0].numpy(), page, sink, scale, tab, n, rd)


# ---- long ranges of units, and the workloads' own shapes -----------------------------------------------------------

@gpu
@pytest.mark.parametrize("b,m,h,rows,topk,page", [
    (1, 4096, 5, 700, 30, 16),            # 27 units a CTA, one short tile each
    (16, 200, 70, 300, 150, 12),          # 42 units a CTA, two tiles each, two groups of heads
    (3, 1001, 16, 900, 260, 7),           # three tiles, cut wherever the ranges end
])
def test_attention_long_ranges_of_units(ds, b, m, h, rows, topk, page):
    """Many units a CTA: messages, phases, both scale buffers and the order from both ends wrap many times.  Some
    tokens list nothing, some are padding; a sample against 64 bits, all against calls of a few tokens."""
    g = torch.Generator().manual_seed(m)
    q, codes, exps, bt, sink, idx, rd, _, tab = attention_inputs(65, b, m, h, rows, topk, 0.2, page, 64)
    first, tab = torch.randint(0, 50, (b,), generator=g, dtype=torch.int32), table_of(50 + m, 64)
    empty = torch.rand((b, m), generator=g) < 0.05
    idx[empty] = -1
    lens = torch.randint(m // 2, m + 1, (b,), generator=g, dtype=torch.int32)
    live = torch.arange(m) < lens[:, None]
    qg, cg, eg, btg, sg, ig, fg, tg, lg = dev(q, codes, exps, bt, sink, idx, first, tab, lens)
    o = ds.sparse_attn_fp4_paged(qg, cg, eg, btg, sg, ig, 512 ** -0.5, rd=rd, table=tg, first=fg, lens=lg,
                                 o=torch.full_like(qg, 7.0))
    assert ds.device_status() == 0
    got = o.cpu()
    assert (got[~live] == 7).all() and (got[live & empty] == 0).all() and got.isfinite().all()
    assert (got[live & ~empty] != 0).any(-1).all()
    for j in np.random.RandomState(2).choice(int(live.sum()), 40, replace=False):
        i, t = (int(v) for v in torch.nonzero(live)[j])
        if not empty[i, t]:
            against_64_bits(got[i, t], q[i, t], codes, exps, bt, i, idx[i, t].numpy(), page, sink, 512 ** -0.5, tab,
                            int(first[i]) + t, rd)
    # every token again in calls of a few (other ranges, other CTAs): a token's result may differ by how its list is cut
    # into parts, which is within twice the bound of a sum |v| <= 6 * 2^3 of probabilities
    for i in range(b):
        for t in range(0, m, 37):
            few = ds.sparse_attn_fp4_paged(qg[i:i + 1, t:t + 37], cg, eg, btg[i:i + 1], sg, ig[i:i + 1, t:t + 37], 512 ** -0.5,
                                           rd=rd, table=tg, first=fg[i:i + 1] + t)
            there = live[i, t:t + 37]
            far = (few[0].cpu().float() - got[i, t:t + 37].float()).abs()[there]
            assert (far <= 2 * (2.0 ** -7 + 2.0 ** -11) * 48).all()
    assert ds.device_status() == 0


@gpu
def test_attention_of_a_causal_prompt(ds):
    """A prompt of 4096 tokens at 64 heads: causal windows of 128 and up to 512 of 1024 compressed rows, of which
    the early tokens see few; a sample of tokens against 64 bits."""
    g = torch.Generator().manual_seed(67)
    n, h, win, comp, topk, page, rd = 4096, 64, 128, 1024, 512, 64, 64
    codes, exps, bt = random_pool(g, 1, n + comp, page, 512)
    q = torch.randn((1, n, h, 512), generator=g).to(torch.bfloat16)
    sink, tab, first = torch.randn((h,), generator=g), table_of(n, rd), ints(0)
    at = torch.arange(n)[:, None]
    w = (at - win + 1).clamp(min=0) + torch.arange(win)
    w = torch.where(w <= at, w, -1)
    keys = torch.rand((n, comp), generator=g)
    keys[torch.arange(comp) >= (at + 1) // 4] = -1
    val, c = keys.topk(topk, dim=-1)
    c = torch.where(val >= 0, c + n, -1)
    idx = torch.cat((w, c), -1).to(torch.int32)[None].contiguous()
    o = ds.sparse_attn_fp4_paged(*dev(q, codes, exps, bt, sink, idx), 512 ** -0.5, rd=rd, table=tab.cuda(), first=first.cuda())
    assert ds.device_status() == 0
    assert o.isfinite().all() and (o != 0).any(-1).all()
    for t in [0, 1, 2, 3, 126, 127, 128, 129, 4095] + np.random.RandomState(4).choice(n, 25, replace=False).tolist():
        against_64_bits(o[0, t], q[0, t], codes, exps, bt, 0, idx[0, t].numpy(), page, sink, 512 ** -0.5, tab, t, rd)


@gpu
def test_attention_of_a_full_decode_batch(ds):
    """256 sequences at 128 heads over 128 ring rows and 2048 of 32768 compressed ones, some entries unseen; a sample."""
    g = torch.Generator(device="cuda").manual_seed(69)
    b, h, win, comp, topk, page, rd = 256, 128, 128, 32768, 2048, 64, 64
    per = (win + comp) // page
    bt = torch.randperm(b * per, generator=g, device="cuda").view(b, per).to(torch.int32)
    codes = torch.randint(0, 256, (b * per, page, 256), generator=g, device="cuda", dtype=torch.uint8)
    exps = torch.randint(-2, 2, (b * per, page, 16), generator=g, device="cuda", dtype=torch.int8)
    q = torch.randn((b, 1, h, 512), generator=g, device="cuda").to(torch.bfloat16)
    sink = torch.randn((h,), generator=g, device="cuda")
    c = torch.rand((b, comp), generator=g, device="cuda").topk(topk, dim=-1).indices + win
    c = torch.where(torch.rand((b, topk), generator=g, device="cuda") < 0.02, -1, c)
    idx = torch.cat((torch.arange(win, device="cuda").expand(b, -1), c), -1).to(torch.int32)[:, None].contiguous()
    first, tab = torch.randint(0, 90, (b,), generator=g, device="cuda", dtype=torch.int32), table_of(100, rd)
    o = ds.sparse_attn_fp4_paged(q, codes, exps, bt, sink, idx, 512 ** -0.5, rd=rd, table=tab.cuda(), first=first)
    assert ds.device_status() == 0 and o.isfinite().all() and (o != 0).any(-1).all()
    for i in np.random.RandomState(6).choice(b, 6, replace=False).tolist():
        pages = bt[i].long()
        mine = torch.arange(per, dtype=torch.int32)[None]                # this sequence's pages alone
        against_64_bits(o[i, 0], q[i, 0], codes[pages].cpu(), exps[pages].cpu(), mine, 0, idx[i, 0].cpu().numpy(), page,
                        sink.cpu(), 512 ** -0.5, tab, int(first[i]), rd)


@gpu
def test_attention_without_its_bad_entries(ds):
    """Entries past the table, without a page or with one that is not there: every element as without them."""
    q, codes, exps, bt, sink, idx, *_ = attention_inputs(71, 3, 2, 40, 200, 150, 0.1, 16, 0)
    g = torch.Generator().manual_seed(71)
    hole = bt.clone()
    hole[0, 3], hole[1, 5], hole[2, 0] = -1, codes.shape[0], -2 ** 31
    wild = torch.where(torch.rand(idx.shape, generator=g) < 0.1,
                       torch.tensor([13 * 16, 13 * 16 + 5, 2 ** 31 - 1, 10 ** 6])[torch.randint(0, 4, idx.shape, generator=g)], idx)
    wild = wild.to(torch.int32)
    # entries of missing pages count as not listed
    page = (wild.clamp(min=0) // 16).long()
    inside = (wild >= 0) & (page < 13)
    there = inside & (torch.gather(hole.long(), 1, page.clamp(max=12).flatten(1)).view(page.shape) >= 0)
    there &= torch.gather(hole.long(), 1, page.clamp(max=12).flatten(1)).view(page.shape) < codes.shape[0]
    kept = torch.where(there, wild, -1)
    assert (there != (wild >= 0)).any(-1).all()
    o = ds.sparse_attn_fp4_paged(*dev(q, codes, exps, hole, sink, wild), 512 ** -0.5)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    for i in range(3):
        for t in range(2):
            ix = kept[i, t].numpy()
            rows, tops = logical_rows(codes, exps, bt, i, ix, 16)
            ref, A, F = attention_by_weight(f64(q[i, t]), rows, ix >= 0, f64(sink), 512 ** -0.5, tops)
            assert (np.abs(f64(o[i, t]) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -17 * F).all()


@gpu
def test_a_refused_launch_does_not_fail_the_next_call(ds):
    """A launch that CUDA refuses (on the legacy stream while a blocking stream is captured) returns its error, and
    only that call does."""
    rt = ctypes.CDLL("libcudart.so.13")
    x = attention_inputs(73, 1, 1, 4, 40, 20, 0.0, 8, 0)
    qg, cg, eg, btg, sg, ig = dev(*x[:6])
    o = torch.empty_like(qg)
    row = torch.ones((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    y, zero = torch.zeros_like(row), ints(0).cuda()
    attend = lambda: ds._lib.ds_sparse_attn_fp4_paged(qg.data_ptr(), cg.data_ptr(), eg.data_ptr(), cg.shape[0], 8, btg.data_ptr(),
                                                      btg.shape[1], sg.data_ptr(), ig.data_ptr(), 20, 0.1, o.data_ptr(), 1, 1, 4,
                                                      512, None, 0, 0, None, 0, None, None)
    norm = lambda: ds._lib.ds_norm_rotary(row.data_ptr(), 64, 64, y.data_ptr(), 1, 1, 1, 64, None, 1e-6, 0, None, 0,
                                          zero.data_ptr(), None, None)
    assert attend() == 0 and norm() == 0
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    for refused in (attend, norm):
        assert rt.cudaStreamBeginCapture(stream, 0) == 0           # 0: global
        first = refused()
        assert rt.cudaStreamEndCapture(stream, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
        assert first == -4
        y.zero_()
        assert norm() == 0 and attend() == 0
        torch.cuda.synchronize()
        assert (y != 0).all() and ds.device_status() == 0
    assert rt.cudaStreamDestroy(stream) == 0


@gpu
@pytest.mark.parametrize("h,W", [(20, 40), (100, 300)])
def test_padded_step_captured_and_replayed(ds, h, W):
    """A step of two tokens captured with lens: each replay takes the lengths, positions and rows of its time; and
    the same on a stream given by hand."""
    from sparse_latent_attention_attn_gb300 import path
    g = torch.Generator().manual_seed(81)
    b, s, d, rd, page, eps = 3, 2, 512, 64, 16, 1e-6
    codes, exps, bt = random_pool(g, b, W, page, d)
    tab, sink = table_of(W + 60, rd).cuda(), torch.randn((h,), generator=g).cuda()
    btg = bt.cuda()
    static = {"q": torch.zeros((b, s, h, d), dtype=torch.bfloat16, device="cuda"),
              "kv": torch.zeros((b, s, d), dtype=torch.bfloat16, device="cuda"),
              "first": torch.zeros((b,), dtype=torch.int32, device="cuda"),
              "lens": torch.full((b,), s, dtype=torch.int32, device="cuda"),
              "idx": torch.zeros((b, s, W), dtype=torch.int32, device="cuda")}
    o = torch.zeros((b, s, h, d), dtype=torch.bfloat16, device="cuda")

    def step(c, e, out, stream=None):
        return path.decode_step_fp4_paged(static["q"], static["kv"], c, e, btg, static["first"], sink, static["idx"], W,
                                          d ** -0.5, rd, tab, eps, lens=static["lens"], o=out, stream=stream)

    one, two = dev(codes, exps), dev(codes, exps)
    step(*dev(codes, exps), torch.zeros_like(o))
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step(*one, o)
    for n, lens in enumerate((ints(2, 1, 0), ints(0, 2, 2), ints(0, 0, 0), ints(1, 2, 9))):
        first = torch.randint(W, W + 50, (b,), generator=g, dtype=torch.int32)
        idx = torch.stack([torch.randperm(W, generator=g) for _ in range(b * s)]).view(b, s, W).to(torch.int32)
        for k, v in (("q", torch.randn((b, s, h, d), generator=g)), ("kv", torch.randn((b, s, d), generator=g)),
                     ("first", first), ("lens", lens), ("idx", idx)):
            static[k].copy_(v)
        live = torch.arange(s) < lens[:, None]
        o.fill_(5.0)
        other = torch.full_like(o, 5.0)
        torch.cuda.synchronize()
        graph.replay()
        step(*two, other, stream=side)
        torch.cuda.synchronize()
        assert ds.device_status() == 0
        assert torch.equal(o, other) and torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        assert (o.cpu()[~live] == 5).all() and (o.cpu()[live] != 5).any(-1).all()
        for i, t in torch.nonzero(live).tolist():
            zq = ds.norm_rotary(static["q"], eps, rd, tab, static["first"])[i, t].cpu()
            against_64_bits(o[i, t], zq, one[0].cpu(), one[1].cpu(), bt, i, idx[i, t].numpy(), page, sink.cpu(), d ** -0.5,
                            tab.cpu(), int(first[i]) + t, rd)
