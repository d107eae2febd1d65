"""The paged 8-bit row store: ds_kv_append_fp8_paged, ds_kv_read_fp8_paged (and ds_kv_read_fp4_paged) and
ds_chunk_attn_fp8_paged against plain implementations in 64 bits, their refusals, and a run of them together.

Tolerances.  Codes, exponents and the rows read back are equal.  An attention output is rounded to bf16, off by half a
step, 2^-8 of its value, and so is each probability before the value product: 2^-8 of A = sum p |v| / l.  A score is
512 products added up in f32, off by at most 512 * 2^-23 of S = scale * sum |q| |k| (each sum rounded, or cut
off), and its exponent, with at most 2^10 octaves between a score and the reference, by 2^10 * 2^-23; both move p and
l, and with them an output by at most twice that of A; exponentials and sums add less than 2^-12 of A.  Hence
2^-8 |o| + (2^-8 + 2^-12 + 2^-12 + 2 * 2^-14 S) A; a rotation adds up both values of a pair.  An output below f32's least
normal number, 2^-126, may come as 0.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
NAN8 = 0x7F                # an e4m3 code that stands for NaN: what slots hold that nothing may read


# ---- plain implementations, 64 bits, on the CPU ---------------------------------------------------

def f64(t):
    return t.detach().cpu().double().numpy()


def table_of(positions, rd):
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rd, 2) / max(rd, 1))[None]
    return torch.from_numpy(np.stack((np.cos(ang), np.sin(ang)), -1)).float().contiguous()


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


def magnitudes(bits):
    """The values of the codes without a sign, from the format's definition."""
    man, bias, n = (3, 7, 127) if bits == 8 else (1, 1, 8)
    out = []
    for c in range(n):
        e, m = c >> man, c & ((1 << man) - 1)
        out.append((m / 2 ** man if e == 0 else 1 + m / 2 ** man) * 2.0 ** (max(e, 1) - bias))
    return np.array(out)


MAG = {4: magnitudes(4), 8: magnitudes(8)}


def quantise(z, bits=8):
    """Codes (sign in the top bit of `bits`) and block exponents, decided value by value against the whole grid."""
    grid = MAG[bits]
    v = z.reshape(z.shape[:-1] + (z.shape[-1] // 32, 32))
    amax = np.maximum(np.abs(v).max(-1), 1e-4)
    k = np.array([next(e for e in range(-40, 130) if a <= grid[-1] * 2.0 ** e) for a in amax.ravel()], dtype=int).reshape(amax.shape)
    y = np.abs(v) / 2.0 ** k[..., None]
    up = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)     # the pair of neighbours around y
    below, above = y - grid[up - 1], grid[up] - y
    near = np.where((below < above) | ((below == above) & ((up - 1) % 2 == 0)), up - 1, up)
    code = near + (1 << (bits - 1)) * np.signbit(v)
    return code.reshape(z.shape).astype(np.uint8), k.astype(np.int8)


def values(code, k, bits=8):
    low = (1 << (bits - 1)) - 1
    mag = np.append(MAG[8], np.nan) if bits == 8 else MAG[4]
    v = mag[code & low] * np.where(code > low, -1.0, 1.0)
    return (v.reshape(k.shape + (32,)) * 2.0 ** k[..., None].astype(float)).reshape(v.shape)


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def seen(p, window, ring, ratio, base):
    """Logical rows that a query at position p sees."""
    rows = [i % ring if ring else i for i in range(max(0, p - window + 1) if window else 0, p + 1)]
    return rows + [base + j for j in range((p + 1) // ratio if ratio and p >= 0 else 0)]


def attention(q, rows, sink, scale):
    """q [h][d], rows [n][d] -> o, and its tolerance before a rotation (header comment)."""
    if not len(rows):
        return np.zeros_like(q), np.zeros_like(q)
    s = scale * q @ rows.T
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    with np.errstate(over="ignore"):
        den = p.sum(-1, keepdims=True) + np.exp(sink[:, None] - top)
    o, A = p @ rows / den, p @ np.abs(rows) / den
    S = abs(scale) * (np.abs(q) @ np.abs(rows).T).max(-1, keepdims=True)
    return o, 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13 * S) * A


def pair_sum(a, rd):
    out = a.copy()
    if rd:
        out[..., -rd::2] = out[..., -rd + 1::2] = a[..., -rd::2] + a[..., -rd + 1::2]
    return out


# ---- helpers on the GPU -----------------------------------------------------------------------------

@pytest.fixture(scope="module")
def ds():
    from sparse_latent_attention_attn_gb300 import dsattn
    dsattn.device_status()
    return dsattn


def dev(*ts):
    out = [t.cuda() if isinstance(t, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(t)).cuda() if t is not None else None
           for t in ts]
    return out[0] if len(out) == 1 else out


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def block_table(g, b, rows, page, spare=3):
    """(pages, table [b][max_pages]): pages in random order, some of them nobody's."""
    per = -(-rows // page) if rows else 1
    order = torch.randperm(b * per + spare, generator=g)[:b * per]
    return b * per + spare, order.view(b, per).to(torch.int32)


def slots(bt, seq, rows, page):
    rows = np.asarray(rows, dtype=np.int64)
    return bt[seq].numpy()[rows // page].astype(np.int64) * page + rows % page


# ---- append ---------------------------------------------------------------------------------------------

def append_reference(x, w, eps, rd, tab, first, lens, step, base, window, codes, exps, bt, page, y):
    b, s, d = x.shape
    for i in range(b):
        n = s if lens is None else min(int(lens[i]), s)
        for t in range(n):
            r = int(first[i]) + t
            z = normed(x[i, t], w, eps) if eps else x[i, t]
            z = rotate(z, tab[r * step]) if rd else z
            c, k = quantise(z)
            y[i, t] = values(c, k)
            if window == 0 or t >= n - window:
                at = slots(bt, i, [base + (r % window if window else r)], page)[0]
                codes.reshape(-1, d)[at] = c
                exps.reshape(-1, d // 32)[at] = k


APPENDS = [
    # b, s, d, rd, page, window, base, step, eps, weight, ragged
    (1, 1, 32, 0, 1, 0, 0, 1, 0.0, False, False),
    (5, 1, 512, 64, 16, 8, 0, 1, 1e-6, True, False),
    (3, 11, 512, 64, 7, 8, 3, 1, 1e-6, False, True),
    (2, 9, 512, 512, 64, 0, 5, 4, 0.0, False, False),
    (4, 6, 96, 40, 5, 0, 2, 2, 1e-3, True, True),
    (2, 5, 64, 8, 3, 4, 0, 1, 1e-6, True, False),
    (2, 3, 224, 224, 4, 2, 1, 3, 0.0, False, True),
    (1, 7, 1024, 128, 8, 0, 0, 1, 1e-6, True, False),
]


@gpu
@pytest.mark.parametrize("b,s,d,rd,page,window,base,step,eps,weight,ragged", APPENDS)
def test_append(ds, b, s, d, rd, page, window, base, step, eps, weight, ragged):
    g = torch.Generator().manual_seed(b * 100 + s + d)
    x = torch.randn((b, s, d + 16), generator=g).to(torch.bfloat16)
    x[0, 0, :32] *= 2.0 ** -14                                      # a block of next to nothing
    first = torch.randint(0, 40, (b,), generator=g, dtype=torch.int32)
    lens = torch.randint(0, s + 1, (b,), generator=g, dtype=torch.int32) if ragged else None
    w = 1 + 0.2 * torch.randn((d,), generator=g) if weight else None
    tab = table_of((40 + s) * step, rd) if rd else None
    pages, bt = block_table(g, b, base + (window or 40 + s), page)
    codes, exps = torch.full((pages, page, d), 77, dtype=torch.uint8), torch.full((pages, page, d // 32), 9, dtype=torch.int8)
    wc, wk, wy = codes.numpy().copy(), exps.numpy().copy(), np.full((b, s, d), 5.0)
    append_reference(f64(x)[..., :d], None if w is None else f64(w), eps, rd, None if tab is None else f64(tab), first, lens,
                     step, base, window, wc, wk, bt, page, wy)
    c, k, y = dev(codes, exps, torch.full((b, s, d), 5.0, dtype=torch.bfloat16))
    ds.kv_append_fp8_paged(dev(x)[..., :d], c, k, dev(bt), dev(first), rd=rd, table=dev(tab), eps=eps, weight=dev(w),
                           lens=dev(lens), pos_step=step, base=base, window=window, y=y)
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(k.cpu().numpy(), wk)
    assert np.array_equal(f64(y), wy)
    assert ds.device_status() == 0
    c2, k2 = dev(codes, exps)                                       # the same without y
    ds.kv_append_fp8_paged(dev(x)[..., :d], c2, k2, dev(bt), dev(first), rd=rd, table=dev(tab), eps=eps, weight=dev(w),
                           lens=dev(lens), pos_step=step, base=base, window=window)
    assert torch.equal(c, c2) and torch.equal(k, k2)


@gpu
def test_append_ties_scales_and_signs(ds):
    """Rows that are stored as they are: every code, every border between two codes, one bf16 step to either side of it,
    the scale's own borders, and zeros of both signs."""
    mag = MAG[8]
    mids = (mag[1:] + mag[:-1]) / 2
    v = np.concatenate([mag, mids, mids * (1 + 2.0 ** -7), mids * (1 - 2.0 ** -8)])
    v = np.concatenate([v, -v])
    rows = []
    for i in range(0, len(v), 30):
        part = np.zeros(32)
        part[:len(v[i:i + 30])] = v[i:i + 30]
        part[30], part[31] = 448.0, -0.0                            # the block's maximum: scale 1
        rows.append(part)
    rows = np.array(rows)
    edge = np.zeros((8, 32))
    edge[:, 0] = [448.0, 450.0, 224.0, 225.0, 1e-4, 448 * 2.0 ** -22, 449.5 * 2.0 ** -22, 0.0]
    rows = np.concatenate([rows, rows * 2.0 ** -9, rows * 2.0 ** 30, edge])
    x = torch.from_numpy(rows).to(torch.bfloat16).view(1, -1, 32)
    n = x.shape[1]
    wc, wk = quantise(f64(x)[0])
    c, k = dev(torch.zeros((n, 1, 32), dtype=torch.uint8), torch.zeros((n, 1, 1), dtype=torch.int8))
    bt = torch.arange(n, dtype=torch.int32).view(1, n)
    y = torch.empty((1, n, 32), dtype=torch.bfloat16, device="cuda")
    ds.kv_append_fp8_paged(dev(x), c, k, dev(bt), dev(ints(0)), y=y)
    assert np.array_equal(c.cpu().numpy()[:, 0], wc) and np.array_equal(k.cpu().numpy()[:, 0], wk)
    assert np.array_equal(f64(y)[0], values(wc, wk))
    assert torch.equal(torch.signbit(y.cpu()), torch.signbit(x))


@gpu
def test_append_is_the_round_trip_of_the_ring_write(ds):
    """The store's rows are those that ds_kv_quant_ring_write leaves behind, and ds_kv_quantize_fp8's codes."""
    g = torch.Generator().manual_seed(3)
    x = dev((torch.randn((2, 40, 512), generator=g) * 3).to(torch.bfloat16))
    pages, bt = block_table(g, 2, 40, 8)
    c = torch.zeros((pages, 8, 512), dtype=torch.uint8, device="cuda")
    k = torch.zeros((pages, 8, 16), dtype=torch.int8, device="cuda")
    ds.kv_append_fp8_paged(x, c, k, dev(bt), dev(ints(0, 0)))
    kv = x.clone()
    ds.kv_quant_ring_write(kv, None, 0, 1)
    assert torch.equal(ds.kv_read_fp8_paged(c, k, dev(bt), 40), kv)
    qc, qk = ds.kv_quantize_fp8(x)
    for i in range(2):
        at = dev(slots(bt, i, range(40), 8))
        assert torch.equal(c.view(-1, 512)[at], qc[i]) and torch.equal(k.view(-1, 16)[at], qk[i])


@gpu
def test_append_bad_pages_and_positions(ds):
    x = torch.ones((4, 2, 32), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((3, 2, 32), 7, dtype=torch.uint8, device="cuda")
    exps = torch.full((3, 2, 1), 5, dtype=torch.int8, device="cuda")
    bt = dev(torch.tensor([[0], [-1], [3], [2]], dtype=torch.int32))
    y = torch.zeros((4, 2, 32), dtype=torch.bfloat16, device="cuda")
    ds.kv_append_fp8_paged(x, codes, exps, bt, dev(ints(1, 0, 0, -1)), y=y)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    c = codes.cpu()
    one = 0x38 + 8 * 8                                              # 1 = 256 * 2^-8
    assert (c[0, 1] == one).all() and (c[0, 0] == 7).all()          # position 1; position 2 has no page
    assert (c[2, 0] == one).all() and (c[2, 1] == 7).all()          # position -1 is refused, position 0 stored
    assert (c[1] == 7).all() and exps.cpu()[1].eq(5).all()
    assert f64(y)[0].min() == 1 and f64(y)[3, 0].max() == 0 and f64(y)[3, 1].min() == 1


@gpu
@pytest.mark.parametrize("rd", [0, 8])
def test_append_of_the_largest_values(ds, rd):
    """Up to bf16's largest value: stored as 2^128 from 31 * 2^123 on (infinity in y)."""
    top = 31 * 2.0 ** 123
    below = 2.0 ** 127 * (1 + 118 / 128)
    x = torch.zeros((1, 2, 32), dtype=torch.bfloat16)
    x[0, 0, 3], x[0, 1, 3] = below, top
    tab = torch.zeros((2, max(rd, 2) // 2, 2))
    tab[..., 0] = 1.0
    c, k = dev(torch.zeros((1, 2, 32), dtype=torch.uint8), torch.zeros((1, 2, 1), dtype=torch.int8))
    y = torch.zeros((1, 2, 32), dtype=torch.bfloat16, device="cuda")
    ds.kv_append_fp8_paged(dev(x), c, k, dev(ints(0).view(1, 1)), dev(ints(0)), rd=rd, table=dev(tab) if rd else None, y=y)
    wc, wk = quantise(f64(x)[0])
    assert np.array_equal(c.cpu().numpy()[0], wc) and np.array_equal(k.cpu().numpy()[0], wk)
    assert f64(y)[0, 0, 3] == 15 * 2.0 ** 124 and f64(y)[0, 1, 3] == math.inf and wk.max() == 120


@gpu
@pytest.mark.parametrize("b,s,d,rd", [(7, 300, 512, 64), (3, 500, 1024, 1024), (40, 64, 128, 8)])
def test_append_many_rows(ds, b, s, d, rd):
    """Enough rows that some of them lie next to a border: equal to a 64-bit evaluation on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((b, s, d), generator=g, device="cuda").to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn((d,), generator=g, device="cuda")
    tab = dev(table_of(s, rd))
    c = torch.zeros((b, s, d), dtype=torch.uint8, device="cuda")
    k = torch.zeros((b, s, d // 32), dtype=torch.int8, device="cuda")
    bt = torch.arange(b, dtype=torch.int32, device="cuda").view(b, 1)
    ds.kv_append_fp8_paged(x, c, k, bt, torch.zeros(b, dtype=torch.int32, device="cuda"), rd=rd, table=tab, eps=1e-6, weight=w)
    z = x.double()
    z = z / ((z * z).mean(-1, keepdim=True) + float(np.float32(1e-6))).sqrt() * w.double()
    a, e, cs = z[..., -rd::2].clone(), z[..., -rd + 1::2].clone(), tab.double()
    z[..., -rd::2] = a * cs[..., 0] - e * cs[..., 1]
    z[..., -rd + 1::2] = a * cs[..., 1] + e * cs[..., 0]
    v = z.unflatten(-1, (-1, 32))
    kk = torch.full(v.shape[:-1], -30, device="cuda")
    for _ in range(40):
        kk = torch.where(v.abs().amax(-1) > 448 * ((kk.long() + 1023) << 52).view(torch.float64), kk + 1, kk)
    assert torch.equal(k.long(), kk)
    y = v.abs() * ((1023 - kk.long()) << 52).view(torch.float64)[..., None]
    grid = dev(MAG[8])
    up = torch.searchsorted(grid, y).clamp(1, 126)
    below, above = y - grid[up - 1], grid[up] - y
    near = torch.where((below < above) | ((below == above) & ((up - 1) % 2 == 0)), up - 1, up)
    assert torch.equal(c.long(), (near + 128 * torch.signbit(v)).flatten(-2))


# ---- read back --------------------------------------------------------------------------------------------

def reader(ds, bits):
    return ds.kv_read_fp8_paged if bits == 8 else ds.kv_read_fp4_paged


def random_store(g, bits, pages, page, d, kmin=-22, kmax=20):
    codes = torch.randint(0, 256, (pages, page, d * bits // 8), generator=g).to(torch.uint8)
    if bits == 8:
        codes[(codes & 127) == NAN8] = 0
    return codes, torch.randint(kmin, kmax + 1, (pages, page, d // 32), generator=g).to(torch.int8)


def plain_values(codes, exps, bits):
    c = codes.numpy()
    if bits == 4:
        c = np.stack((c & 15, c >> 4), -1).reshape(c.shape[:-1] + (-1,))
    return values(c, exps.numpy(), bits)


@gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("b,n,d,page,how,ragged", [
    (1, 1, 32, 1, "first", False), (3, 7, 512, 5, "first", False), (2, 150, 512, 64, "idx", True), (5, 33, 96, 3, "idx", False),
    (2, 64, 1024, 7, "first", True), (130, 9, 64, 16, "none", True), (9, 700, 224, 24, "idx", True)])
def test_read(ds, bits, b, n, d, page, how, ragged):
    g = torch.Generator().manual_seed(b + n + d)
    held = n + 10
    pages, bt = block_table(g, b, held, page)
    codes, exps = random_store(g, bits, pages, page, d)
    first = torch.randint(0, 11, (b,), generator=g, dtype=torch.int32) if how == "first" else None
    idx = torch.randint(-3, held, (b, n), generator=g, dtype=torch.int32) if how == "idx" else None
    lens = torch.randint(-1, n + 2, (b,), generator=g, dtype=torch.int32) if ragged else None
    all_rows = plain_values(codes, exps, bits).reshape(-1, d)
    want = np.full((b, n, d), 3.0)
    for i in range(b):
        for t in range(n if lens is None else max(0, min(n, int(lens[i])))):
            r = int(idx[i, t]) if idx is not None else t + (int(first[i]) if first is not None else 0)
            want[i, t] = all_rows[slots(bt, i, [r], page)[0]] if r >= 0 else 0
    y = torch.full((b, n, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got = reader(ds, bits)(dev(codes), dev(exps), dev(bt), n, first=dev(first), idx=dev(idx), lens=dev(lens), y=y)
    assert got is y and np.array_equal(f64(y), want) and ds.device_status() == 0
    new = reader(ds, bits)(dev(codes), dev(exps), dev(bt), n, first=dev(first), idx=dev(idx), lens=dev(lens))
    for i in range(b):
        m = n if lens is None else max(0, min(n, int(lens[i])))
        assert torch.equal(new[i, :m], y[i, :m]) and not new[i, m:].any()


@gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_read_every_code_at_every_exponent(ds, bits):
    per = 2 if bits == 4 else 1
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8).view(-1, 32 // per)       # blocks of 32 codes
    nb = codes.shape[0]
    codes = codes.repeat(256, 1).view(1, 256, -1).contiguous()                             # one row an exponent
    exps = torch.arange(-128, 128).to(torch.int8).view(1, 256, 1).expand(1, 256, nb).contiguous()
    y = reader(ds, bits)(dev(codes), dev(exps), dev(ints(0).view(1, 1)), 256)
    c = codes.numpy()
    c = np.stack((c & 15, c >> 4), -1).reshape(1, 256, -1) if bits == 4 else c
    with np.errstate(over="ignore"):
        want = torch.from_numpy(values(c, exps.numpy(), bits).astype(np.float32)).to(torch.bfloat16)   # exact in f32 up to 2^128
    assert torch.equal(torch.nan_to_num(y.cpu().float(), nan=-7.0), torch.nan_to_num(want.float(), nan=-7.0))
    assert torch.equal(torch.signbit(y.cpu())[~want.isnan()], torch.signbit(want)[~want.isnan()])


@gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_read_bad_rows(ds, bits):
    codes = torch.full((2, 2, 32 * bits // 8), 0x44 if bits == 4 else 0x38, dtype=torch.uint8, device="cuda")
    exps = torch.zeros((2, 2, 1), dtype=torch.int8, device="cuda")
    bt = dev(torch.tensor([[0, -1], [1, 2]], dtype=torch.int32))
    idx = dev(torch.tensor([[0, 1, 2, -1], [1, 3, 4, (1 << 31) - 1]], dtype=torch.int32))
    one = f64(reader(ds, bits)(codes, exps, bt, 1))[0, 0, 0]
    y = reader(ds, bits)(codes, exps, bt, 4, idx=idx)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX
    assert f64(y)[..., 0].tolist() == [[one, one, 0, 0], [one, 0, 0, 0]]
    assert ds.device_status() == 0
    reader(ds, bits)(codes, exps, bt, 4, idx=torch.full_like(idx, -5))           # nothing listed is nothing bad
    assert ds.device_status() == 0
    y = reader(ds, bits)(codes, exps, bt, 2, first=dev(ints(-1, 1)))
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX and f64(y)[..., 0].tolist() == [[0, one], [one, 0]]
    y = torch.full((2, 2, 32), 3.0, dtype=torch.bfloat16, device="cuda")          # a store without pages
    reader(ds, bits)(codes[:0], exps[:0], bt, 2, lens=dev(ints(0, 1)), y=y)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX and f64(y)[..., 0].tolist() == [[3, 3], [0, 3]]


# ---- the attention of a chunk -------------------------------------------------------------------------------

class Store:
    """A pool that holds garbage (NaN codes, the largest exponents) but for the rows that are put there."""

    def __init__(self, seed, b, rows, page, d=512, spare=3, garbage=True):
        self.g = torch.Generator().manual_seed(seed)
        self.b, self.page, self.d = b, page, d
        self.pages, self.bt = block_table(self.g, b, rows, page, spare)
        self.codes = torch.full((self.pages, page, d), NAN8 if garbage else 0, dtype=torch.uint8)
        self.exps = torch.full((self.pages, page, d // 32), 127 if garbage else 0, dtype=torch.int8)

    def put(self, seq, rows, v):
        c, k = quantise(np.asarray(v, dtype=float))
        at = torch.from_numpy(slots(self.bt, seq, rows, self.page))
        self.codes.view(-1, self.d)[at] = torch.from_numpy(c)
        self.exps.view(-1, self.d // 32)[at] = torch.from_numpy(k)

    def get(self, seq, rows):
        at = torch.from_numpy(slots(self.bt, seq, rows, self.page))
        return values(self.codes.view(-1, self.d)[at].numpy(), self.exps.view(-1, self.d // 32)[at].numpy())

    def on_gpu(self):
        return dev(self.codes), dev(self.exps), dev(self.bt)


def check(ds, st, q, first, sink, window, ring, ratio, base, lens=None, rd=0, tab=None, scale=512 ** -0.5, tokens=None,
          status=0, rows_of=None, **more):
    """One call against 64 bits, all tokens (or the listed (sequence, token) pairs)."""
    b, m, h, d = q.shape
    o = torch.full((b, m, h, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got = ds.chunk_attn_fp8_paged(dev(q), *st.on_gpu(), dev(first), dev(sink), scale, window, ring=ring, ratio=ratio, base=base,
                                  lens=dev(lens), rd=rd, table=dev(tab), o=o, **more)
    assert got is o
    assert ds.device_status() == status
    got, qq, sk = f64(o), f64(q), f64(sink)
    for i, t in tokens or [(i, t) for i in range(b) for t in range(m)]:
        if lens is not None and t >= int(lens[i]):
            assert (got[i, t] == 3.0).all()
            continue
        p = int(first[i]) + t
        rows = seen(p, window, ring, ratio, base)
        if rows_of:
            rows = rows_of(i, rows)
        want, tol = attention(qq[i, t], st.get(i, rows) if len(rows) else np.zeros((0, d)), sk, scale)
        if rd and 0 <= p < tab.shape[0]:
            want, tol = rotate(want, f64(tab)[p], True), pair_sum(tol, rd)
        off = np.abs(got[i, t] - want)
        assert (off <= tol + 2.0 ** -126).all(), (i, t, float((off - tol).max()), float(off.max()), np.argwhere(off > tol)[:4].tolist())
    return o


def filled(seed, b, m, h, window, ring, ratio, base, page, first, lens=None, qscale=1.0, spread=1.0):
    """A store with the rows that the step's queries see, q and sink."""
    last = int(first.max()) + m
    top = max(ring if ring else last, base + last // ratio if ratio else 0)
    st = Store(seed, b, top, page)
    for i in range(b):
        n = m if lens is None else min(m, int(lens[i]))
        rows = sorted({r for t in (range(n) if window else [n - 1]) if n for r in seen(int(first[i]) + t, window, ring, ratio, base)})
        if rows:
            v = torch.randn((len(rows), 512), generator=st.g).numpy() * np.exp(spread * torch.randn((len(rows), 1), generator=st.g).numpy())
            st.put(i, rows, v)
    q = (qscale * torch.randn((b, m, h, 512), generator=st.g)).to(torch.bfloat16)
    return st, q, torch.randn((h,), generator=st.g)


ATTNS = [
    # b, m, h, window, ring, ratio, base, contexts, page, rd, ragged
    (1, 1, 1, 1, 1, 0, 0, (0, 0), 1, 0, False),                  # one row, one query
    (1, 1, 16, 128, 128, 0, 0, (500, 500), 64, 64, False),       # a full ring
    (3, 1, 64, 128, 128, 4, 128, (0, 700), 16, 64, False),       # decode at positions of their own
    (2, 1, 128, 100, 130, 2, 140, (300, 900), 24, 512, False),
    (2, 5, 40, 57, 61, 3, 61, (0, 400), 24, 40, True),           # odd everywhere
    (1, 130, 3, 16, 200, 8, 200, (30, 60), 7, 8, False),         # tokens over several tiles of queries
    (1, 300, 1, 0, 0, 0, 0, (0, 0), 64, 64, False),              # a causal prompt from position 0
    (2, 37, 7, 0, 0, 0, 0, (0, 200), 5, 0, True),
    (1, 3, 128, 1, 3, 1, 3, (250, 250), 16, 64, False),          # a window of one, every position compressed
    (4, 2, 9, 128, 129, 4, 129, (0, 3), 64, 64, False),          # next to nothing seen
    (1, 64, 64, 128, 0, 4, 400, (0, 0), 64, 64, False),          # a prompt's first chunk, no ring
    (1, 1, 16, 128, 128, 4, 128, (9001, 9001), 64, 64, False),   # few queries, a long axis
    (1, 2, 128, 0, 0, 0, 0, (1500, 1500), 64, 64, False),
    (5, 1, 33, 300, 300, 0, 0, (0, 2000), 100, 64, True),
    (2, 65, 2, 127, 256, 16, 300, (100, 1000), 256, 64, True),
]


@gpu
@pytest.mark.parametrize("b,m,h,window,ring,ratio,base,ctx,page,rd,ragged", ATTNS)
def test_attention(ds, b, m, h, window, ring, ratio, base, ctx, page, rd, ragged):
    g = torch.Generator().manual_seed(b * 7 + m + h)
    first = torch.randint(ctx[0], ctx[1] + 1, (b,), generator=g, dtype=torch.int32)
    lens = torch.randint(0, m + 1, (b,), generator=g, dtype=torch.int32) if ragged else None
    st, q, sink = filled(m + h, b, m, h, window, ring, ratio, base, page, first, lens, spread=0.3)
    tab = table_of(ctx[1] + m, rd) if rd else None
    check(ds, st, q, first, sink, window, ring, ratio, base, lens, rd, tab)


@gpu
@pytest.mark.parametrize("n", [1, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 384, 385])
@pytest.mark.parametrize("h", [5, 64, 100])
def test_attention_lengths_around_a_tile(ds, n, h):
    """n rows seen, as a window alone, as compressed rows behind a window, and as positions."""
    first = ints(n - 1)
    st, q, sink = filled(n, 1, 1, h, n, n, 0, 0, 16, first)
    check(ds, st, q, first, sink, n, n, 0, 0)
    st, q, sink = filled(n, 1, 1, h, 3, 3, 2, 3, 16, ints(2 * n + 1))
    check(ds, st, q, ints(2 * n + 1), sink, 3, 3, 2, 3)
    st, q, sink = filled(n, 1, 2, h, 0, 0, 0, 0, 16, first)
    check(ds, st, q, first, sink, 0, 0, 0, 0)


@gpu
@pytest.mark.parametrize("h", [3, 64, 128])
@pytest.mark.parametrize("how", ["growing", "falling", "peak late", "flat", "one head"])
def test_attention_maximum_that_moves(ds, how, h):
    """Scores that climb by far more than a softmax's references allow without a change, tile after tile."""
    n, m = 700, 2
    st = Store(5, 1, n + m, 16)
    u = np.zeros(512)
    u[::2] = 1.0                                                     # q is a multiple of u: a row's score is u . row
    level = {"growing": np.linspace(-4, 4, n + m), "falling": np.linspace(4, -4, n + m), "flat": np.zeros(n + m),
             "peak late": np.where(np.arange(n + m) == n - 50, 4.0, -4.0), "one head": np.linspace(-4, 4, n + m)}[how]
    noise = torch.randn((n + m, 512), generator=st.g).numpy() * 0.05
    st.put(0, range(n + m), level[:, None] * u + noise)
    q = torch.ones((1, m, h, 512)) * torch.from_numpy(u).float()
    q = (q * (4.0 if how != "one head" else torch.where(torch.arange(h) == h - 1, 4.0, 0.01).view(1, 1, h, 1))).to(torch.bfloat16)
    sink = torch.linspace(-3, 3, h)
    # |score| up to 512 / 2 * 4 * 4 / 22.6 = 181, 261 octaves: over a range of 523
    check(ds, st, q, ints(n), sink, 0, 0, 0, 0)
    check(ds, st, -q, ints(n), sink, 0, 0, 0, 0)


@gpu
def test_attention_sinks(ds):
    first = ints(300, 20)
    st, q, sink = filled(3, 2, 3, 40, 64, 70, 4, 70, 16, first)
    for s in (-1e30, -math.inf, 300.0, 1e30, 0.0):
        check(ds, st, q, first, torch.full((40,), s), 64, 70, 4, 70)
    check(ds, st, q, first, torch.linspace(-200, 200, 40), 64, 70, 4, 70)


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.05, 3e-5, 0.5])
def test_attention_scales(ds, scale):
    first = ints(300, 20)
    st, q, sink = filled(3, 2, 3, 40, 64, 70, 4, 70, 16, first)
    check(ds, st, q, first, sink, 64, 70, 4, 70, scale=scale)


@gpu
@pytest.mark.parametrize("k", [100, 20, 8, 7, -30, -90])
def test_attention_exponents(ds, k):
    """Rows of large and of tiny values: q is scaled the other way, the scores stay."""
    first = ints(200)
    st, q, sink = filled(4, 1, 2, 20, 0, 0, 0, 0, 16, first)
    at = torch.from_numpy(slots(st.bt, 0, range(202), 16))
    e = st.exps.view(-1, 16)
    e[at] = (e[at].int() + k).to(torch.int8)
    check(ds, st, (q.float() * 2.0 ** -k).to(torch.bfloat16), first, sink, 0, 0, 0, 0)


@gpu
def test_attention_exponents_of_a_row_apart(ds):
    first = ints(150)
    st, q, sink = filled(4, 1, 2, 20, 0, 0, 0, 0, 16, first)
    at = torch.from_numpy(slots(st.bt, 0, range(152), 16))
    st.exps.view(-1, 16)[at] = torch.randint(-40, 6, (152, 16), generator=st.g).to(torch.int8)
    check(ds, st, q * 0.05, first, sink, 0, 0, 0, 0)


@gpu
def test_attention_rows_without_pages(ds):
    """Entries of the block table that are no page are skipped and flagged; a query left without rows gives zeros."""
    first = ints(200, 90, 40)
    st, q, sink = filled(6, 3, 2, 70, 64, 80, 4, 80, 16, first)
    st.bt[0, 1], st.bt[0, 7], st.bt[1, :] = -1, st.pages, -7
    st.bt[2, 6] = (1 << 31) - 1
    bad = {0: {1, 7}, 1: set(range(st.bt.shape[1])), 2: {6}}
    check(ds, st, q, first, sink, 64, 80, 4, 80, status=ds.DS_DEV_BAD_INDEX,
          rows_of=lambda i, rows: [r for r in rows if r // 16 not in bad[i]])
    # rows beyond the block table: positions without a ring, compressed rows
    st, q, sink = filled(6, 1, 2, 70, 0, 0, 0, 0, 16, ints(100))
    st.bt = st.bt[:, :5].contiguous()
    check(ds, st, q, ints(100), sink, 0, 0, 0, 0, status=ds.DS_DEV_BAD_INDEX, rows_of=lambda i, rows: [r for r in rows if r < 80])
    st, q, sink = filled(6, 1, 2, 70, 20, 32, 2, 32, 16, ints(100))
    st.bt = st.bt[:, :4].contiguous()
    check(ds, st, q, ints(100), sink, 20, 32, 2, 32, status=ds.DS_DEV_BAD_INDEX, rows_of=lambda i, rows: [r for r in rows if r < 64])


@gpu
def test_attention_store_without_pages(ds):
    q, o = torch.ones((2, 2, 3, 512), dtype=torch.bfloat16, device="cuda"), torch.full((2, 2, 3, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros((0, 16, 512), dtype=torch.uint8, device="cuda"), torch.zeros((0, 16, 16), dtype=torch.int8, device="cuda")
    for bt in (torch.zeros((2, 0), dtype=torch.int32, device="cuda"), torch.zeros((2, 3), dtype=torch.int32, device="cuda")):
        o.fill_(3.0)
        ds.chunk_attn_fp8_paged(q, *none, bt, dev(ints(4, 9)), torch.zeros(3, device="cuda"), 0.1, 0, lens=dev(ints(2, 1)), o=o)
        assert ds.device_status() == ds.DS_DEV_BAD_INDEX
        assert not o[0].any() and not o[1, 0].any() and (o[1, 1] == 3.0).all()


@gpu
def test_attention_positions_at_the_ends(ds):
    """Negative positions give zeros and are flagged; the last position of an int is one like any other."""
    first = ints(-2, 30)
    st, q, sink = filled(6, 2, 4, 10, 8, 16, 0, 0, 16, ints(0, 30))
    st.put(0, range(16), torch.randn((16, 512), generator=st.g).numpy())
    check(ds, st, q, first, sink, 8, 16, 0, 0, status=ds.DS_DEV_BAD_INDEX)
    last = (1 << 31) - 1
    st, q, sink = filled(6, 1, 1, 10, 8, 11, 0, 0, 16, ints(100))
    st.put(0, range(11), torch.randn((11, 512), generator=st.g).numpy())
    check(ds, st, q, ints(last), sink, 8, 11, 0, 0)
    # outside the rotation's table: unrotated and flagged
    st, q, sink = filled(6, 1, 3, 10, 8, 11, 0, 0, 16, ints(50))
    check(ds, st, q, ints(50), sink, 8, 11, 0, 0, rd=64, tab=table_of(51, 64), status=ds.DS_DEV_BAD_INDEX)


@gpu
@pytest.mark.parametrize("m,h", [(1, 20), (2, 128), (3, 128), (30, 24)])
def test_attention_last_positions_with_a_row_each(ds, m, h):
    """Positions around 2^31 with one compressed row a position, of which the table holds some: the quotient passes an int."""
    first, ring, base = ints((1 << 31) - 1), 40, 40
    st = Store(3, 1, 120, 16)
    cap = 16 * st.bt.shape[1]
    st.put(0, range(cap), torch.randn((cap, 512), generator=st.g).numpy())
    q, sink = torch.randn((1, m, h, 512), generator=st.g).to(torch.bfloat16), torch.randn((h,), generator=st.g)
    o = torch.empty((1, m, h, 512), dtype=torch.bfloat16, device="cuda")
    ds.chunk_attn_fp8_paged(dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, 8, ring=ring, ratio=1, base=base, o=o)
    assert ds.device_status() == ds.DS_DEV_BAD_INDEX                 # rows beyond the table
    for t in sorted({0, 1, m // 2, m - 1} & set(range(m))):
        p = int(first[0]) + t
        rows = [i % ring for i in range(p - 7, p + 1)] + list(range(base, cap))
        want, tol = attention(f64(q)[0, t], st.get(0, rows), f64(sink), 512 ** -0.5)
        assert (np.abs(f64(o)[0, t] - want) <= tol).all(), t


@gpu
@pytest.mark.parametrize("m,h", [(1, 20), (1, 128), (3, 128)])
def test_attention_compressed_rows_begin_beyond_the_table(ds, m, h):
    """A table that ends before the first compressed row's place: right as long as there is none, flagged from the first on."""
    st, q, sink = filled(6, 1, m, h, 20, 32, 0, 0, 16, ints(20))
    st.put(0, range(32), torch.randn((32, 512), generator=st.g).numpy())
    assert st.bt.shape[1] * 16 < 80
    check(ds, st, q, ints(20), sink, 20, 32, 64, 80)
    check(ds, st, q, ints(64), sink, 20, 32, 64, 80, status=ds.DS_DEV_BAD_INDEX, rows_of=lambda i, rows: [r for r in rows if r < 80])


@gpu
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_attention_of_queries_that_are_not_finite(ds, what):
    """A head of q with an infinity or a NaN touches no other head, and no other token."""
    first = ints(300)
    st, q, sink = filled(8, 1, 4, 33, 64, 70, 4, 70, 16, first)
    clean = f64(check(ds, st, q, first, sink, 64, 70, 4, 70))
    q[0, 1, 7, 100] = what
    got = ds.chunk_attn_fp8_paged(dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, 64, ring=70, ratio=4, base=70)
    other = np.ones((1, 4, 33), dtype=bool)
    other[0, 1, 7] = False
    assert np.array_equal(f64(got)[other], clean[other])
    assert ds.device_status() == 0


@gpu
def test_attention_in_a_large_pool(ds):
    """Slots whose byte offset passes 32 bits."""
    page, pages = 64, 140000                                       # 4.6 GB of codes
    codes = torch.full((pages, page, 512), NAN8, dtype=torch.uint8, device="cuda")
    exps = torch.full((pages, page, 16), 127, dtype=torch.int8, device="cuda")
    first = ints(900)
    st, q, sink = filled(9, 1, 1, 30, 128, 128, 4, 128, page, first)
    high = torch.arange(pages - st.bt.shape[1], pages, dtype=torch.int32).view(1, -1)
    for j, src in enumerate(st.bt[0].tolist()):
        codes[int(high[0, j])], exps[int(high[0, j])] = dev(st.codes[src]), dev(st.exps[src])
    a = ds.chunk_attn_fp8_paged(dev(q), codes, exps, dev(high), dev(first), dev(sink), 512 ** -0.5, 128, ring=128, ratio=4, base=128)
    b = check(ds, st, q, first, sink, 128, 128, 4, 128)
    assert torch.equal(a, b) and ds.device_status() == 0
    rows = ds.kv_read_fp8_paged(codes, exps, dev(high), 353)
    assert np.array_equal(f64(rows)[0], st.get(0, range(353)))
    x = torch.randn((1, 5, 512), device="cuda").to(torch.bfloat16)
    ds.kv_append_fp8_paged(x, codes, exps, dev(high), dev(ints(40)))
    y = x.clone()
    ds.kv_quant_ring_write(y, None, 0, 1)
    assert torch.equal(ds.kv_read_fp8_paged(codes, exps, dev(high), 5, first=dev(ints(40))), y)


@gpu
def test_attention_equals_listed_rows_read_back(ds):
    """The library's own path over the same rows: window rows listed by position, read back to bf16, ds_sparse_attn."""
    s, h, W = 200, 64, 128
    first = ints(0)
    st, q, sink = filled(11, 1, s, h, W, 0, 0, 0, 16, first, spread=0.2)
    o = check(ds, st, q, first, sink, W, 0, 0, 0, tokens=[(0, t) for t in (0, 1, 127, 128, 199)])
    c, k, bt = st.on_gpu()
    kv = ds.kv_read_fp8_paged(c, k, bt, s)
    idx = torch.empty((1, s, W), dtype=torch.int32, device="cuda")
    ds.window_topk_idxs(idx, 1, s, 0, W)
    ref = ds.sparse_attn(dev(q), kv, dev(sink), idx, 512 ** -0.5)
    # each is within the header comment's bound of the exact value, and A, a weighted mean of |v| with weights that add up to
    # less than 1, is at most the largest |v| of its column; S likewise at most sum |q| max |v|
    top = kv.abs().amax(1).double()[:, None, None]
    S = 512 ** -0.5 * (dev(q).abs().double() * top).sum(-1, keepdim=True)
    tol = 2 * (2.0 ** -8 * ref.double().abs() * (1 + 2.0 ** -6) + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13 * S) * top)
    assert ((o.double() - ref.double()).abs() <= tol).all()
    # the pool as an fp8 row store, entries as slots
    at = dev(torch.from_numpy(slots(st.bt, 0, range(s), 16)).to(torch.int32))
    phys = torch.where(idx >= 0, at[idx.clamp(min=0).long()], -1).contiguous()
    got = ds.sparse_attn_fp8kv(dev(q), c.view(1, -1, 512), k.view(1, -1, 16), dev(sink), phys, 512 ** -0.5)
    assert ((got.double() - ref.double()).abs() <= tol).all()
    assert ds.device_status() == 0


@gpu
def test_attention_calls_at_once_and_captured(ds):
    """Two streams at the same time, and two captured graphs replayed in turn, give what single calls give."""
    calls = []
    for seed, (b, m, h, window, ring, ratio, base) in enumerate([(3, 1, 16, 128, 128, 4, 128), (1, 40, 64, 64, 110, 2, 120)]):
        first = ints(*[900 + 7 * i for i in range(b)])
        st, q, sink = filled(seed, b, m, h, window, ring, ratio, base, 16, first)
        args = (dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, window)
        kw = dict(ring=ring, ratio=ratio, base=base)
        calls.append((args, kw, ds.chunk_attn_fp8_paged(*args, **kw)))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    outs = [torch.empty_like(c[2]) for c in calls]
    for _ in range(20):
        for s, (args, kw, _), o in zip(streams, calls, outs):
            o.zero_()
        torch.cuda.synchronize()
        for s, (args, kw, _), o in zip(streams, calls, outs):
            ds.chunk_attn_fp8_paged(*args, **kw, o=o, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(o, c[2]) for o, c in zip(outs, calls))
    graphs = []
    for (args, kw, _), o in zip(calls, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ds.chunk_attn_fp8_paged(*args, **kw, o=o)
        graphs.append(gr)
    for _ in range(3):
        for gr, o in zip(graphs, outs):
            o.zero_()
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, c[2]) for o, c in zip(outs, calls))
    assert ds.device_status() == 0


@gpu
def test_attention_captured_with_other_positions(ds):
    """A captured step replayed after its positions, lengths and rows changed."""
    from sparse_latent_attention_attn_gb300 import path
    b, s, h, W, ring, page = 3, 2, 20, 30, 40, 16
    g = torch.Generator().manual_seed(4)
    pages, bt = block_table(g, b, ring + 100, page)
    codes = torch.zeros((pages, page, 512), dtype=torch.uint8, device="cuda")
    exps = torch.zeros((pages, page, 16), dtype=torch.int8, device="cuda")
    past = dev(torch.randn((b, 300, 512), generator=g).to(torch.bfloat16))
    comp = dev(torch.randn((b, 100, 512), generator=g).to(torch.bfloat16))
    tab = dev(table_of(400, 64))
    zero = torch.zeros(b, dtype=torch.int32, device="cuda")
    ds.kv_append_fp8_paged(comp, codes, exps, dev(bt), zero, rd=64, table=tab, eps=1e-6, pos_step=4, base=ring)
    sink = torch.zeros(h, device="cuda")
    first, lens = torch.zeros(b, dtype=torch.int32, device="cuda"), torch.zeros(b, dtype=torch.int32, device="cuda")
    q = torch.zeros((b, s, h, 512), dtype=torch.bfloat16, device="cuda")
    new = torch.zeros((b, s, 512), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)

    def step(out):
        path.chunk_step_fp8_paged(q, new, codes, exps, table, first, sink, W, ring, 0.05, 64, tab, 1e-6,
                                  lens=lens, ratio=4, base=ring, o=out)

    table = dev(bt)
    step(o)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(o)
    pos = [5, 17, 0]
    for turn in range(6):
        n = [int(v) for v in torch.randint(0, s + 1, (b,), generator=g)]
        q.copy_(torch.randn(q.shape, generator=g))
        for i in range(b):
            new[i, :] = past[i, pos[i]:pos[i] + s]
        first.copy_(ints(*pos))
        lens.copy_(ints(*n))
        o.zero_()
        gr.replay()
        want = torch.zeros_like(o)
        step(want)
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        pos = [p + k for p, k in zip(pos, n)]
    assert ds.device_status() == 0


@gpu
def test_attention_workspace_refused(ds):
    first = ints(9001)
    need = ds.chunk_attn_fp8_paged_workspace_bytes(1, 1, 16, 512, 128, 4, 64, 50)
    if need == 0:
        pytest.skip("the shape needs no workspace")
    st, q, sink = filled(1, 1, 1, 16, 128, 128, 4, 128, 64, first)
    need = ds.chunk_attn_fp8_paged_workspace_bytes(1, 1, 16, 512, 128, 4, 64, st.bt.shape[1])
    args = (dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, 128)
    o = torch.full((1, 1, 16, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"), torch.empty(need + 256, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(ds.DsError) as e:
            ds.chunk_attn_fp8_paged(*args, ring=128, ratio=4, base=128, o=o, workspace=ws)
        assert e.value.status == ds.DS_EWORKSPACE
    torch.cuda.synchronize()
    assert (o == 3.0).all()
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")       # whatever it holds, and nothing beyond it
    check(ds, st, q, first, sink, 128, 128, 4, 128, workspace=ws[:need])
    assert (ws[need:] == 255).all()


@gpu
def test_attention_is_the_same_every_time(ds):
    first = ints(700, 300, 900)
    st, q, sink = filled(2, 3, 20, 64, 128, 150, 4, 150, 16, first)
    args = (dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, 128)
    ref = ds.chunk_attn_fp8_paged(*args, ring=150, ratio=4, base=150)
    for _ in range(50):
        assert torch.equal(ds.chunk_attn_fp8_paged(*args, ring=150, ratio=4, base=150), ref)


# One tile of queries a sequence (its rows are widened in the kernel), several (widened once, before), and either in parts of a
# long axis: b, m, h, window, ring, ratio, base, context.
FORMS = {"one tile": (3, 1, 64, 128, 128, 4, 128, 700), "parts": (1, 1, 16, 128, 128, 4, 128, 9001),
         "several tiles": (2, 40, 64, 64, 110, 2, 120, 500), "several tiles in parts": (1, 3, 128, 0, 0, 0, 0, 3000)}


def of_form(name, seed=1, **more):
    b, m, h, window, ring, ratio, base, ctx = FORMS[name]
    first = ints(*[ctx - 97 * i for i in range(b)])
    return (*filled(seed, b, m, h, window, ring, ratio, base, 16, first, **more), first, (window, ring, ratio, base))


def some_tokens(q, n=7):
    b, m = q.shape[:2]
    every = [(i, t) for i in range(b) for t in range(m)]
    return every[::-(-len(every) // n)]


@gpu
@pytest.mark.parametrize("form", FORMS)
def test_attention_wait_that_runs_out(ds, form):
    """With the hook on, the first tile's rows are withheld: the call ends, says so, and the next is clean."""
    st, q, sink, first, how = of_form(form)
    args = (dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, how[0])
    assert ds.device_status() == 0
    ds.test_set_stall(True)
    try:
        ds.chunk_attn_fp8_paged(*args, ring=how[1], ratio=how[2], base=how[3])
        bits = ds.device_status()
    finally:
        ds.test_set_stall(False)
    assert bits == ds.DS_DEV_TIMEOUT
    check(ds, st, q, first, sink, *how, tokens=some_tokens(q))


@gpu
@pytest.mark.parametrize("form", FORMS)
def test_attention_sink_that_is_nan(ds, form):
    """As in ds_sparse_attn: NaN for its head, nothing for the others; a query that sees no row gives zeros all the same."""
    st, q, sink, first, how = of_form(form, seed=4)
    clean = check(ds, st, q, first, sink, *how, tokens=some_tokens(q, 3))
    sink[5] = math.nan
    args = (dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, how[0])
    got = ds.chunk_attn_fp8_paged(*args, ring=how[1], ratio=how[2], base=how[3])
    assert got[:, :, 5].isnan().all() and ds.device_status() == 0
    got[:, :, 5] = clean[:, :, 5]
    assert torch.equal(got, clean)
    got = ds.chunk_attn_fp8_paged(*args[:3], torch.full_like(args[3], -1), *args[4:], ring=how[1], ratio=how[2], base=how[3])
    assert not got.any() and ds.device_status() == ds.DS_DEV_BAD_INDEX


@gpu
@pytest.mark.parametrize("form", FORMS)
def test_attention_workspace_ends(ds, form):
    """Whatever the workspace holds, and nothing beyond it."""
    st, q, sink, first, how = of_form(form, seed=3)
    need = ds.chunk_attn_fp8_paged_workspace_bytes(*q.shape, how[0], how[2], 16, st.bt.shape[1])
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    check(ds, st, q, first, sink, *how, tokens=some_tokens(q), workspace=ws[:need])
    assert (ws[need:] == 255).all()


@gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_attention_forms_at_scales(ds, form, scale):
    st, q, sink, first, how = of_form(form, seed=5)
    check(ds, st, q, first, sink, *how, scale=scale, tokens=some_tokens(q))


@gpu
@pytest.mark.parametrize("form", FORMS)
def test_attention_forms_are_the_same_every_time(ds, form):
    st, q, sink, first, how = of_form(form, seed=6)
    args = (dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, how[0])
    ref = ds.chunk_attn_fp8_paged(*args, ring=how[1], ratio=how[2], base=how[3])
    for _ in range(30):
        assert torch.equal(ds.chunk_attn_fp8_paged(*args, ring=how[1], ratio=how[2], base=how[3]), ref)


@gpu
@pytest.mark.parametrize("m,h", [(2, 60), (1, 20), (30, 24)])
def test_attention_forms_without_pages(ds, m, h):
    """As in the test of rows without pages, with a tile of queries or several of them."""
    first = ints(200, 90, 40)
    st, q, sink = filled(6, 3, m, h, 64, 100, 4, 100, 16, first)
    st.bt[0, 1], st.bt[0, 8], st.bt[1, :] = -1, st.pages, -7
    bad = {0: {1, 8}, 1: set(range(st.bt.shape[1])), 2: set()}
    check(ds, st, q, first, sink, 64, 100, 4, 100, status=ds.DS_DEV_BAD_INDEX, tokens=[(i, t) for i in range(3) for t in {0, m // 2, m - 1}],
          rows_of=lambda i, rows: [r for r in rows if r // 16 not in bad[i]])


@gpu
@pytest.mark.parametrize("m,h", [(1, 20), (1, 128), (12, 20), (4, 100)])
@pytest.mark.parametrize("k", [110, 8, -40])
def test_attention_forms_at_exponents(ds, m, h, k):
    """Rows of large and of tiny values beside each other (q is scaled the other way), and a block of zeros by its exponent."""
    first = ints(300)
    st, q, sink = filled(4, 1, m, h, 0, 0, 0, 0, 16, first)
    at = torch.from_numpy(slots(st.bt, 0, range(300 + m), 16))
    e = st.exps.view(-1, 16)
    e[at] = (e[at].int() + k - torch.randint(0, 9, (300 + m, 16), generator=st.g)).to(torch.int8)
    e[at[::5], 3] = -128                                 # counts as zeros: 448 * 2^-128 is nothing beside the others
    check(ds, st, (q.float() * 2.0 ** -k).to(torch.bfloat16), first, sink, 0, 0, 0, 0, tokens=some_tokens(q, 4))


@gpu
@pytest.mark.parametrize("m,h", [(1, 16), (1, 128), (3, 128)])
def test_attention_maximum_that_moves_in_parts(ds, m, h):
    """A long axis of climbing, falling and flat scores: parts of a unit with references of their own."""
    n = 4000
    u = np.zeros(512)
    u[::2] = 1.0
    q = torch.from_numpy(np.broadcast_to(u * 4, (1, m, h, 512)).copy()).to(torch.bfloat16)
    sink = torch.linspace(-3, 3, h)
    for level in (np.linspace(-4, 4, n + m), np.linspace(4, -4, n + m), np.where(np.arange(n + m) == n // 3, 4.0, -4.0)):
        st = Store(5, 1, n + m, 64)
        st.put(0, range(n + m), level[:, None] * u + torch.randn((n + m, 512), generator=st.g).numpy() * 0.05)
        check(ds, st, q, ints(n), sink, 0, 0, 0, 0)


@gpu
@pytest.mark.parametrize("b,m", [(40, 1), (20, 1), (13, 3), (7, 3)])
@pytest.mark.parametrize("order", [(0, 2, 1, 3), (2, 0, 3, 1), (0, 1, 2, 3), (3, 1, 0, 2)])
def test_attention_maxima_that_move_in_turn(ds, b, m, order):
    """Heads in four blocks of 32 (two blocks a CTA, a warp's queries each), and every second tile one block's maximum jumps: a
    block's O^T is lowered at one tile, another block's at the tile where the first one's factors are set back.  Rows read by one tile
    of queries and by several, units whole and in parts."""
    n, h, page = 30 * 128, 128, 64
    block = torch.arange(h) // 32                        # block i: values i, i + 4, ... of a row
    st = Store(8, 1, n + m, page)
    v = torch.randn((n + m, 512), generator=st.g).numpy() * 0.05
    v -= 4
    for j, t in enumerate(range(1, 30, 2)):              # a step of 1 moves a score by 128 * 4 / 512^0.5 = 22.6, 32 octaves
        v[128 * t + 9 * j, order[j % 4]::4] += 1 + j // 4
    st.put(0, range(n + m), v)
    st.bt = st.bt.expand(b, -1).contiguous()             # every sequence has the same rows
    on = (torch.arange(512) % 4 == block[:, None]).float() * 4
    q = (on + 0.01 * torch.randn((b, m, h, 512), generator=st.g)).to(torch.bfloat16)
    first = torch.full((b,), n, dtype=torch.int32)
    o = check(ds, st, q, first, torch.linspace(-3, 3, h), 0, 0, 0, 0, tokens=some_tokens(q, 5))
    for _ in range(20):
        assert torch.equal(o, ds.chunk_attn_fp8_paged(dev(q), *st.on_gpu(), dev(first), dev(torch.linspace(-3, 3, h)), 512 ** -0.5, 0))


@gpu
@pytest.mark.parametrize("m,h", [(1, 20), (5, 128), (40, 24)])
def test_attention_window_beyond_the_table(ds, m, h):
    """A window wider than the table has rows is one over all positions, in the workspace too."""
    first = ints(300, 77)
    st, q, sink = filled(12, 2, m, h, 0, 0, 0, 0, 16, first)
    o = check(ds, st, q, first, sink, 0, 0, 0, 0, tokens=some_tokens(q, 6))
    for window in (16 * st.bt.shape[1], 1 << 20, (1 << 31) - 1):
        assert (ds.chunk_attn_fp8_paged_workspace_bytes(2, m, h, 512, window, 0, 16, st.bt.shape[1])
                == ds.chunk_attn_fp8_paged_workspace_bytes(2, m, h, 512, 0, 0, 16, st.bt.shape[1]))
        assert torch.equal(o, ds.chunk_attn_fp8_paged(dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, window))
    assert ds.device_status() == 0


@gpu
@pytest.mark.parametrize("window,ring,m", [(30, 64, 200), (30, 64, 40), (1, 16, 300)])
def test_attention_padded_longer_than_the_table(ds, window, ring, m):
    """Padded chunks with more tokens than the ring, or the table, has rows: what lens says is there is right.  A sequence that its
    ring does not hold, which lens tells on the device only, sees what lies in the slots of its positions."""
    b, h = 2, 9
    st = Store(2, b, ring, 16)
    for i in range(b):
        st.put(i, range(ring), torch.randn((ring, 512), generator=st.g).numpy())
    q, sink, first = torch.randn((b, m, h, 512), generator=st.g).to(torch.bfloat16), torch.randn((h,), generator=st.g), ints(100, 3)
    fits = ring - window + 1
    for lens in (ints(fits, 2), ints(m, fits)):
        check(ds, st, q, first, sink, window, ring, 0, 0, lens=lens, tokens=some_tokens(q, 30))


@gpu
@pytest.mark.parametrize("b,m,h,window,ratio", [(1, 12, 60, 0, 0), (2, 304, 128, 40, 4), (1, 700, 3, 0, 0), (3, 9, 128, 64, 2),
                                                (2, 40, 128, 0, 0)])
def test_attention_of_a_table_too_wide_to_widen(ds, b, m, h, window, ratio):
    """Tables of 2^21 rows, next to all of them without a page: several tiles of queries a sequence, whose rows, had they to be
    widened for the whole table, would pass the workspace's 2 GB, and are widened by each unit; in parts and whole."""
    page, first = 256, ints(*[430 - 60 * i for i in range(b)])
    base = (500 + m) // page * page + page if ratio else 0
    st, q, sink = filled(14, b, m, h, window, 0, ratio, base, page, first)
    st.bt = torch.cat((st.bt, torch.full((b, 8192 - st.bt.shape[1]), -1, dtype=torch.int32)), dim=1)
    assert ds.chunk_attn_fp8_paged_workspace_bytes(b, m, h, 512, window, ratio, page, 8192) < 1 << 31
    check(ds, st, q, first, sink, window, 0, ratio, base, rd=64, tab=table_of(440 + m, 64), tokens=some_tokens(q, 9))
    lens = ints(*[max(1, m - 3 * i) for i in range(b)])
    check(ds, st, q, first, sink, window, 0, ratio, base, lens=lens, tokens=some_tokens(q, 5))


@gpu
@pytest.mark.parametrize("b,m,h,ctx,ragged", [(80, 1, 128, 1300, False), (90, 1, 70, 1300, True), (7, 12, 128, 1400, False),
                                              (5, 40, 60, 1500, True)])
def test_attention_of_many_sequences(ds, b, m, h, ctx, ragged):
    """A little more work than the GPU does at once: whole units, and the last ones in parts."""
    g = torch.Generator().manual_seed(b)
    first = torch.randint(ctx - 200, ctx + 1, (b,), generator=g, dtype=torch.int32)
    lens = torch.randint(0, m + 1, (b,), generator=g, dtype=torch.int32) if ragged else None
    page, top = 64, ctx + m
    st = Store(b, b, top, page, garbage=False)
    v = torch.randn((top, 512), generator=g).numpy()
    for i in range(b):
        st.put(i, range(int(first[i]) + m), np.roll(v, 31 * i, 0)[:int(first[i]) + m])
    q = torch.randn((b, m, h, 512), generator=g).to(torch.bfloat16)
    tokens = [(i, t) for i in range(0, b, max(1, b // 12)) for t in sorted({0, m // 2, m - 1})]
    check(ds, st, q, first, torch.zeros(h), 0, 0, 0, 0, lens, 64, table_of(top, 64), tokens=tokens)


@gpu
@pytest.mark.parametrize("b,m,h", [(126, 93, 2), (2, 700, 100), (400, 1, 2), (300, 1, 128), (90, 5, 23)])
def test_attention_of_one_row_a_query(ds, b, m, h):
    """Units of a single tile, one behind the other: their factors must not meet."""
    first = torch.arange(b, dtype=torch.int32) % 11
    st, q, sink = filled(2, b, m, h, 1, m, 0, 0, 64, first)
    args = (dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, 1)
    o = check(ds, st, q, first, sink, 1, m, 0, 0)
    for _ in range(20):
        assert torch.equal(ds.chunk_attn_fp8_paged(*args, ring=m), o)


@gpu
@pytest.mark.parametrize("b,m,h", [(126, 93, 2), (2, 700, 100), (300, 1, 128), (90, 5, 23)])
def test_attention_of_one_row_a_query_under_sinks(ds, b, m, h):
    """Units of a single tile whose factors lie decades apart, from head to head and from unit to unit: one unit's factors are
    written only when both CTAs have read those of two units ago."""
    first = torch.arange(b, dtype=torch.int32) % 11
    st, q, _ = filled(5, b, m, h, 1, m, 0, 0, 64, first)
    sink = 12.0 * torch.randn((h,), generator=st.g)
    q = (q.float() * torch.linspace(0.1, 2.0, b * m).view(b, m, 1, 1)).to(torch.bfloat16)
    o = check(ds, st, q, first, sink, 1, m, 0, 0, tokens=some_tokens(q, 60))
    for _ in range(20):
        assert torch.equal(ds.chunk_attn_fp8_paged(dev(q), *st.on_gpu(), dev(first), dev(sink), 512 ** -0.5, 1, ring=m), o)


@gpu
@pytest.mark.parametrize("how", [dict(window=64, ring=70, ratio=4, base=70), dict(window=0, ring=0, ratio=0, base=0)])
def test_attention_padding_and_empty_sequences(ds, how):
    """lens of 0, of more than m and below 0; tokens behind a sequence's last are left as they were."""
    for m, h in ((3, 40), (7, 40)):
        first = ints(300, 5, 0, 90)
        st, q, sink = filled(7, 4, m, h, page=16, first=first, **how)
        for lens in (ints(0, 0, 0, 0), ints(-3, 1, m + 5, 0), ints(2, m, 1, m - 1)):
            check(ds, st, q, first, sink, how["window"], how["ring"], how["ratio"], how["base"], lens)


# ---- a run of them together -------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("ragged", [False, True])
def test_prompt_in_chunks_then_decode(ds, ragged):
    """Prompts appended and attended to in chunks behind one another, with the compressed rows of each, then
    decode steps; every token against 64 bits from the raw rows, and the cache read back at the end."""
    from sparse_latent_attention_attn_gb300 import path
    b, h, W, ratio, rd, page, eps = 2, 12, 20, 4, 64, 16, 1e-6
    chunks = [9, 7, 16, 1, 1, 1]
    total, ring = 40, W + 16 - 1
    base = ring
    g = torch.Generator().manual_seed(21)
    pages, bt = block_table(g, b, base + total // ratio + 1, page)
    codes = torch.full((pages, page, 512), NAN8, dtype=torch.uint8, device="cuda")
    exps = torch.full((pages, page, 16), 127, dtype=torch.int8, device="cuda")
    raw = torch.randn((b, total, 512), generator=g).to(torch.bfloat16)
    comp = torch.randn((b, total // ratio, 512), generator=g).to(torch.bfloat16)
    q = torch.randn((b, total, h, 512), generator=g).to(torch.bfloat16)
    w = 1 + 0.1 * torch.randn((512,), generator=g)
    sink = torch.randn((h,), generator=g)
    tab = table_of(total, rd)
    t64, scale = f64(tab), 512 ** -0.5

    def stored(x, pos):
        return values(*quantise(rotate(normed(f64(x), f64(w), float(np.float32(eps))), t64[pos])))

    pos = [0, 0]
    table, dtab, dw, dsink = dev(bt), dev(tab), dev(w), dev(sink)
    for n in chunks:
        take = [n if not ragged or i == 0 else max(1, n - 3) for i in range(b)]
        x = torch.zeros((b, n, 512), dtype=torch.bfloat16)
        qq = torch.full((b, n, h, 512), math.nan, dtype=torch.bfloat16)
        new = [list(range(p // ratio, (p + k) // ratio)) for p, k in zip(pos, take)]
        xc = torch.zeros((b, max(1, max(len(v) for v in new)), 512), dtype=torch.bfloat16)
        for i in range(b):
            x[i, :take[i]], qq[i, :take[i]] = raw[i, pos[i]:pos[i] + take[i]], q[i, pos[i]:pos[i] + take[i]]
            xc[i, :len(new[i])] = comp[i, new[i]]
        first, lens = dev(ints(*pos)), dev(ints(*take)) if ragged else None
        ds.kv_append_fp8_paged(dev(xc), codes, exps, table, dev(ints(*[p // ratio for p in pos])), rd=rd, table=dtab, eps=eps,
                               weight=dw, lens=dev(ints(*[len(v) for v in new])), pos_step=ratio, base=base)
        o = path.chunk_step_fp8_paged(dev(qq), dev(x), codes, exps, table, first, dsink, W, ring, scale, rd, dtab, eps,
                                      kv_weight=dw, lens=lens, ratio=ratio, base=base)
        assert ds.device_status() == 0
        got = f64(o)
        for i in range(b):
            assert not o[i, take[i]:].any()
            for t in range(take[i]):
                p = pos[i] + t
                lo, nc = max(0, p - W + 1), (p + 1) // ratio
                rows = np.concatenate([stored(raw[i, lo:p + 1], range(lo, p + 1)),
                                       stored(comp[i, :nc], [j * ratio for j in range(nc)])])
                qz = rotate(normed(f64(q[i, p]), None, float(np.float32(eps))), t64[p])
                want, tol = attention(qz, rows, f64(sink), scale)
                # q was rounded to bf16 in between: each score off by at most 2^-8 of S, and l and p with it
                S = scale * (np.abs(qz) @ np.abs(rows).T).max(-1, keepdims=True)
                s = scale * qz @ rows.T
                pr = np.exp(s - s.max(-1, keepdims=True))
                A = pr @ np.abs(rows) / (pr.sum(-1, keepdims=True) + np.exp(f64(sink)[:, None] - s.max(-1, keepdims=True)))
                tol = pair_sum(tol + 2 * (np.exp(2.0 ** -8 * S) - 1) * A, rd)
                assert (np.abs(got[i, t] - rotate(want, t64[p], True)) <= tol).all(), (n, i, t)
        pos = [p + k for p, k in zip(pos, take)]
    for i in range(b):                                              # what the store holds now
        kept = list(range(pos[i] - W, pos[i]))
        y = ds.kv_read_fp8_paged(codes, exps, table[i:i + 1], W, idx=dev(ints(*[p % ring for p in kept]).view(1, -1)))
        assert np.array_equal(f64(y)[0], stored(raw[i, kept], kept))


# ---- refusals, no GPU needed ---------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    from sparse_latent_attention_attn_gb300 import build
    build.build()
    from sparse_latent_attention_attn_gb300 import dsattn
    return dsattn._lib


FAKE = 4096   # never dereferenced: every call below fails its checks first


def call(fn, base, /, **change):
    return fn(*{**base, **change}.values())


def test_append_refusals(lib):
    base = dict(x=FAKE, xb=64, xt=64, y=None, b=2, s=1, d=64, w=None, eps=1e-6, rd=16, table=FAKE, rows=10, first=FAKE,
                lens=None, step=1, base=0, window=8, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, stream=None)
    f = lib.ds_kv_append_fp8_paged
    for bad in (dict(b=-1), dict(s=-1), dict(d=0), dict(d=48), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=2.0 ** -101),
                dict(step=0), dict(base=-1), dict(window=-1), dict(rd=12), dict(rd=72), dict(table=None), dict(table=FAKE + 4),
                dict(pages=-1), dict(page=0), dict(mp=-1), dict(x=None), dict(x=FAKE + 8), dict(y=FAKE + 8),
                dict(first=None), dict(lens=FAKE + 2), dict(w=FAKE + 2), dict(codes=None), dict(codes=FAKE + 4),
                dict(exps=None), dict(bt=None), dict(bt=FAKE + 2), dict(xb=60), dict(xb=56), dict(s=2, xb=128, xt=56)):
        assert call(f, base, **bad) == -1, bad
    for bad in (dict(d=1056, xb=1056, xt=1056), dict(pages=1 << 27), dict(b=1 << 16, s=1 << 16)):
        assert call(f, base, **bad) == -2, bad
    assert call(f, base, b=0, x=None, codes=None, exps=None, bt=None, first=None) == 0


@pytest.mark.parametrize("name", ["ds_kv_read_fp8_paged", "ds_kv_read_fp4_paged"])
def test_read_refusals(lib, name):
    base = dict(codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=1, idx=None, first=None, lens=None, y=FAKE, b=2, n=3,
                d=64, stream=None)
    f = getattr(lib, name)
    for bad in (dict(b=-1), dict(n=-1), dict(d=0), dict(d=48), dict(pages=-1), dict(page=0), dict(mp=-1), dict(y=None),
                dict(y=FAKE + 8), dict(idx=FAKE + 2), dict(first=FAKE + 1), dict(lens=FAKE + 2), dict(codes=None),
                dict(codes=FAKE + 8), dict(exps=None), dict(bt=None), dict(bt=FAKE + 2)):
        assert call(f, base, **bad) == -1, bad
    for bad in (dict(d=1056), dict(pages=1 << 27), dict(b=1 << 16, n=1 << 16)):
        assert call(f, base, **bad) == -2, bad
    assert call(f, base, b=0, y=None, codes=None, exps=None, bt=None) == 0
    assert call(f, base, n=0, y=None, codes=None, exps=None, bt=None) == 0


def test_attention_refusals(lib):
    base = dict(q=FAKE, codes=FAKE, exps=FAKE, pages=4, page=16, bt=FAKE, mp=20, sink=FAKE, scale=0.1, o=FAKE, b=1, m=3, h=4,
                d=512, first=FAKE, lens=None, window=128, ring=130, ratio=4, base=130, ws=None, wsb=0, rd=0, table=None, rows=0,
                stream=None)
    f = lib.ds_chunk_attn_fp8_paged
    rot = dict(rd=16, table=FAKE, rows=9)
    for bad in (dict(b=-1), dict(m=-1), dict(h=0), dict(pages=-1), dict(page=0), dict(mp=-1), dict(window=-1), dict(ring=-1),
                dict(ratio=-1), dict(base=-1), dict(q=None), dict(q=FAKE + 8), dict(o=None), dict(o=FAKE + 8), dict(sink=None),
                dict(sink=FAKE + 2), dict(first=None), dict(first=FAKE + 2), dict(lens=FAKE + 2), dict(codes=None),
                dict(codes=FAKE + 8), dict(exps=None), dict(exps=FAKE + 8), dict(bt=None), dict(bt=FAKE + 1),
                {**rot, "rd": 12}, {**rot, "rd": 520}, {**rot, "table": None}, {**rot, "table": FAKE + 4}, {**rot, "rows": -1},
                dict(window=0), dict(ring=127), dict(ring=129), dict(m=4), dict(ring=129, m=3), dict(mp=8), dict(base=129),
                dict(ring=127, lens=FAKE)):
        assert call(f, base, **bad) == -1, bad
    for bad in (dict(d=256), dict(h=129), dict(pages=1 << 27), dict(b=1 << 15, m=1 << 15, window=0, ring=0),
                dict(ring=(1 << 29) + 1, base=1 << 30, mp=1 << 26)):
        assert call(f, base, **bad) == -2, bad
    assert call(f, base, ws=FAKE + 16, wsb=1 << 30) == -3
    assert call(f, base, b=0, q=None, o=None, sink=None, first=None) == 0
    w = lib.ds_chunk_attn_fp8_paged_workspace_bytes
    assert w(1, 1, 4, 256, 8, 0, 16, 4) == 0 and w(1, 1, 129, 512, 8, 0, 16, 4) == 0 and w(-1, 1, 4, 512, 8, 0, 16, 4) == 0
    assert w(1 << 15, 1 << 15, 4, 512, 8, 0, 16, 4) == 0 and w(1, 1, 4, 512, -1, 0, 16, 4) == 0


def test_bindings_refuse_cpu_tensors_and_shapes(lib):
    from sparse_latent_attention_attn_gb300 import dsattn, path
    codes, exps, bt = torch.zeros((1, 1, 64), dtype=torch.uint8), torch.zeros((1, 1, 2), dtype=torch.int8), ints(0).view(1, 1)
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dsattn.kv_append_fp8_paged(x, codes, exps, bt, ints(0))
    with pytest.raises(ValueError, match="x must be"):
        dsattn.kv_append_fp8_paged(x[0], codes, exps, bt, ints(0))
    for read in (dsattn.kv_read_fp8_paged, dsattn.kv_read_fp4_paged):
        with pytest.raises(ValueError, match="CUDA"):
            read(codes, exps, bt, 1)
        with pytest.raises(ValueError, match="codes must be"):
            read(codes[0], exps, bt, 1)
    q = torch.zeros((1, 3, 2, 512), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dsattn.chunk_attn_fp8_paged(q, torch.zeros((1, 1, 512), dtype=torch.uint8), torch.zeros((1, 1, 16), dtype=torch.int8), bt,
                                    ints(0), torch.zeros(2), 0.1, 8)
    with pytest.raises(ValueError, match="does not hold"):
        path.chunk_step_fp8_paged(q, torch.zeros((1, 3, 512), dtype=torch.bfloat16), codes, exps, bt, ints(0), torch.zeros(2), 8,
                                  9, 0.1, 0, None, 1e-6)


LAYOUTS = [dict(window=0, ring=8), dict(window=9, ring=8, lens=True), dict(window=8, ring=9), dict(window=30, ring=50),
           dict(window=8, ring=16, ratio=4, base=15)]


def layout_step(path, how, on):
    """A step whose ring and rows do not fit together; the store must be as it was."""
    q, x = torch.ones((1, 3, 2, 512), dtype=torch.bfloat16), torch.ones((1, 3, 512), dtype=torch.bfloat16)
    st = Store(1, 1, 48, 16, garbage=False)
    how = dict(how)
    lens = on(ints(1)) if how.pop("lens", False) else None
    codes, exps, bt = (on(t) for t in (st.codes, st.exps, st.bt))
    with pytest.raises(ValueError, match="ring"):
        path.chunk_step_fp8_paged(on(q), on(x), codes, exps, bt, on(ints(5)), on(torch.zeros(2)), scale=0.1, rd=0, table=None,
                                  eps=1e-6, lens=lens, **how)
    assert not codes.any() and not exps.any()


@pytest.mark.parametrize("how", LAYOUTS)
def test_step_refuses_a_ring_before_it_stores(lib, how):
    from sparse_latent_attention_attn_gb300 import path
    layout_step(path, how, lambda t: t)


@gpu
@pytest.mark.parametrize("how", LAYOUTS)
def test_step_refuses_a_ring_before_it_stores_on_the_gpu(ds, how):
    from sparse_latent_attention_attn_gb300 import path
    layout_step(path, how, dev)
    assert ds.device_status() == 0


@gpu
def test_bindings_refuse_what_does_not_fit(ds):
    st = Store(1, 2, 40, 16, garbage=False)
    c, k, bt = st.on_gpu()
    q, sink, first = torch.zeros((2, 1, 4, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros(4, device="cuda"), dev(ints(5, 6))
    good = dict(q=q, codes=c, exps=k, block_table=bt, first=first, sink=sink, scale=0.1, window=8, ring=8)
    ds.chunk_attn_fp8_paged(**good)
    tab = dev(table_of(20, 64))
    for bad in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(codes=c.to(torch.int8)), dict(codes=c[..., :256]), dict(exps=k[..., :8]),
                dict(exps=k[:-1]), dict(block_table=bt.long()), dict(block_table=bt[:1]), dict(first=first[:1]), dict(first=first.long()),
                dict(sink=sink[:3]), dict(sink=sink.double()), dict(lens=first[:1]), dict(lens=first.cpu()), dict(o=q[:1]),
                dict(o=q.float()), dict(rd=64), dict(rd=64, table=tab[:, :8]), dict(rd=64, table=tab.double()), dict(workspace=torch.empty(9))):
        with pytest.raises((TypeError, ValueError)):
            ds.chunk_attn_fp8_paged(**{**good, **bad})
    for bad, status in ((dict(window=9), ds.DS_EINVAL), (dict(window=1 << 31), ds.DS_EUNSUPPORTED), (dict(ring=-1), ds.DS_EINVAL),
                        (dict(base=1 << 32, ratio=2), ds.DS_EUNSUPPORTED), (dict(ratio=2, base=7), ds.DS_EINVAL)):
        with pytest.raises(ds.DsError) as e:
            ds.chunk_attn_fp8_paged(**{**good, **bad})
        assert e.value.status == status, bad
    read = dict(codes=c, exps=k, block_table=bt, n=3)
    ds.kv_read_fp8_paged(**read)
    idx = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    for bad in (dict(codes=c.float()), dict(exps=k[:-1]), dict(block_table=bt.long()), dict(first=first[:1]), dict(idx=idx[:, :2]),
                dict(idx=idx.long()), dict(lens=first.long()), dict(y=q[0]), dict(first=first, idx=idx)):
        with pytest.raises((TypeError, ValueError)):
            ds.kv_read_fp8_paged(**{**read, **bad})
    for n in (-1, 1 << 31):
        with pytest.raises((ds.DsError, RuntimeError)):
            ds.kv_read_fp8_paged(c, k, bt, n)
    assert ds.device_status() == 0


def test_the_plain_quantiser():
    """The reference's own rule: nearest value, ties to the even code, the least power of two."""
    c, k = quantise(np.array([[448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -0.0] + [0.0] * 24]))
    assert k[0, 0] == 0 and c[0, :8].tolist() == [126, 88, 90, 216, 0, 2, 0, 128]
    assert quantise(np.full((1, 32), 449.0))[1][0, 0] == 1 and quantise(np.zeros((1, 32)))[1][0, 0] == -22
    assert np.array_equal(values(*quantise(np.full((1, 32), 3.0, dtype=float))), np.full((1, 32), 3.0))
