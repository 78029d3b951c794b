"""The batched calls (paged cache write, read, decode attention) against plain float64
implementations on the host (needs a B200).

Tolerances, before any run.  u = half a step of a type: 2^-11 for fp16, 2^-8 for bf16, 2^-24
for fp32, relative to the value.

* Write: codes and scales are equal bit for bit to the quantiser's steps in numpy's IEEE fp32.
* Read: code * scale is exact in fp32, so the values are equal to its one rounding.
* Decode, errors relative to A = sum_c p_c |v_c| (what the dim would be without cancellation):
  fp16 / bf16: the output's rounding u * |o| <= u * A, the weights' 2^-11 and the V values'
  2^-11 (V below fp16's normal range is not drawn), ex2 and fp32 sums below 2^-17, q exact in
  fp16: together u + 2 * 2^-11, with 30 % for the rest u + 2.6 * 2^-11.
  fp16 / bf16 calls also round K = code * scale to fp16: each product q_d k_d of a score is off by
  an independent rounding of at most 2^-11 |q_d k_d|, variance a third of its square at most, so a
  score by 2^-11 / sqrt(3) * scale * |q o k| (the 2-norm of the products) in standard deviation; six
  of them, for the row and cell where that is largest, bound every weight's relative error and so the
  output's share of A.  That is added for these types.
  A weight below fp16's normal range is off by up to 2^-25 (half its subnormal step) where the
  largest weight is at least 1, whatever the weight: in a dim whose heavy cells hold codes of 0
  that is no fraction of A but up to sum_c 2^-25 |v_c| <= cells * 2^-25 * max|v|, and an fp32
  call's V residual adds 2^-25 of the weights' sum.  So every type has the absolute part
  (cells + 1) * 2^-25 * max(1, max|v|) on top.
  fp32: pairs of fp16 lose at most 2^-21 in each of q, weights and V (residuals below 2^-24 absolute: V
  is of order 1), scores up to 40 have fp32 errors of 40 * 2^-24 * (number of roundings, 16 + 8) in the exponent,
  ex2 2^-22: 40 * 24 * 2^-24 + 3 * 2^-21 + 2^-21 < 6e-5.
  The gate multiplies by a factor below 1 with a relative error below 2^-21.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, NG = 256, 8
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TOL = {torch.float16: 2.0 ** -11 + 2.6 * 2.0 ** -11, torch.bfloat16: 2.0 ** -8 + 2.6 * 2.0 ** -11, torch.float32: 6e-5}
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def quantise(x):
    """numpy fp32 [..., 256] -> codes int8, scales fp16 [..., 8] (every step in IEEE fp32)."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], NG, 32)
    with np.errstate(over="ignore"):
        s = (np.abs(g).max(-1) * (np.float32(1) / np.float32(127))).astype(np.float16)
    s = np.minimum(s, np.float16(65504))
    f = s.astype(np.float32)[..., None]
    code = np.rint(np.divide(g, f, out=np.zeros_like(g), where=f > 0)).clip(-127, 127)
    return code.reshape(x.shape).astype(np.int8), s


class Case:
    """A batch on the device and, on the host, each sequence's cells as float64 values."""

    def __init__(self, qsa, lens, rows, page, hkv, seed=0, spare=2, fill=True, scales=(0.005, 0.03)):
        r = np.random.RandomState(seed)
        self.lens, self.rows, self.page, self.hkv = list(lens), list(rows), page, hkv
        used = [-(-n // page) for n in lens]
        width = max(1, max(used))
        pages = sum(used) + spare
        order = r.permutation(pages)
        self.table = np.full((len(lens), width), -1, np.int64)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        self.free = order[at:]
        shape = (pages, page, hkv)
        if fill:
            self.k = r.randint(-127, 128, shape + (D,)).astype(np.int8)
            self.v = r.randint(-127, 128, shape + (D,)).astype(np.int8)
            self.ks = r.uniform(*scales, shape + (NG,)).astype(np.float16)
            self.vs = r.uniform(*scales, shape + (NG,)).astype(np.float16)
        else:
            self.k, self.v = np.zeros(shape + (D,), np.int8), np.zeros(shape + (D,), np.int8)
            self.ks, self.vs = np.zeros(shape + (NG,), np.float16), np.zeros(shape + (NG,), np.float16)
        self.cu = np.concatenate([[0], np.cumsum(rows)])
        self.cache = qsa.PagedCache(*(torch.from_numpy(a).to(DEV) for a in (self.k, self.v, self.ks, self.vs)))
        self.batch = qsa.Batch(self.ints(self.table), self.ints(self.lens), self.ints(self.cu))

    @staticmethod
    def ints(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)

    def cells(self, s, lo, hi):
        p = np.arange(lo, hi)
        return self.table[s, p // self.page], p % self.page

    def values(self, codes, scales, s, lo, hi):
        at = self.cells(s, lo, hi)
        return codes[at].astype(np.float64) * np.repeat(scales[at].astype(np.float64), 32, axis=-1)


def attention(q, k, v, scale, gate=None):
    """float64: q [n, hq, D], k / v [m, hkv, D]; row i sees keys <= i + m - n.  (out, A)."""
    n, hq, _ = q.shape
    m, hkv = k.shape[0], k.shape[1]
    out, mag = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    for i in range(n):
        seen = i + m - n + 1
        if seen <= 0:
            continue
        for h in range(hq):
            g = h // (hq // hkv)
            x = scale * (k[:seen, g] @ q[i, h])
            p = np.exp(x - x.max())
            p /= p.sum()
            out[i, h], mag[i, h] = p @ v[:seen, g], p @ np.abs(v[:seen, g])
    if gate is not None:
        f = 1 / (1 + np.exp(-gate))
        out, mag = out * f, mag * f
    return out, mag


def draw_rows(seed, shape, dtype, scale=1.0):
    x = torch.from_numpy(np.random.RandomState(seed).standard_normal(shape).astype(np.float32) * np.float32(scale))
    return x.to(dtype).to(DEV)


def check_decode(qsa, c, hq, dtype, gated=False, max_q=None, max_len=None, scale=1 / 16, q_scale=1.0, tail=3):
    """Run paged_decode with `tail` padded rows and compare every row; the tail stays."""
    rows = int(c.cu[-1])
    q = draw_rows(1, (rows + tail, hq, D), dtype, q_scale)
    gate = draw_rows(2, (rows + tail, hq, D), dtype) if gated else None
    out = torch.full((rows + tail, hq, D), 7.0, dtype=dtype, device=DEV)
    max_q = max_q or max(c.rows)
    max_len = max_len or max(1, max(c.lens))
    qsa.paged_decode(c.cache, c.batch, q, scale=scale, max_q=max_q, max_len=max_len, gate=gate, out=out)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert np.all(got[rows:] == 7.0), "rows behind the last sequence changed"
    worst = 0.0
    for s in range(len(c.lens)):
        a, b = c.cu[s], c.cu[s + 1]
        if a == b:
            continue
        ref, mag = attention(q[a:b].double().cpu().numpy(), c.values(c.k, c.ks, s, 0, c.lens[s]),
                             c.values(c.v, c.vs, s, 0, c.lens[s]), scale,
                             None if gate is None else gate[a:b].double().cpu().numpy())
        err = np.abs(got[a:b] - ref)
        assert np.all(np.isfinite(got[a:b]))
        assert np.all(err[mag == 0] == 0.0)
        if c.lens[s] and dtype != torch.float32:
            k2 = np.square(c.values(c.k, c.ks, s, 0, c.lens[s]))
            q2 = np.square(q[a:b].double().cpu().numpy()).reshape(b - a, c.hkv, -1, D)
            norm = np.sqrt(max((q2[:, g].reshape(-1, D) @ k2[:, g].T).max() for g in range(c.hkv)))
            err = np.maximum(err - 6 * 2.0 ** -11 / 3 ** 0.5 * scale * norm * mag, 0)
        if c.lens[s]:
            err = np.maximum(err - (c.lens[s] + 1) * 2.0 ** -25 * max(1.0, np.abs(c.values(c.v, c.vs, s, 0, c.lens[s])).max()), 0)
        worst = max(worst, float((err / np.maximum(mag, 1e-30)).max()))
    assert worst <= TOL[dtype], f"error {worst:.3e} of the sum of magnitudes, above {TOL[dtype]:.3e}"
    return out


# ------------------------------------------------------------------ write and read

PATTERNS = ["normal", "zero", "tiny", "huge", "half_ties"]


def pattern(name, shape, seed):
    r = np.random.RandomState(seed)
    x = r.standard_normal(shape).astype(np.float32)
    if name == "zero":
        x[...] = 0
        x[0] = -0.0
    if name == "tiny":
        x *= np.float32(1e-6)
    if name == "huge":
        x *= np.float32(3e4)
    if name == "half_ties":
        x = (r.randint(-254, 255, shape) / 2).astype(np.float32)
        x[..., ::32] = 127.0
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", PATTERNS)
def test_write_bit_exact(gpu, dtype, name):
    qsa = gpu
    c = Case(qsa, [13, 1, 40, 7], [5, 1, 33, 0], page=8, hkv=2, fill=False)
    n = int(c.cu[-1])
    wide = torch.from_numpy(pattern(name, (n + 2, 2, 2, D), 3)).to(dtype).to(DEV)  # K and V of a wider row
    qsa.paged_write(c.cache, c.batch, wide[:, 0], wide[:, 1])
    torch.cuda.synchronize()
    x = wide.float().cpu().numpy()
    want = [np.zeros_like(a) for a in (c.k, c.v, c.ks, c.vs)]
    for s in range(4):
        a, b = c.cu[s], c.cu[s + 1]
        at = c.cells(s, c.lens[s] - (b - a), c.lens[s])
        for i in range(2):
            want[i][at], want[2 + i][at] = quantise(x[a:b, i])
    for t, w in zip((c.cache.k, c.cache.v, c.cache.ks, c.cache.vs), want):
        assert np.array_equal(t.cpu().numpy(), w)  # the cells of other positions stay 0


def test_write_matches_the_contiguous_cache(gpu):
    """fp32 rows of one sequence: scales within one fp16 step of qsa_cache_write's, and the same
    codes where the scale is the same."""
    qsa = gpu
    n = 77
    k, v = draw_rows(4, (n, 2, D), torch.float32), draw_rows(5, (n, 2, D), torch.float32)
    flat = qsa.DeviceCache.empty(n, DEV)
    qsa.cache_write(flat, 0, k, v, torch.zeros(n, 64, dtype=torch.float16, device=DEV))
    c = Case(qsa, [n], [n], page=16, hkv=2, fill=False)
    qsa.paged_write(c.cache, c.batch, k, v)
    at = c.cells(0, 0, n)
    for codes, scales in (("k", "ks"), ("v", "vs")):
        bits, want = (t.cpu().numpy().view(np.int16).astype(int) for t in (getattr(c.cache, scales), getattr(flat, scales)))
        bits = bits[at]
        assert np.abs(bits - want).max() <= 1
        same = np.repeat(bits == want, 32, axis=-1)
        assert same.mean() > 0.99
        assert np.array_equal(getattr(c.cache, codes).cpu().numpy()[at][same], getattr(flat, codes).cpu().numpy()[same])


@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
def test_write_skips_what_has_no_cell(gpu, hkv):
    """More rows than positions, pages outside the pool and past the table: nothing else changes."""
    qsa = gpu
    c = Case(qsa, [3, 20, 9], [5, 20, 9], page=4, hkv=hkv, seed=1)
    before = [t.clone() for t in (c.cache.k, c.cache.ks)]
    table = c.table.copy()
    table[1, 2] = -5
    table[1, 3] = c.cache.pages
    batch = qsa.Batch(c.ints(table), c.ints([3, 20, 9 + 4 * 5]), c.ints(c.cu))
    n = int(c.cu[-1])
    rows = draw_rows(6, (n, hkv, D), torch.float32)
    qsa.paged_write(c.cache, batch, rows, rows)
    torch.cuda.synchronize()
    x = rows.cpu().numpy()
    want = [t.cpu().numpy().copy() for t in before]
    def put(s, first_row, lo, hi):
        at = c.cells(s, lo, hi)
        want[0][at], want[1][at] = quantise(x[first_row:first_row + hi - lo])
    put(0, 2, 0, 3)       # rows 0 and 1 have positions -2 and -1
    put(1, 5, 0, 8)
    put(1, 5 + 16, 16, 20)
    # sequence 2's positions 20 .. 28 lie past its table of 5 pages of 4
    assert np.array_equal(c.cache.k.cpu().numpy(), want[0])
    assert np.array_equal(c.cache.ks.cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,hkv", [(1, 2), (7, 1), (16, 2), (64, 5)])
def test_read_whole_sequences(gpu, dtype, page, hkv):
    qsa = gpu
    lens = [0, 1, 130, 17, 0, 64]
    c = Case(qsa, lens, lens, page=page, hkv=hkv, seed=2)
    n = int(c.cu[-1])
    out = torch.full((n + 3, 2, hkv, D), 7.0, dtype=dtype, device=DEV)
    qsa.paged_read(c.cache, c.batch, n + 3, dtype, k=out[:, 0], v=out[:, 1])
    assert torch.all(out[n:] == 7.0)
    for s, L in enumerate(lens):
        for i, (codes, scales) in enumerate(((c.k, c.ks), (c.v, c.vs))):
            want = torch.from_numpy(c.values(codes, scales, s, 0, L).astype(np.float32)).to(dtype)
            assert torch.equal(out[c.cu[s]:c.cu[s + 1], i].cpu(), want)


def test_read_absent_cells_are_zero(gpu):
    qsa = gpu
    c = Case(qsa, [10], [14], page=4, hkv=2, seed=3)
    table = c.table.copy()
    table[0, 1] = -1
    k, v = qsa.paged_read(c.cache, qsa.Batch(c.ints(table), c.ints([10]), c.ints([0, 14])), 14, torch.float32)
    got = k.cpu().numpy()
    assert np.all(got[:4] == 0) and np.all(got[8:12] == 0)
    assert np.array_equal(got[4:8], c.values(c.k, c.ks, 0, 0, 4).astype(np.float32))
    assert np.array_equal(got[12:], c.values(c.k, c.ks, 0, 8, 10).astype(np.float32))


def test_many_sequences_find_their_rows(gpu):
    """More than 32 * 32 sequences, many of them empty: the search for a row's sequence."""
    qsa = gpu
    r = np.random.RandomState(8)
    lens = r.randint(0, 4, 1500)
    lens[:40] = 0
    lens[700:760] = 0
    lens[-3:] = 0
    c = Case(qsa, lens, lens, page=2, hkv=1, seed=4)
    n = int(c.cu[-1])
    k, _ = qsa.paged_read(c.cache, c.batch, n, torch.float32)
    want = np.concatenate([c.values(c.k, c.ks, s, 0, L).astype(np.float32) for s, L in enumerate(lens)])
    assert np.array_equal(k.cpu().numpy(), want)


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [0, 63, 64, 65, 1], [700], [1000, 3, 257]])
def test_decode_one_token(gpu, dtype, lens):
    c = Case(gpu, lens, [1] * len(lens), page=16, hkv=2, seed=10)
    check_decode(gpu, c, 24, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode_drafts(gpu, dtype, n):
    """Every row-tile count, drafts of different lengths, a draft longer than its cells (rows
    that see nothing are 0), a sequence without rows, the gate."""
    lens = [n, 100, 40, max(1, n - 1), 333]
    rows = [n, max(1, n - 1), 0, n, n]
    c = Case(gpu, lens, rows, page=32, hkv=2, seed=11)
    check_decode(gpu, c, 24, dtype, gated=True, max_q=n)


@pytest.mark.parametrize("hq,hkv,n", [(1, 1, 1), (8, 8, 8), (16, 1, 6), (6, 2, 8), (40, 4, 2), (5, 5, 3), (96, 1, 1)])
def test_decode_head_layouts(gpu, hq, hkv, n):
    c = Case(gpu, [200, 31], [n, 1], page=16, hkv=hkv, seed=12)
    check_decode(gpu, c, hq, torch.bfloat16, max_q=n)
    check_decode(gpu, c, hq, torch.float32, max_q=n)


@pytest.mark.parametrize("page", [1, 5, 16, 48, 1000])
def test_decode_page_sizes(gpu, page):
    c = Case(gpu, [1, 333, 50], [1, 2, 1], page=page, hkv=2, seed=13)
    check_decode(gpu, c, 4, torch.float16, max_q=2)


@pytest.mark.parametrize("dtype", TYPES)
def test_decode_many_blocks(gpu, dtype):
    """Enough cells that CTAs take several blocks and sequences, and units split over CTAs."""
    c = Case(gpu, [8000, 1, 0, 5000, 16, 7001, 300], [1, 1, 1, 2, 1, 1, 1], page=64, hkv=2, seed=14)
    check_decode(gpu, c, 8, dtype, gated=True, max_q=2)


def test_decode_many_sequences(gpu):
    r = np.random.RandomState(15)
    lens = r.randint(0, 90, 400)
    c = Case(gpu, lens, [1] * 400, page=16, hkv=2, seed=15)
    check_decode(gpu, c, 4, torch.float16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,hq", [(1, 4), (3, 24)])
def test_decode_ragged_with_empty_ones(gpu, dtype, n, hq):
    """Long sequences between short ones and empty ones, whose CTAs hold pieces and whole units."""
    r = np.random.RandomState(16)
    lens = np.where(r.rand(70) < 0.3, 0, np.exp(r.uniform(0, np.log(3000), 70)).astype(int))
    rows = r.randint(0, n + 1, 70)
    c = Case(gpu, lens, rows, page=48, hkv=2, seed=17)
    check_decode(gpu, c, hq, dtype, max_q=n)


def test_decode_default_one_row_each_and_max_len(gpu):
    """cu_q None is one row per sequence; the default max_len is the table's extent."""
    qsa = gpu
    c = Case(qsa, [90, 0, 33], [1, 1, 1], page=16, hkv=2, seed=16)
    q = draw_rows(1, (3, 24, D), torch.float32)
    a = qsa.paged_decode(c.cache, c.batch, q)
    b = qsa.paged_decode(c.cache, qsa.Batch(c.batch.table, c.batch.kv_len), q)
    assert torch.equal(a, b)
    assert torch.all(a[1] == 0)


def test_decode_absent_pages_and_shared_pages(gpu):
    """A page outside the pool has no cells; two sequences may share their prefix pages."""
    qsa = gpu
    c = Case(qsa, [64, 64], [1, 1], page=16, hkv=2, seed=17)
    table = c.table.copy()
    table[1, 0] = table[0, 0]   # shared
    table[1, 2] = 10 ** 6       # absent
    batch = qsa.Batch(c.ints(table), c.ints([64, 64]), c.ints([0, 1, 2]))
    q = draw_rows(3, (2, 24, D), torch.float32)
    out = qsa.paged_decode(c.cache, batch, q, max_len=64).double().cpu().numpy()
    c.table[1, 0] = c.table[0, 0]
    keep = np.r_[0:32, 48:64]
    k, v = c.values(c.k, c.ks, 1, 0, 64)[keep], c.values(c.v, c.vs, 1, 0, 64)[keep]
    ref, mag = attention(q[1:].double().cpu().numpy(), k, v, 1 / 16)
    assert (np.abs(out[1:] - ref) / mag).max() <= TOL[torch.float32]


def test_decode_large_and_rising_scores(gpu):
    """Scores of some hundreds that rise along the sequence: the maximum moves, weights underflow."""
    c = Case(gpu, [500, 900], [1, 2], page=16, hkv=2, seed=18)
    for s, L in enumerate(c.lens):
        at = c.cells(s, 0, L)
        c.ks[at] = (np.linspace(0.01, 0.2, L)[:, None, None] * np.ones((1, 2, NG))).astype(np.float16)
    c.cache.ks.copy_(torch.from_numpy(c.ks))
    # scores of up to 600 carry 600 * 24 * 2^-24 in the exponent: within the 16-bit types' bound
    check_decode(gpu, c, 24, torch.float16, max_q=2, q_scale=1.0)


def test_decode_stale_cells_do_not_matter(gpu):
    """What lies behind a sequence's end in its last page, NaN scales among it, is not read."""
    qsa = gpu
    c = Case(qsa, [21, 5], [1, 1], page=16, hkv=2, seed=19)
    q = draw_rows(4, (2, 24, D), torch.bfloat16)
    a = qsa.paged_decode(c.cache, c.batch, q)
    nan = torch.full((NG,), float("nan"), dtype=torch.float16, device=DEV)
    for s, L in enumerate(c.lens):
        pg = int(c.table[s, (L - 1) // 16])
        c.cache.ks[pg, L % 16:] = nan
        c.cache.vs[pg, L % 16:] = nan
    b = qsa.paged_decode(c.cache, c.batch, q)
    assert torch.equal(a, b) and torch.isfinite(b).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[40], [6000]])
@pytest.mark.parametrize("n", [1, 3])
def test_decode_nan_rows_stay_nan(gpu, dtype, lens, n):
    """A NaN query gives NaN in its own row and head alone: in whole and in joined pieces."""
    qsa = gpu
    c = Case(qsa, lens, [n], page=16, hkv=2, seed=23)
    q = draw_rows(9, (n, 24, D), dtype)
    want = qsa.paged_decode(c.cache, c.batch, q, max_q=n, max_len=lens[0])
    q[0, 5, 100] = float("nan")
    got = qsa.paged_decode(c.cache, c.batch, q, max_q=n, max_len=lens[0])
    torch.cuda.synchronize()
    assert torch.isnan(got[0, 5]).all()
    got[0, 5] = want[0, 5]
    assert torch.equal(got, want)


def test_decode_runs_are_equal_and_strides(gpu):
    """The same bits in every run; q, gate and out as slices of wider rows."""
    qsa = gpu
    c = Case(qsa, [3000, 777], [3, 2], page=64, hkv=2, seed=20)
    wide = draw_rows(5, (5, 3, 24, D), torch.float16)
    ref = qsa.paged_decode(c.cache, c.batch, wide[:, 0].contiguous(), max_q=3, gate=wide[:, 1].contiguous())
    for _ in range(3):
        qsa.paged_decode(c.cache, c.batch, wide[:, 0], max_q=3, gate=wide[:, 1], out=wide[:, 2])
        assert torch.equal(wide[:, 2], ref)


def test_decode_graph_follows_the_batch(gpu):
    """A captured call reads lengths and tables when it is replayed."""
    qsa = gpu
    c = Case(qsa, [200, 150], [1, 1], page=16, hkv=2, seed=21)
    q = draw_rows(6, (2, 24, D), torch.float32)
    out = torch.empty_like(q)
    ws = qsa.workspace(qsa.paged_decode_workspace_bytes(2, 24, 2, 1, 208), DEV)
    args = dict(max_len=208, out=out, ws=ws)
    qsa.paged_decode(c.cache, c.batch, q, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.paged_decode(c.cache, c.batch, q, **args)
    for lens in ([200, 150], [1, 0], [37, 150]):
        c.batch.kv_len.copy_(c.ints(lens))
        g.replay()
        got = out.clone()
        want = qsa.paged_decode(c.cache, c.batch, q, max_len=208)
        assert torch.equal(got, want), lens


def test_decode_on_another_stream(gpu):
    qsa = gpu
    c = Case(qsa, [900, 40], [1, 1], page=16, hkv=2, seed=22)
    q = draw_rows(7, (2, 24, D), torch.float16)
    want = qsa.paged_decode(c.cache, c.batch, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = qsa.paged_decode(c.cache, c.batch, q, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_write_then_decode_then_read(gpu):
    """A served step: the new tokens are written, attend, and read back."""
    qsa = gpu
    c = Case(qsa, [130, 64, 9], [2, 1, 3], page=16, hkv=2, seed=23)
    k, v = draw_rows(8, (6, 2, D), torch.bfloat16), draw_rows(9, (6, 2, D), torch.bfloat16)
    qsa.paged_write(c.cache, c.batch, k, v)
    for name in ("k", "v", "ks", "vs"):
        setattr(c, name, getattr(c.cache, name).cpu().numpy())
    check_decode(qsa, c, 24, torch.bfloat16, gated=True, max_q=3)
    kk, _ = qsa.paged_read(c.cache, c.batch, 6, torch.float32)
    codes, s = quantise(k.float().cpu().numpy())
    assert np.array_equal(kk.cpu().numpy(), codes.astype(np.float32) * np.repeat(s.astype(np.float32), 32, -1))


@pytest.mark.parametrize("dtype,n", [(torch.float32, 1), (torch.bfloat16, 1), (torch.float16, 3)])
def test_pages_far_into_the_pool(gpu, dtype, n):
    """Byte offsets past 2^32: a pool of 9 million cells whose last pages are in use."""
    qsa = gpu
    pages, page, L = 70000, 128, 300
    cache = qsa.PagedCache.empty(pages, page, 2, DEV)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device=DEV)
    kv_len = torch.tensor([L], dtype=torch.int32, device=DEV)
    k, v = draw_rows(40, (L, 2, D), dtype), draw_rows(41, (L, 2, D), dtype)
    whole = qsa.Batch(table, kv_len, torch.tensor([0, L], dtype=torch.int32, device=DEV))
    qsa.paged_write(cache, whole, k, v)
    kk, vv = qsa.paged_read(cache, whole, L, torch.float32)
    for x, got in ((k, kk), (v, vv)):
        codes, s = quantise(x.float().cpu().numpy())
        assert np.array_equal(got.cpu().numpy(), codes.astype(np.float32) * np.repeat(s.astype(np.float32), 32, -1))
    q = draw_rows(42, (n, 24, D), dtype)
    new = qsa.Batch(table, kv_len, torch.tensor([0, n], dtype=torch.int32, device=DEV))
    out = qsa.paged_decode(cache, new, q, max_q=n).double().cpu().numpy()
    kd, vd = kk.double().cpu().numpy(), vv.double().cpu().numpy()
    ref, mag = attention(q.double().cpu().numpy(), kd, vd, 1 / 16)
    norm = float(q.double().norm(dim=-1).max()) * np.abs(kd).max()   # |q o k| <= |q| max|k|
    extra = 0 if dtype == torch.float32 else 6 * 2.0 ** -11 / 3 ** 0.5 / 16 * norm
    assert (np.abs(out - ref) / mag).max() <= TOL[dtype] + extra


@pytest.mark.parametrize("dtype", TYPES)
def test_decode_rows_past_max_q_stay(gpu, dtype):
    """A sequence with more rows than max_q: its first max_q rows are computed, the others stay."""
    qsa = gpu
    c = Case(qsa, [100, 50], [4, 2], page=16, hkv=2, seed=24)
    q = draw_rows(1, (6, 24, D), dtype)
    want = qsa.paged_decode(c.cache, c.batch, q, max_q=4)
    out = torch.full_like(q, 7.0)
    qsa.paged_decode(c.cache, c.batch, q, max_q=2, out=out)
    assert torch.all(out[2:4] == 7.0)
    for r in (0, 1, 4, 5):
        assert (out[r].double() - want[r].double()).abs().max() <= 4 * TOL[dtype] * want[r].double().abs().max()


def test_decode_length_past_the_table(gpu):
    """Positions that the table does not reach, or past max_len, are not attended."""
    qsa = gpu
    c = Case(qsa, [64, 64], [1, 1], page=16, hkv=2, seed=25)
    q = draw_rows(2, (2, 24, D), torch.float32)
    want = qsa.paged_decode(c.cache, c.batch, q)
    longer = qsa.Batch(c.batch.table, c.ints([1000, 64]), c.batch.cu_q)
    assert torch.equal(qsa.paged_decode(c.cache, longer, q), want)
    short = qsa.paged_decode(c.cache, qsa.Batch(c.batch.table, c.ints([48, 64]), c.batch.cu_q), q)
    cut = qsa.paged_decode(c.cache, c.batch, q, max_len=48)
    assert torch.equal(cut[0], short[0])


def test_calls_on_two_streams_at_once(gpu):
    """Calls of all kinds on two streams, each with its own workspace, beside each other."""
    qsa = gpu
    c = Case(qsa, [5000, 1200, 333], [3, 3, 3], page=64, hkv=2, seed=26)
    q16, q32 = draw_rows(3, (9, 24, D), torch.bfloat16), draw_rows(4, (9, 24, D), torch.float32)
    pq, pk, pv = (draw_rows(i, (700, h, D), torch.bfloat16) for i, h in ((5, 24), (6, 2), (7, 2)))
    cu = c.ints([0, 700])
    calls = [lambda s: qsa.paged_decode(c.cache, c.batch, q16, max_q=3, stream=s),
             lambda s: qsa.paged_decode(c.cache, c.batch, q32, max_q=3, stream=s),
             lambda s: qsa.prompt_attn(pq, pk, pv, cu, stream=s),
             lambda s: qsa.prompt_attn(pq[:40].contiguous(), pk, pv, c.ints([0, 40]), cu, stream=s),
             lambda s: qsa.paged_read(c.cache, c.batch, 9, torch.float16, stream=s)[0]]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[] for _ in calls]
    for rep in range(4):
        for i, f in enumerate(calls):
            got[i].append(f(streams[(i + rep) % 2]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    assert qsa.device_status() == 0


def test_binding_refusals_on_the_gpu(gpu):
    """Shapes, types, strides, devices that the binding refuses; nothing is launched."""
    qsa = gpu
    c = Case(qsa, [40, 20], [1, 1], page=16, hkv=2, seed=27)
    q = draw_rows(1, (2, 24, D), torch.float16)
    before = qsa.launch_count()
    for args in (dict(q=q.cpu()), dict(q=q[:, :, :128]), dict(q=q.double()), dict(gate=q.float()), dict(gate=q[:1]),
                 dict(out=q[:1]), dict(ws=torch.empty(16, dtype=torch.uint8))):
        a = dict(q=q)
        a.update(args)
        with pytest.raises(ValueError):
            qsa.paged_decode(c.cache, c.batch, a.pop("q"), **a)
    with pytest.raises(qsa.QSAError, match="WORKSPACE"):
        qsa.paged_decode(c.cache, c.batch, q, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(qsa.QSAError, match="multiple"):
        qsa.paged_decode(c.cache, c.batch, draw_rows(1, (2, 23, D), torch.float16))
    with pytest.raises(ValueError):
        qsa.paged_write(c.cache, c.batch, q[:, :2], q[:, :3])
    with pytest.raises(ValueError):
        qsa.Batch(c.batch.table, c.batch.kv_len[:1])
    with pytest.raises(qsa.QSAError, match="QSA_F16"):
        x = q.float()
        qsa.prompt_attn(x, x, x, c.ints([0, 2]))
    assert qsa.launch_count() == before
