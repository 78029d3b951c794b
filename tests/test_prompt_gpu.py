"""Causal attention over packed prompts (qsa_prompt_attn) against a plain float64
implementation on the host (needs a B200).

Tolerance, before any run, relative to A = sum_j p_j |v_j|: the output's rounding u, the weights'
rounding u (they enter the tensor cores in the input type), fp32 scores below 40 with 256 products
(40 * 2^-24 * 16 in the exponent), ex2 2^-22 and sums below 2^-17: 2 u + 2^-14 together.  fp16 weights
below fp16's normal range are off by 2^-25 where the largest is at least 1 (2^-8 times that when the
reference maximum lags): an absolute keys * 2^-25 * max|v| on top.
The gate multiplies by a factor below 1 with a relative error below 2^-21.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_paged_gpu import DEV, D, U, Case, attention, draw_rows

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def tol(dtype):
    return 2 * U[dtype] + 2.0 ** -14


def reference(q, k, v, scale, gate=None):
    """attention() of the decode tests, all rows of a head at once."""
    n, hq, _ = q.shape
    m, hkv = k.shape[0], k.shape[1]
    out, mag = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    if m:
        hide = np.arange(m)[None, :] > np.arange(n)[:, None] + (m - n)
        for h in range(hq):
            g = h // (hq // hkv)
            x = scale * (q[:, h] @ k[:, g].T)
            x[hide] = -np.inf
            top = np.maximum(x.max(-1, keepdims=True), -1e300)
            p = np.exp(x - top)
            p[hide] = 0
            total = p.sum(-1, keepdims=True)
            p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
            out[:, h], mag[:, h] = p @ v[:, g], p @ np.abs(v[:, g])
    if gate is not None:
        f = 1 / (1 + np.exp(-gate))
        out, mag = out * f, mag * f
    return out, mag


def check(qsa, n, m, hq, hkv, dtype, gated=False, tail=5, seed=0, q_scale=1.0, scale=1 / 16):
    """Prompts of n[s] rows against m[s] keys, `tail` rows and keys of no sequence behind them
    (the keys there are NaN), q, gate, k, v as slices of wider rows."""
    cq, ck = np.concatenate([[0], np.cumsum(n)]), np.concatenate([[0], np.cumsum(m)])
    rows, keys = int(cq[-1]), int(ck[-1])
    qg = draw_rows(seed, (rows + tail, 2, hq, D), dtype, q_scale)
    kv = draw_rows(seed + 1, (keys + tail, 2, hkv, D), dtype)
    kv[keys:] = float("nan")
    out = torch.full((rows + tail, hq, D), 7.0, dtype=dtype, device=DEV)
    gate = qg[:, 1] if gated else None
    qsa.prompt_attn(qg[:, 0], kv[:, 0], kv[:, 1], ints(cq), ints(ck), scale=scale, gate=gate, out=out)
    torch.cuda.synchronize()
    assert qsa.device_status() == 0
    assert torch.all(out[rows:] == 7.0), "rows behind the last prompt changed"
    got = out.double().cpu().numpy()
    q, g = qg[:, 0].double().cpu().numpy(), qg[:, 1].double().cpu().numpy()
    k, v = kv[:, 0].double().cpu().numpy(), kv[:, 1].double().cpu().numpy()
    for s in range(len(n)):
        a, b, c, d = cq[s], cq[s + 1], ck[s], ck[s + 1]
        if a == b:
            continue
        ref, mag = reference(q[a:b], k[c:d], v[c:d], scale, g[a:b] if gated else None)
        assert np.all(np.isfinite(got[a:b])), s
        err = np.abs(got[a:b] - ref)
        assert np.all(err[mag == 0] == 0), s
        floor = (d - c) * 2.0 ** -25 * (np.abs(v[c:d]).max() if d > c else 0)
        worst = float((np.maximum(err - floor, 0) / np.maximum(mag, 1e-30)).max())
        assert worst <= tol(dtype), f"sequence {s}: error {worst:.3e} above {tol(dtype):.3e}"
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [[1], [128], [129], [300], [7, 0, 64, 200, 1, 65, 127]])
def test_prompt_lengths(gpu, dtype, n):
    check(gpu, n, n, 4, 2, dtype, gated=len(n) > 1)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_longer_than_the_ring(gpu, dtype):
    check(gpu, [1000, 1537], [1000, 1537], 2, 1, dtype)


@pytest.mark.parametrize("n,m", [([5], [700]), ([130, 1, 64], [1000, 257, 64]), ([1, 1], [1, 4000]), ([256], [384])])
def test_prompt_with_prefix(gpu, n, m):
    check(gpu, n, m, 4, 2, torch.bfloat16, gated=True)


@pytest.mark.parametrize("n,m", [([200], [50]), ([40, 3], [0, 2]), ([300, 10], [129, 10]), ([4], [0])])
def test_prompt_rows_that_see_nothing(gpu, n, m):
    """Fewer keys than rows: the first rows see none and are 0."""
    check(gpu, n, m, 4, 2, torch.float16, gated=True)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (24, 2), (8, 8), (6, 1), (40, 4)])
def test_prompt_head_layouts(gpu, hq, hkv):
    check(gpu, [140, 33], [140, 50], hq, hkv, torch.float16)


@pytest.mark.parametrize("n,m,hq,hkv", [([3], [9000], 24, 2), ([1, 130], [3000, 5000], 6, 2), ([140], [6000], 3, 1),
                                        ([300, 0, 2], [4000, 0, 1], 5, 5), ([2, 2], [1, 8000], 4, 2)])
def test_prompt_keys_in_parts(gpu, n, m, hq, hkv):
    """Few rows against many keys: the keys are cut and joined, also for sequences whose keys fill
    one part only, or none."""
    assert gpu.prompt_attn_workspace_bytes(len(n), sum(n) + 5, sum(m) + 5, hq, hkv) > 0
    check(gpu, n, m, hq, hkv, torch.float16, gated=True)
    check(gpu, n, m, hq, hkv, torch.bfloat16)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_large_scores(gpu, dtype):
    """Scores of tens and rising maxima: O is rescaled along the keys."""
    n = 700
    q, k = draw_rows(3, (n, 2, D), dtype), draw_rows(4, (n, 1, D), dtype)
    k = (k.float() * torch.linspace(0.1, 3, n, device=DEV)[:, None, None]).to(dtype)
    v = draw_rows(5, (n, 1, D), dtype)
    got = gpu.prompt_attn(q, k, v, ints([0, n])).double().cpu().numpy()
    ref, mag = reference(q.double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(), 1 / 16)
    floor = n * 2.0 ** -25 * float(v.abs().max())
    assert (np.maximum(np.abs(got - ref) - floor, 0) / np.maximum(mag, 1e-30)).max() <= tol(dtype)


def test_prompt_many_sequences(gpu):
    r = np.random.RandomState(6)
    n = r.randint(0, 40, 300)
    n[:33] = 0
    check(gpu, n, n + r.randint(0, 30, 300), 2, 2, torch.bfloat16)


def test_prompt_neighbours_do_not_matter(gpu):
    """NaN rows of the sequences around leave a sequence's rows as they are."""
    qsa = gpu
    cu = ints([0, 100, 230, 300])
    q, k, v = (draw_rows(i, (300, h, D), torch.bfloat16) for i, h in ((7, 4), (8, 2), (9, 2)))
    want = qsa.prompt_attn(q, k, v, cu)
    for t in (q, k, v):
        t[:100] = float("nan")
        t[230:] = float("inf")
    got = qsa.prompt_attn(q, k, v, cu)
    assert torch.equal(got[100:230], want[100:230])


@pytest.mark.parametrize("rows,keys,split", [(300, 300, False), (40, 9000, True)])
def test_prompt_keys_to_come_do_not_matter(gpu, rows, keys, split):
    """A row's result does not change with the keys behind it: NaN and infinite K, other V."""
    qsa = gpu
    g = torch.Generator(device=DEV).manual_seed(61)
    q = torch.randn(rows, 4, D, generator=g, device=DEV).to(torch.bfloat16)
    kv = torch.randn(2, keys, 2, D, generator=g, device=DEV).to(torch.bfloat16)
    cq = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    ck = torch.tensor([0, keys], dtype=torch.int32, device=DEV)
    assert (qsa.prompt_attn_workspace_bytes(1, rows, keys, 4, 2) > 0) == split
    want = qsa.prompt_attn(q, kv[0], kv[1], cq, ck)
    seen = rows // 2  # the first rows, and the keys that the last of them sees
    other = kv.clone()
    last = keys - rows + seen
    other[0, last:] = float("nan")
    other[0, last + 1::2] = float("inf")
    other[1, last:] = 30000.0
    got = qsa.prompt_attn(q, other[0], other[1], cq, ck)
    torch.cuda.synchronize()
    assert torch.equal(got[:seen], want[:seen])
    assert not torch.isfinite(got[seen:]).any()


def test_prompt_runs_are_equal_and_on_another_stream(gpu):
    qsa = gpu
    cu = ints([0, 500, 900])
    q, k, v = (draw_rows(i, (900, h, D), torch.float16) for i, h in ((7, 6), (8, 2), (9, 2)))
    want = qsa.prompt_attn(q, k, v, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = qsa.prompt_attn(q, k, v, cu, stream=side)
    again = qsa.prompt_attn(q, k, v, cu)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


def test_prompt_graph_follows_the_lengths(gpu):
    qsa = gpu
    q, k, v = (draw_rows(i, (400, h, D), torch.float16) for i, h in ((7, 4), (8, 2), (9, 2)))
    cu, out = ints([0, 150, 400]), torch.empty(400, 4, D, dtype=torch.float16, device=DEV)
    qsa.prompt_attn(q, k, v, cu, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.prompt_attn(q, k, v, cu, out=out)
    for c in ([0, 150, 400], [0, 400, 400], [0, 1, 300]):
        cu.copy_(ints(c))
        out.fill_(0)
        g.replay()
        got = out.clone()
        want = qsa.prompt_attn(q, k, v, cu)
        assert torch.equal(got[:c[-1]], want[:c[-1]])
        assert torch.all(got[c[-1]:] == 0)


def test_served_requests_together(gpu):
    """What a server does: prompts are written and attended, their next chunk is written, the
    cached prefix read back and attended, then tokens are decoded, all against float64."""
    qsa = gpu
    dtype, page, hq, hkv = torch.bfloat16, 16, 6, 2
    n1, n2 = [70, 33], [40, 129]
    c = Case(qsa, [a + b + 1 for a, b in zip(n1, n2)], [1, 1], page=page, hkv=hkv, seed=30, fill=False)
    table = c.batch.table
    first = qsa.Batch(table, ints(n1), ints(np.concatenate([[0], np.cumsum(n1)])))
    k1, v1 = draw_rows(31, (sum(n1), hkv, D), dtype), draw_rows(32, (sum(n1), hkv, D), dtype)
    qsa.paged_write(c.cache, first, k1, v1)
    q1 = draw_rows(33, (sum(n1), hq, D), dtype)
    qsa.prompt_attn(q1, k1, v1, first.cu_q)
    total = [a + b for a, b in zip(n1, n2)]
    cu2, cut = np.concatenate([[0], np.cumsum(n2)]), np.concatenate([[0], np.cumsum(total)])
    k2, v2 = draw_rows(34, (sum(n2), hkv, D), dtype), draw_rows(35, (sum(n2), hkv, D), dtype)
    qsa.paged_write(c.cache, qsa.Batch(table, ints(total), ints(cu2)), k2, v2)
    whole = qsa.Batch(table, ints(total), ints(cut))
    kk, vv = qsa.paged_read(c.cache, whole, sum(total), dtype)
    q2 = draw_rows(36, (sum(n2), hq, D), dtype)
    out2 = qsa.prompt_attn(q2, kk, vv, ints(cu2), whole.cu_q)
    k3, v3, q3 = (draw_rows(37 + i, (2, h, D), dtype) for i, h in enumerate((hkv, hkv, hq)))
    qsa.paged_write(c.cache, c.batch, k3, v3)
    out3 = qsa.paged_decode(c.cache, c.batch, q3).double().cpu().numpy()
    for name in ("k", "v", "ks", "vs"):
        setattr(c, name, getattr(c.cache, name).cpu().numpy())
    for s in range(2):
        a, b, e, f = cu2[s], cu2[s + 1], cut[s], cut[s + 1]
        # the chunk against the values as read back, which are the cells' values to one rounding
        kd, vd = kk[e:f].double().cpu().numpy(), vv[e:f].double().cpu().numpy()
        held = c.values(c.v, c.vs, s, 0, total[s])
        assert np.all(np.abs(vd - held) <= U[dtype] * np.abs(held) * 1.01)
        ref, mag = reference(q2[a:b].double().cpu().numpy(), kd, vd, 1 / 16)
        assert (np.abs(out2[a:b].double().cpu().numpy() - ref) / mag).max() <= tol(dtype)
        # the values held are within half a code step, and half a step of the scale, of those written
        wrote = torch.cat([v1[[0, 70][s]:[70, 103][s]], v2[a:b]]).double().cpu().numpy()
        step = np.repeat(c.vs[c.cells(s, 0, total[s])].astype(np.float64), 32, -1)
        assert np.all(np.abs(held - wrote) <= step * 0.5 * 1.001 + 127 * step * 2.0 ** -11)
        L = total[s] + 1
        ref, mag = attention(q3[s:s + 1].double().cpu().numpy(), c.values(c.k, c.ks, s, 0, L), c.values(c.v, c.vs, s, 0, L),
                             1 / 16)
        # the decode's tolerance, with its six deviations of the rounded K: |q o k| <= |q| max|k|
        kmax, qn = np.abs(c.values(c.k, c.ks, s, 0, L)).max(), float(q3[s].double().norm(dim=-1).max())
        extra = 6 * 2.0 ** -11 / 3 ** 0.5 / 16 * qn * kmax
        assert (np.abs(out3[s:s + 1] - ref) / mag).max() <= U[dtype] + 2.6 * 2.0 ** -11 + extra
