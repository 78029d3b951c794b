"""The operators of batched serving next to the QSA step, as their users call them, for timing and comparison.

Three operators share one batch of sequences:

* ``cache``   K/V rows of packed sequences are quantised into the paged int8 cache as they are written
              (one fp16 scale per 32 values), and read back as the values they stand for;
* ``read``    the cells of whole sequences are read back, packed;
* ``decode``  the newest tokens of each sequence attend all its cells in the paged cache;
* ``prompt``  packed prompts of different lengths attend causally over fp16 / bf16 K/V rows.

Sequence s of a batch has rows cu[s] .. cu[s+1]-1 of the packed arrays, and they are its last
positions: with n rows and a length of L, row j is position L - n + j.  Position p is held in
cell p % page of page table[s][p // page].
"""
import math
import random

import numpy as np
import torch

own = False

D = 256        # head dim
GROUP = 32     # values per scale
NG = D // GROUP
SCALE = 1.0 / 16.0
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decode step's write for eight sequences: the smallest call, where latency counts.
        dict(name="cache 8x1", op="cache", nseq=8, lo=40, hi=900, mix=1, rows=1, hkv=2, page=64, dtype="fp16"),
        # A prompt chunk of 2048 tokens of five requests, K and V inside a wider projection row.
        dict(name="cache chunk", op="cache", nseq=5, lo=300, hi=600, mix=2, rows=600, hkv=2, page=64, dtype="bf16"),
        # A whole long prompt in fp32, the type of the step calls' rows.
        dict(name="cache 40000 fp32", op="cache", nseq=1, lo=40000, hi=40000, mix=3, rows=40000, hkv=2, page=128, dtype="fp32"),
        # The cached prefixes of a few requests, read back for their next chunk.
        dict(name="read prefixes", op="read", nseq=6, lo=100, hi=4097, mix=4, hkv=2, page=16, dtype="bf16"),
        # One 256K context read back whole.
        dict(name="read 262144", op="read", nseq=1, lo=262144, hi=262144, mix=5, hkv=2, page=128, dtype="fp16"),
        # One short request, one token, fp32 as the step calls: latency.
        dict(name="decode 1x700 fp32", op="decode", nseq=1, lo=700, hi=700, mix=6, rows=1, hq=24, hkv=2, page=64, dtype="fp32", gate=False),
        # An ordinary serving batch of ragged contexts.
        dict(name="decode 32 ragged", op="decode", nseq=32, lo=50, hi=8192, mix=7, rows=1, hq=24, hkv=2, page=64, dtype="bf16", gate=True),
        # Draft verification: up to four tokens per sequence, gate on.
        dict(name="decode 16 draft", op="decode", nseq=16, lo=1000, hi=16384, mix=8, rows=4, hq=24, hkv=2, page=32, dtype="fp16", gate=True),
        # The longest contexts, two sequences.
        dict(name="decode 2x262144", op="decode", nseq=2, lo=250001, hi=262144, mix=9, rows=1, hq=24, hkv=2, page=128, dtype="bf16", gate=False),
        # Short prompts of different lengths.
        dict(name="prompt short", op="prompt", nseq=7, lo=1, hi=300, mix=10, prefix=0, hq=24, hkv=2, dtype="fp16", gate=False),
        # An ordinary batch: four prompts of up to 4096.
        dict(name="prompt 4x4096", op="prompt", nseq=4, lo=1500, hi=4096, mix=11, prefix=0, hq=24, hkv=2, dtype="bf16", gate=True),
        # A 2048-token chunk at the end of a 65536-token context.
        dict(name="prompt chunk 65536", op="prompt", nseq=1, lo=2048, hi=2048, mix=12, prefix=63488, hq=24, hkv=2, dtype="bf16", gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "read", "decode", "decode", "prompt", "prompt"])
    mix = rng.randrange(1 << 20)
    hkv = rng.choice([1, 2, 2, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["fp32", "fp16", "bf16"])
    if op in ("cache", "read"):
        total = _log(rng, 8, 80000 // hkv)
        nseq = _log(rng, 1, min(64, total))
        hi = max(1, total // nseq)
        c = dict(op=op, nseq=nseq, lo=max(1, hi // 3), hi=hi, mix=mix, hkv=hkv, page=page, dtype=dtype)
        if op == "cache":
            c["rows"] = rng.choice([1, 3, max(1, hi // 2), hi])
        return c
    if op == "decode":
        group = rng.choice([1, 3, 4, 6, 8, 12, 12, 16])
        hi = _log(rng, 1, 262144)
        nseq = _log(rng, 1, max(1, min(64, (1 << 20) // (hi * hkv))))
        rows = rng.choice([1, 1, 1, 2, 3, 4, 8])
        rows = max(1, min(rows, hi, 96 // group))
        return dict(op=op, nseq=nseq, lo=max(rows, hi // rng.choice([1, 4, 30])), hi=hi, mix=mix, rows=rows,
                    hq=group * hkv, hkv=hkv, page=page, dtype=dtype, gate=rng.random() < 0.5)
    group = rng.choice([1, 2, 4, 6, 12, 12])
    hq = group * hkv
    hi = _log(rng, 1, 8192)
    prefix = rng.choice([0, 0, _log(rng, 1, 32768)])
    most = 3200000000 // 2 // hq  # padded scores of the largest listed case, halved
    while hi * (hi + prefix) > most:
        hi = hi * 2 // 3
    nseq = _log(rng, 1, max(1, min(32, most // (hi * (hi + prefix)))))
    return dict(op=op, nseq=nseq, lo=max(1, hi // rng.choice([1, 3, 20])), hi=hi, mix=mix, prefix=prefix, hq=hq,
                hkv=hkv, dtype=rng.choice(["fp16", "bf16"]), gate=rng.random() < 0.5)


def _lengths(case):
    """Sequence lengths between lo and hi, spread over their logarithm; one sequence has hi."""
    r = np.random.RandomState(case["mix"])
    n = np.exp(r.uniform(math.log(case["lo"]), math.log(case["hi"]), case["nseq"])).round().astype(np.int64)
    n = np.clip(n, case["lo"], case["hi"])
    n[r.randint(case["nseq"])] = case["hi"]
    return n


def _rows(case, length):
    """New rows of each sequence: at most case["rows"]; drafts differ between sequences."""
    if case["op"] == "read":
        return length
    if case["op"] == "decode" and case["rows"] > 1:
        r = np.random.RandomState(case["mix"] + 1)
        n = r.randint(1, case["rows"] + 1, case["nseq"])
        n[r.randint(case["nseq"])] = case["rows"]
        return np.minimum(n, length)
    return np.minimum(case["rows"], length)


def _cu(n):
    return np.concatenate([[0], np.cumsum(n)])


def _visible(n, total):
    """Keys that the n last rows of `total` positions see, summed."""
    return int((n * (total - n) + n * (n + 1) // 2).sum())


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "prompt":
        n = _lengths(case)
        total = n + case["prefix"]
        io = int(n.sum()) * case["hq"] * (3 if case["gate"] else 2) + 2 * int(total.sum()) * case["hkv"]
        return {"bytes": io * D * size, "flops": 4 * D * case["hq"] * _visible(n, total)}
    length = _lengths(case)
    n = _rows(case, length)
    cell = case["hkv"] * 2 * (D + 2 * NG)   # codes and scales of K and V
    if case["op"] == "decode":
        io = int(n.sum()) * case["hq"] * D * size * (3 if case["gate"] else 2)
        return {"bytes": int(length.sum()) * cell + io, "flops": 4 * D * case["hq"] * _visible(n, length)}
    value = int(n.sum()) * case["hkv"] * 2 * D * size
    if case["op"] == "read":
        return {"bytes": int(n.sum()) * cell + value, "flops": 0}
    # written and read back: the rows in, the cells out and in, the values out
    return {"bytes": 2 * value + 2 * int(n.sum()) * cell, "flops": 0}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    def ints(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")

    st = {"op": case["op"], "dtype": dt, "hkv": case["hkv"]}
    length = _lengths(case)
    if case["op"] == "prompt":
        hq, hkv = case["hq"], case["hkv"]
        total = length + case["prefix"]
        rows, cells = int(length.sum()), int(total.sum())
        st.update(cu_q=ints(_cu(length)), cu_k=ints(_cu(total)), max_q=int(length.max()), max_k=int(total.max()), hq=hq)
        # the projection gives the query and the gate in one row
        qg = normal(rows, 2, hq, D).to(dt)
        st["q"] = qg[:, 0]
        st["gate"] = qg[:, 1] if case["gate"] else None
        kv = normal(cells, 2, hkv, D).to(dt)
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
        return st
    n = _rows(case, length)
    page, hkv = case["page"], case["hkv"]
    used = -(-length // page)
    width = int(used.max())
    pages = int(used.sum()) + 3
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(pages)
    table = np.full((case["nseq"], width), -1, np.int64)
    table[np.arange(width)[None, :] < used[:, None]] = order[: int(used.sum())]
    rows = int(n.sum())
    st.update(table=ints(table), kv_len=ints(length), cu=ints(_cu(n)), max_q=int(n.max()), max_len=int(length.max()),
              page=page, rows=rows)
    if case["op"] == "cache":
        st["ck"] = torch.zeros(pages, page, hkv, D, dtype=torch.int8, device="cuda")
        st["cv"] = torch.zeros_like(st["ck"])
        st["ks"] = torch.zeros(pages, page, hkv, NG, dtype=torch.float16, device="cuda")
        st["vs"] = torch.zeros_like(st["ks"])
        kv = normal(rows, 2, hkv, D).to(dt)   # one projection row holds a token's K and V
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
        return st
    for name, scales in (("ck", "ks"), ("cv", "vs")):
        # normal rows quantised at their group's maximum: codes of about 127 / 2.3 deviations
        codes = torch.empty(pages, page, hkv, D, dtype=torch.int8, device="cuda")
        for part in codes.split(max(1, (1 << 27) // (page * hkv * D))):
            part.copy_((normal(*part.shape) * 55).round_().clamp_(-127, 127))
        st[name] = codes
        st[scales] = (torch.rand(pages, page, hkv, NG, generator=gen, device="cuda") * 0.012 + 0.012).half()
    if case["op"] == "decode":
        st["hq"] = case["hq"]
        st["q"] = normal(rows, case["hq"], D).to(dt)
        st["gate"] = normal(rows, case["hq"], D).to(dt) if case["gate"] else None
    return st


# ------------------------------------------------------------------ the framework's calls

def _own(st):
    from top_sparse_attention_score_b200 import qsa
    if st["op"] == "prompt":
        return qsa.prompt_attn(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], scale=SCALE, gate=st["gate"])
    if "cache" not in st:  # a server keeps its cache and its batch
        st["cache"] = qsa.PagedCache(st["ck"], st["cv"], st["ks"], st["vs"])
        st["batch"] = qsa.Batch(st["table"], st["kv_len"], st["cu"])
    cache, batch = st["cache"], st["batch"]
    if st["op"] == "decode":
        return qsa.paged_decode(cache, batch, st["q"], scale=SCALE, max_q=st["max_q"], max_len=st["max_len"],
                                gate=st["gate"])
    if st["op"] == "cache":
        qsa.paged_write(cache, batch, st["k"], st["v"])
    return qsa.paged_read(cache, batch, st["rows"], st["dtype"])


# ------------------------------------------------------------------ the plain forms

def _row_positions(st):
    """For each packed row: its sequence and its position."""
    cu, length = st["cu"].long(), st["kv_len"].long()
    r = torch.arange(st["rows"], device=cu.device)
    s = torch.searchsorted(cu[1:], r, right=True)
    return s, length[s] - cu[s + 1] + r


def _cells(st, s, p):
    """The cache cell of position p of sequence s (any shapes that broadcast)."""
    page = st["table"].long()[s, p // st["page"]].clamp(min=0)
    return page * st["page"] + p % st["page"]


def _values(codes, scales, cell):
    """Dequantised rows of the given cells: [..., hkv, 256] in fp32."""
    hkv = codes.shape[2]
    c = codes.view(-1, hkv, NG, GROUP)[cell].float()
    return (c * scales.view(-1, hkv, NG, 1)[cell].float()).flatten(-2)


def _quantise(x):
    g = x.float().unflatten(-1, (NG, GROUP))
    s = (g.abs().amax(-1) / 127.0).clamp(max=65504.0).half()
    f = s.float().unsqueeze(-1)
    code = torch.where(f > 0, torch.round(g / torch.where(f > 0, f, 1.0)), 0.0).clamp(-127, 127)
    return code.flatten(-2).to(torch.int8), s


def _attend(q, k, v, seen, gate):
    """q [S, n, hq, D], k / v [S, m, hkv, D], seen [S, n]: keys each row sees (below the first
    when it is <= 0).  In fp32; a row that sees nothing is 0."""
    S, n, hq, _ = q.shape
    m, hkv = k.shape[1], k.shape[2]
    grp = hq // hkv
    qq = q.view(S, n, hkv, grp, D).permute(0, 2, 1, 3, 4).reshape(S, hkv, n * grp, D)
    kk, vv = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    s = torch.matmul(qq, kk.transpose(-1, -2)).mul_(SCALE).view(S, hkv, n, grp, m)
    hidden = torch.arange(m, device=q.device) >= seen[:, :, None]
    s.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, hkv, n * grp, m), vv).view(S, hkv, n, grp, D)
    o = torch.where(total > 0, o / total.clamp(min=1e-30), 0.0).permute(0, 2, 1, 3, 4).reshape(S, n, hq, D)
    return o if gate is None else o * torch.sigmoid(gate.float())


def _padded(cu, width, most):
    """Index [S, width] of packed rows, clamped into the arrays."""
    at = cu[:-1, None] + torch.arange(width, device=cu.device)
    return at.clamp(max=most - 1)


def _unpack(cu, rows, o):
    """Padded results [S, n, ...] as packed rows."""
    r = torch.arange(rows, device=cu.device)
    s = torch.searchsorted(cu[1:], r, right=True)
    return o[s, r - cu[s]]


def _plain(st):
    dt = st["dtype"]
    if st["op"] == "prompt":
        q, k, v, gate = st["q"], st["k"], st["v"], st["gate"]
        cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
        at_q, at_k = _padded(cu_q, st["max_q"], q.shape[0]), _padded(cu_k, st["max_k"], k.shape[0])
        n, m = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
        seen = (m - n)[:, None] + 1 + torch.arange(st["max_q"], device=q.device)
        o = _attend(q[at_q].float(), k[at_k].float(), v[at_k].float(), torch.minimum(seen, m[:, None]),
                    None if gate is None else gate[at_q])
        return _unpack(cu_q, q.shape[0], o).to(dt)
    if st["op"] == "decode":
        cu, length = st["cu"].long(), st["kv_len"].long()
        S = length.shape[0]
        p = torch.arange(st["max_len"], device=cu.device)[None, :]
        cell = _cells(st, torch.arange(S, device=cu.device)[:, None], p)
        at = _padded(cu, st["max_q"], st["rows"])
        n = cu[1:] - cu[:-1]
        seen = (length - n)[:, None] + 1 + torch.arange(st["max_q"], device=cu.device)
        o = _attend(st["q"][at].float(), _values(st["ck"], st["ks"], cell), _values(st["cv"], st["vs"], cell),
                    torch.minimum(seen, length[:, None]), None if st["gate"] is None else st["gate"][at])
        return _unpack(cu, st["rows"], o).to(dt)
    s, p = _row_positions(st)
    cell = _cells(st, s, p)
    hkv = st["hkv"]
    if st["op"] == "cache":
        for x, codes, scales in ((st["k"], st["ck"], st["ks"]), (st["v"], st["cv"], st["vs"])):
            c, sc = _quantise(x)
            codes.view(-1, hkv, D)[cell] = c
            scales.view(-1, hkv, NG)[cell] = sc
    return _values(st["ck"], st["ks"], cell).to(dt), _values(st["cv"], st["vs"], cell).to(dt)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits, sequence by sequence

def _exact_attention(q, k, v, gate):
    """One sequence: q [n, hq, D], k / v [m, hkv, D] in fp64; row i sees keys <= i + m - n."""
    n, hq, _ = q.shape
    m, hkv = k.shape[0], k.shape[1]
    out = torch.zeros_like(q)
    hide = torch.arange(m, device=q.device)[None, :] > torch.arange(n, device=q.device)[:, None] + (m - n)
    for h in range(hq):
        g = h // (hq // hkv)
        logits = (q[:, h] @ k[:, g].T) * SCALE
        logits[hide] = -math.inf
        out[:, h] = torch.softmax(logits, dim=-1) @ v[:, g]
    return out if gate is None else out / (1.0 + torch.exp(-gate.double()))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prompt":
        outs = []
        cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
        for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
            outs.append(_exact_attention(st["q"][a:b].double(), st["k"][c:d].double(), st["v"][c:d].double(),
                                         None if st["gate"] is None else st["gate"][a:b]))
        return torch.cat(outs)
    table, length, cu = st["table"].cpu().numpy(), st["kv_len"].tolist(), st["cu"].tolist()
    page = st["page"]

    def cells(s, first, last):
        p = np.arange(first, last)
        return torch.from_numpy(table[s, p // page].astype(np.int64) * page + p % page).cuda()

    def held(codes, scales, at):
        c = codes.reshape(-1, *codes.shape[2:])[at].double()
        return c * scales.reshape(-1, *scales.shape[2:])[at].double().repeat_interleave(GROUP, dim=-1)

    if case["op"] == "decode":
        outs = []
        for s in range(len(length)):
            a, b = cu[s], cu[s + 1]
            at = cells(s, 0, length[s])
            outs.append(_exact_attention(st["q"][a:b].double(), held(st["ck"], st["ks"], at), held(st["cv"], st["vs"], at),
                                         None if st["gate"] is None else st["gate"][a:b]))
        return torch.cat(outs)
    if case["op"] == "read":
        at = torch.cat([cells(s, length[s] - (cu[s + 1] - cu[s]), length[s]) for s in range(len(length))])
        return held(st["ck"], st["ks"], at), held(st["cv"], st["vs"], at)
    got = []
    for x in (st["k"], st["v"]):
        g = x.float().cpu().numpy().reshape(-1, GROUP)
        # the quantiser is defined by its fp32 quotients; everything after them is exact in 64 bits
        s = np.minimum(np.abs(g).max(-1) / np.float32(127), np.float32(65504)).astype(np.float16)
        f = s.astype(np.float32)[:, None]
        code = np.rint(np.divide(g, f, out=np.zeros_like(g), where=f > 0)).clip(-127, 127)
        got.append(torch.from_numpy((code.astype(np.float64) * f.astype(np.float64)).reshape(x.shape)))
    return tuple(got)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(3)]:
        print(c.get("name", "drawn"), work(c))
