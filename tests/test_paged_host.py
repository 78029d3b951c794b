"""Host-side checks of the batched calls: the C ABI refuses bad arguments before it touches a
GPU, its workspace sizes, and the binding's checks of shapes, types and strides."""
import ctypes

import pytest
import torch

OK, ARG, WORKSPACE = 0, 1, 2
P = 0x100000


@pytest.fixture(scope="module")
def lib():
    from top_sparse_attention_score_b200 import build, qsa
    build.build()
    return qsa.load()


def paged(**kw):
    from top_sparse_attention_score_b200 import qsa
    a = dict(k=P, v=P, ks=P, vs=P, pages=10, page_cells=16, hkv=2)
    a.update(kw)
    return qsa.PagedCacheStruct(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page_cells"], a["hkv"])


def batch(**kw):
    from top_sparse_attention_score_b200 import qsa
    a = dict(table=P, kv_len=P, cu_q=P, nseq=3, table_ld=4)
    a.update(kw)
    return qsa.BatchStruct(a["table"], a["kv_len"], a["cu_q"], a["nseq"], a["table_ld"])


def write(lib, c=None, b=None, rows=5, dtype=0, k=P, ldk=512, v=P, ldv=512, fn="qsa_paged_write"):
    c, b = c or paged(), b or batch()
    return getattr(lib, fn)(ctypes.byref(c), ctypes.byref(b), rows, dtype, k, ldk, v, ldv, None)


@pytest.mark.parametrize("fn", ["qsa_paged_write", "qsa_paged_read"])
def test_write_and_read_refuse(lib, fn):
    from top_sparse_attention_score_b200 import qsa
    assert getattr(lib, fn)(None, ctypes.byref(batch()), 5, 0, P, 512, P, 512, None) == ARG
    assert getattr(lib, fn)(ctypes.byref(paged()), None, 5, 0, P, 512, P, 512, None) == ARG
    for c in (paged(k=None), paged(vs=None), paged(ks=P + 8), paged(pages=0), paged(page_cells=0), paged(hkv=0),
              paged(hkv=1025), paged(pages=1 << 20, page_cells=1 << 11)):
        assert write(lib, c=c, fn=fn) == ARG and "cache" in qsa.last_error()
    for b in (batch(table=None), batch(kv_len=None), batch(nseq=0), batch(nseq=65536), batch(table_ld=0)):
        assert write(lib, b=b, fn=fn) == ARG and "batch" in qsa.last_error()
    assert write(lib, rows=-1, fn=fn) == ARG and "rows" in qsa.last_error()
    assert write(lib, rows=(1 << 24) + 1, fn=fn) == ARG
    assert write(lib, dtype=3, fn=fn) == ARG and "dtype" in qsa.last_error()
    assert write(lib, k=None, fn=fn) == ARG
    assert write(lib, v=P + 4, fn=fn) == ARG and "aligned" in qsa.last_error()
    assert write(lib, ldk=511, fn=fn) == ARG and "stride" in qsa.last_error()
    assert write(lib, dtype=1, ldv=516, fn=fn) == ARG           # 1032 bytes
    assert write(lib, rows=0, k=None, v=None, fn=fn) == OK      # nothing to do, nothing launched


def decode(lib, c=None, b=None, rows=5, max_q=2, max_len=64, dtype=0, hq=24, q=P, ldq=24 * 256, gate=None, ldg=0, ws=P,
           ws_bytes=1 << 40, out=P, ldo=24 * 256, scale=0.0625):
    c, b = c or paged(), b or batch()
    return lib.qsa_paged_decode(ctypes.byref(c), ctypes.byref(b), rows, max_q, max_len, dtype, hq, q, ldq, gate, ldg,
                                scale, ws, ws_bytes, out, ldo, None)


def test_decode_refuses(lib):
    from top_sparse_attention_score_b200 import qsa
    assert decode(lib, max_q=0) == ARG
    assert decode(lib, max_q=9) == ARG and "max_q" in qsa.last_error()
    assert decode(lib, hq=25) == ARG and "multiple" in qsa.last_error()
    assert decode(lib, hq=0) == ARG
    assert decode(lib, hq=26, max_q=8, ldq=26 * 256, ldo=26 * 256) == ARG and "96" in qsa.last_error()
    assert decode(lib, max_len=0) == ARG
    assert decode(lib, b=batch(nseq=65535), max_len=(1 << 31) - 1) == ARG   # the flat block list
    assert decode(lib, c=paged(pages=0)) == ARG
    assert decode(lib, dtype=-1) == ARG
    assert decode(lib, q=P + 2) == ARG
    assert decode(lib, out=None) == ARG
    assert decode(lib, gate=P, ldg=100) == ARG and "gate" in qsa.last_error()
    for scale in (0.0, -0.0625, float("nan"), float("inf"), 2.0e30):
        assert decode(lib, scale=scale) == ARG and "scale" in qsa.last_error()
        assert prompt(lib, scale=scale) == ARG and "scale" in qsa.last_error()
    assert decode(lib, ws=None) == WORKSPACE
    assert decode(lib, ws=P + 8) == ARG
    assert decode(lib, rows=0, q=None, out=None) == OK


def test_decode_workspace(lib):
    f = lib.qsa_paged_decode_workspace_bytes
    assert f(0, 24, 2, 1, 100) == 0 and f(1, 25, 2, 1, 100) == 0 and f(1, 24, 2, 9, 100) == 0 and f(1, 24, 2, 1, 0) == 0
    small, long_, drafts, many = f(1, 24, 2, 1, 64), f(1, 24, 2, 1, 262144), f(1, 24, 2, 8, 262144), f(1000, 24, 2, 8, 262144)
    assert 0 < small < long_ < drafts < many
    assert many - drafts <= 1000 * 2 * 8 + 4096   # the partials do not grow with the sequences


def prompt(lib, nseq=2, cu_q=P, cu_k=P, rows_q=300, rows_k=300, dtype=2, hq=24, hkv=2, q=P, ldq=24 * 256, k=P, ldk=512,
           v=P, ldv=512, gate=None, ldg=0, ws=P, ws_bytes=1 << 40, out=P, ldo=24 * 256, scale=0.0625):
    return lib.qsa_prompt_attn(nseq, cu_q, cu_k, rows_q, rows_k, dtype, hq, hkv, q, ldq, k, ldk, v, ldv, gate, ldg, scale,
                               ws, ws_bytes, out, ldo, None)


def test_prompt_refuses(lib):
    from top_sparse_attention_score_b200 import qsa
    assert prompt(lib, dtype=0) == ARG and "QSA_F16" in qsa.last_error()
    assert prompt(lib, nseq=0) == ARG
    assert prompt(lib, cu_k=None) == ARG
    assert prompt(lib, hq=23) == ARG
    assert prompt(lib, rows_q=-1) == ARG
    assert prompt(lib, rows_k=(1 << 24) + 1) == ARG
    assert prompt(lib, q=P + 8) == ARG
    assert prompt(lib, k=None) == ARG
    assert prompt(lib, ldv=500) == ARG
    assert prompt(lib, gate=P, ldg=6000) == ARG
    assert prompt(lib, out=None) == ARG
    need = lib.qsa_prompt_attn_workspace_bytes(1, 16, 32768, 24, 2)
    assert need > 0
    assert prompt(lib, nseq=1, rows_q=16, rows_k=32768, ws_bytes=need - 1) == WORKSPACE
    assert prompt(lib, nseq=1, rows_q=16, rows_k=32768, ws=None) == WORKSPACE
    assert prompt(lib, nseq=1, rows_q=16, rows_k=32768, ws=P + 8) == ARG
    assert lib.qsa_prompt_attn_workspace_bytes(1, 8192, 8192, 24, 2) == 0   # rows enough for the GPU
    assert prompt(lib, rows_q=0, q=None, out=None) == OK


def test_binding_refuses():
    """The binding's own checks, on CPU tensors and fake caches."""
    from top_sparse_attention_score_b200 import qsa
    z = torch.zeros(2, 4, 2, 256, dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.PagedCache(z, z, z, z)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.Batch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    x = torch.zeros(5, 2, 256, dtype=torch.float16)
    assert qsa._packed(x, 2, torch.float16, x.device, "x") == (x.data_ptr(), 512)
    wide = torch.zeros(5, 3, 2, 256, dtype=torch.float16)[:, 1]
    assert qsa._packed(wide, 2, torch.float16, wide.device, "x")[1] == 1536
    assert qsa._packed(wide[:1], 2, torch.float16, wide.device, "x")[1] == 512   # one row has no stride
    for bad, text in ((x[:, :, :128], "256"), (x[:, :1], "rows"), (x.float(), "float16"), (x.transpose(0, 1), "rows"),
                      (x.view(5, 256, 2).transpose(1, 2), "contiguous"), (x[0], "rows")):
        with pytest.raises(ValueError, match=text):
            qsa._packed(bad, 2, torch.float16, x.device, "x")
    with pytest.raises(ValueError, match="float32"):
        qsa._dtype_code(torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.prompt_attn(x, x, x, torch.zeros(2, dtype=torch.int32))
