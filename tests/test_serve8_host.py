"""Host-side checks of the 8-bit serving entry points (INT8 product, paged cache append, attention): invalid
arguments are rejected before anything is enqueued. No test here launches a kernel."""
import ctypes

import pytest
import torch

from semi_structured_sparsity_online_b200 import ss24

ALIGNED, ODD = 0x7F0000000000, 0x7F0000000008  # never dereferenced
OK, NULL, SHAPE, ALIGN, DTYPE, FORMAT, WORKSPACE, ARG = 0, 1, 2, 3, 4, 5, 6, 8


def ws_bytes():
    return ss24.lib().ss24_workspace_bytes()


def gemm(a=ALIGNED, sa=ALIGNED, b=ALIGNED, sb=ALIGNED, m=4, n=8, k=64, y=ALIGNED, dt=ss24.BF16, ldy=None, ws=ALIGNED,
         wsb=None):
    return ss24.lib().ss24_gemm_int8(a, sa, b, sb, m, n, k, y, dt, n if ldy is None else ldy, ws,
                                     ws_bytes() if wsb is None else wsb, None)


@pytest.mark.parametrize("kw,expected", [
    (dict(dt=7), DTYPE), (dict(m=-1), SHAPE), (dict(n=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=24), SHAPE),
    (dict(k=131072), SHAPE), (dict(ldy=7), SHAPE), (dict(a=None), NULL), (dict(sa=None), NULL), (dict(b=None), NULL),
    (dict(sb=None), NULL), (dict(y=None), NULL), (dict(a=ODD), ALIGN), (dict(b=ODD), ALIGN), (dict(sa=ODD + 2), ALIGN),
    (dict(y=ODD + 1), ALIGN), (dict(y=ODD + 2, dt=ss24.F32), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(wsb=16), WORKSPACE), (dict(ws=ALIGNED + 16), WORKSPACE), (dict(m=0, a=None), OK), (dict(n=0, b=None), OK),
])
def test_gemm_int8_rejects(kw, expected):
    assert gemm(**kw) == expected


def cache(**kw):
    c = dict(k=ALIGNED, v=ALIGNED, k_scales=ALIGNED, v_scales=ALIGNED, kind=ss24.FMT_INT, page=64, pages=10, kv_heads=2,
             head_dim=128)
    c.update(kw)
    return ss24.KvCache(*(c[n] for n, _ in ss24.KvCache._fields_))


def batch(**kw):
    b = dict(page_table=ALIGNED, starts=ALIGNED, lengths=ALIGNED, seqs=3, table_ld=4, tokens=5, max_new=2, max_len=200)
    b.update(kw)
    return ss24.KvBatch(*(b[n] for n, _ in ss24.KvBatch._fields_))


def rows(heads=2, **kw):
    r = dict(x=ALIGNED, dtype=ss24.BF16, heads=heads, token_stride=heads * 128, head_stride=128)
    r.update(kw)
    return ss24.HeadRows(*(r[n] for n, _ in ss24.HeadRows._fields_))


def append(c=None, b=None, k=None, v=None, ws=ALIGNED):
    c, b, k, v = c or cache(), b or batch(), k or rows(), v or rows()
    return ss24.lib().ss24_kv_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(k), ctypes.byref(v), ws, ws_bytes(),
                                     None)


def attend(q=None, c=None, b=None, out=None, scale=0.1, causal=1, lse=None, scratch=ALIGNED, room=1 << 40, ws=ALIGNED):
    q, c, b, out = q or rows(4), c or cache(), b or batch(), out or rows(4)
    return ss24.lib().ss24_kv_attention(ctypes.byref(q), ctypes.byref(c), ctypes.byref(b), scale, causal,
                                        ctypes.byref(out), lse, scratch, room, ws, ws_bytes(), None)


CACHES = [
    (dict(kind=ss24.FMT_NVFP4), FORMAT), (dict(kind=ss24.FMT_NONE), FORMAT), (dict(page=8), SHAPE),
    (dict(page=48), SHAPE), (dict(page=256), SHAPE), (dict(head_dim=96), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(pages=-1), SHAPE), (dict(k=None), NULL), (dict(v_scales=None), NULL), (dict(v=ODD), ALIGN),
    (dict(k_scales=ODD + 2), ALIGN),
]
BATCHES = [
    (dict(seqs=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(max_new=6), SHAPE), (dict(max_new=-1), SHAPE),
    (dict(max_len=257), SHAPE), (dict(max_len=-1), SHAPE), (dict(table_ld=-1), SHAPE), (dict(max_len=2**31 - 1), SHAPE),
    (dict(starts=None), NULL), (dict(lengths=None), NULL), (dict(page_table=None), NULL), (dict(starts=ODD + 1), ALIGN),
]


@pytest.mark.parametrize("kw,expected", CACHES)
def test_cache_is_checked(kw, expected):
    assert append(c=cache(**kw)) == expected and attend(c=cache(**kw)) == expected
    assert ss24.lib().ss24_kv_attention_scratch_bytes(ctypes.byref(cache(**kw)), ctypes.byref(batch()), 4) == -1


@pytest.mark.parametrize("kw,expected", BATCHES)
def test_batch_is_checked(kw, expected):
    assert append(b=batch(**kw)) == expected and attend(b=batch(**kw)) == expected
    assert ss24.lib().ss24_kv_attention_scratch_bytes(ctypes.byref(cache()), ctypes.byref(batch(**kw)), 4) == -1


def test_rows_are_checked():
    assert append(k=rows(4)) == SHAPE                                   # not the cache's heads
    assert append(k=rows(dtype=ss24.F32), v=rows()) == DTYPE            # k and v of two types
    assert append(k=rows(dtype=5)) == DTYPE
    assert append(k=rows(x=None)) == NULL and append(v=rows(x=ODD)) == ALIGN
    assert append(k=rows(token_stride=100)) == SHAPE and append(k=rows(token_stride=260)) == ALIGN
    assert append(k=rows(head_stride=64)) == SHAPE and append(k=rows(head_stride=132)) == ALIGN
    assert attend(q=rows(3), out=rows(3)) == SHAPE                      # 3 query heads on 2 KV heads
    assert attend(q=rows(4), out=rows(2)) == SHAPE
    assert attend(q=rows(4, dtype=ss24.F32)) == DTYPE and attend(out=rows(4, dtype=ss24.F32)) == DTYPE
    assert attend(q=rows(4, x=None)) == NULL and attend(out=rows(4, x=None)) == NULL
    assert attend(scale=float("nan")) == ARG and attend(scale=float("inf")) == ARG and attend(causal=2) == ARG
    assert attend(lse=ODD + 2) == ALIGN and attend(ws=None) == WORKSPACE and append(ws=None) == WORKSPACE


def test_null_descriptors():
    L, z = ss24.lib(), None
    c, b, r = ctypes.byref(cache()), ctypes.byref(batch()), ctypes.byref(rows())
    assert L.ss24_kv_append(z, b, r, r, ALIGNED, ws_bytes(), None) == NULL
    assert L.ss24_kv_append(c, z, r, r, ALIGNED, ws_bytes(), None) == NULL
    assert L.ss24_kv_append(c, b, z, r, ALIGNED, ws_bytes(), None) == NULL
    assert L.ss24_kv_attention(z, c, b, 0.1, 1, r, None, ALIGNED, 1 << 40, ALIGNED, ws_bytes(), None) == NULL
    assert L.ss24_kv_attention(r, c, b, 0.1, 1, z, None, ALIGNED, 1 << 40, ALIGNED, ws_bytes(), None) == NULL


def test_scratch_is_checked_and_empty_calls_launch_nothing():
    long = batch(table_ld=2048, max_len=131072, tokens=3, max_new=1)
    need = ss24.lib().ss24_kv_attention_scratch_bytes(ctypes.byref(cache()), ctypes.byref(long), 4)
    assert need > 0
    assert attend(b=long, scratch=None) == WORKSPACE and attend(b=long, room=need - 1) == WORKSPACE
    assert attend(b=long, scratch=ODD) == WORKSPACE
    none = dict(page_table=None, starts=None, lengths=None, seqs=0, tokens=0, max_new=0, max_len=0)
    for b in (batch(**none), batch(tokens=0, max_new=0), batch(max_new=0)):
        assert append(b=b, k=rows(x=None), v=rows(x=None)) == OK
        assert attend(b=b, q=rows(4, x=None), out=rows(4, x=None)) == OK
        assert ss24.lib().ss24_kv_attention_scratch_bytes(ctypes.byref(cache()), ctypes.byref(b), 4) == 0
    assert append(b=batch(max_len=0), k=rows(x=None), v=rows(x=None)) == OK  # nothing has a place


def test_python_checks_before_the_library():
    i8 = {"values": torch.zeros(4, 64, dtype=torch.int8), "scales": torch.ones(4, 1)}
    with pytest.raises(ValueError, match="differ in k"):
        ss24.gemm_int8(i8, {"values": torch.zeros(4, 32, dtype=torch.int8), "scales": torch.ones(4, 1)})
    with pytest.raises(ValueError, match="int8"):
        ss24.gemm_int8({"values": torch.zeros(4, 64), "scales": torch.ones(4, 1)}, i8)
    with pytest.raises(ValueError, match="contiguous int8"):
        ss24.gemm_int8({"values": torch.zeros(64, 4, dtype=torch.int8).t(), "scales": torch.ones(4, 1)}, i8)
    with pytest.raises(ValueError, match="one per row"):
        ss24.gemm_int8({"values": i8["values"], "scales": torch.ones(4, 2)}, i8)
    with pytest.raises(TypeError, match="y must be"):
        ss24.gemm_int8(i8, i8, dtype=torch.float16)
    with pytest.raises(ValueError, match="y must be"):
        ss24.gemm_int8(i8, i8, y=torch.zeros(4, 5))
    with pytest.raises(ValueError, match="format"):
        ss24.kv_cache(2, 1, 64, fmt="nvfp4", device="cpu")
    c = ss24.kv_cache(4, 2, 64, page=16, device="cpu")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    where = (i32(0, 1).view(1, 2), i32(0, 3), i32(20))
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="differ in shape"):
        ss24.kv_append(c, x, x[:2], *where)
    with pytest.raises(ValueError, match="must be .tokens, heads, 64"):
        ss24.kv_append(c, x[..., :32], x[..., :32], *where)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        ss24.kv_append(c, x.half(), x.half(), *where)
    with pytest.raises(ValueError, match="starts must be int32"):
        ss24.kv_append(c, x, x, where[0], where[1].long(), where[2])
    with pytest.raises(ValueError, match="starts must be int32"):
        ss24.kv_append(c, x, x, where[0], i32(0, 1, 3), where[2])
    with pytest.raises(ValueError, match="max_len"):
        ss24.kv_append(c, x, x, *where, max_len=33)
    with pytest.raises(ValueError, match="page_table must have contiguous rows"):
        ss24.kv_append(c, x, x, i32(0, 0, 0, 0).view(2, 2).t(), i32(0, 1, 3), i32(5, 5))
    with pytest.raises(ValueError, match="codes must be contiguous"):
        ss24.kv_append({**c, "k": c["k"].float()}, x, x, *where)
    with pytest.raises(ValueError, match="scales must be contiguous"):
        ss24.kv_append({**c, "v_scales": c["v_scales"][:2]}, x, x, *where)
