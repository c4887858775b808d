"""A wait of a serving kernel that runs out, made on purpose (the SS24_TEST_SKIP_TILE hook: the first CTA leaves out one
copy or hand-over, waits give up after 10 ms): the call returns, the error word says so, and the next call is right."""
import time

import pytest
import torch

from test_serve8 import Layer, attend, check_product, gen, i32, int8_operand, ss  # noqa: F401 (ss: the fixture)

pytestmark = pytest.mark.gpu


def runs_out(ss, monkeypatch, call, skip, code):  # noqa: F811
    ws = ss.Workspace()
    call(ws)  # the kernels are loaded
    torch.cuda.synchronize()
    assert ws.error() == 0
    monkeypatch.setenv("SS24_TEST_SKIP_TILE", str(skip))
    t0 = time.perf_counter()
    call(ws)
    assert ws.error() == code
    assert time.perf_counter() - t0 < 1.5  # 10 ms a wait, not two seconds
    monkeypatch.delenv("SS24_TEST_SKIP_TILE")


# the split product without and with a cluster, more and fewer stages than its ring; the product by pairs likewise
@pytest.mark.parametrize("m,n,k,skip", [(1, 300, 256, 1), (1, 300, 1920, 2), (1, 4096, 4096, 3), (40, 512, 4096, 0),
                                        (100, 4096, 1024, 7), (260, 9800, 256, 1), (260, 9800, 2048, 9),
                                        (2000, 9800, 1024, 8)])
def test_a_product_gives_up(ss, monkeypatch, m, n, k, skip):  # noqa: F811
    a, b = int8_operand(m, k, 1), int8_operand(n, k, 2)
    runs_out(ss, monkeypatch, lambda ws: ss.gemm_int8(a, b, ws=ws), skip, 14)
    check_product(ss.gemm_int8(a, b), a, b)


# few rows in one part and in several; one CTA's row tiles and pairs, one row tile and two, one part and several
@pytest.mark.parametrize("d,group,new,keys", [(64, 4, 1, 500), (128, 4, 1, 500), (64, 8, 2, 9000), (128, 1, 1, 20000),
                                              (64, 1, 40, 900), (64, 4, 60, 900), (128, 1, 100, 3000), (128, 2, 100, 700),
                                              (128, 4, 90, 700), (128, 4, 128, 5000)])
@pytest.mark.parametrize("skip", [0, 1])
def test_attention_gives_up(ss, monkeypatch, d, group, new, keys, skip):  # noqa: F811
    layer = Layer(ss, "int", d, 64, 1, keys, 1, seed=1).fill([keys])
    q = torch.randn(new, group, d, generator=gen(2), device="cuda").bfloat16()
    where = (layer.table([keys]), i32([0, new]), i32([keys]))
    kw = dict(max_new=new, max_len=keys)
    runs_out(ss, monkeypatch, lambda ws: ss.kv_attention(q, layer.cache, *where, ws=ws, **kw), skip, 15)
    attend(ss, layer, [keys], [new], group, True, seed=3, spare=0, **kw)
