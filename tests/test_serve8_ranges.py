"""Attention over the 8-bit cache where a row's weights lie far apart, against binary64.

A key may take nearly all of a row's weight and add nothing to the result (its value codes are 0): an attention sink.
A page may have a large V scale from one channel and zero codes in the others. In both, the result is formed by small
weights, so it shows how many bits they keep."""
import math

import pytest
import torch

from test_serve8 import U16, UB, U32, Layer, check_attention, gen, i32, ss  # noqa: F401 (ss: the fixture)

pytestmark = pytest.mark.gpu

# (head size, page, query heads, new tokens): few rows, one CTA's row tiles, pairs of CTAs
FORMS = [(128, 64, 4, 1), (64, 16, 4, 1), (64, 16, 4, 40), (128, 32, 2, 50), (128, 64, 4, 100)]


def flat_layer(ss, fmt, d, page, keys, seed):  # noqa: F811
    """One sequence of `keys` tokens; K's first channel 0, scales such that unit queries give logits of order 1."""
    layer = Layer(ss, fmt, d, page, 1, keys, 1, seed=seed).fill([keys], seed)
    for n in ("k", "v"):
        layer.cache[n + "_scales"].fill_(1 / (50 if fmt == "int" else 200))
    layer.cache["k"][..., 0] = 0
    return layer


def key_at(layer, j):
    return int(layer.order[0, j // layer.page]), j % layer.page


def compare(ss, layer, q, keys, unit, channels=None, causal=False, table=None, seen=None, error=0):  # noqa: F811
    """Elements against their bound and, with `channels`, those channels' norm. unit: a small weight's absolute error
    over the largest weight among its keys, where that weight is far above all others. table: another page table than
    the layer's, with which only the keys `seen` are seen and the error word is `error`."""
    new, heads, d = q.shape
    ws = ss.Workspace()
    table = layer.table([keys]) if table is None else table
    out, lse = ss.kv_attention(q, layer.cache, table, i32([0, new]), i32([keys]), causal=causal, max_new=new,
                               max_len=keys, lse=True, ws=ws)
    assert ws.error() == error
    k, v = layer.values("k", 0, keys)[:, 0], layer.values("v", 0, keys)[:, 0]
    z = q.double().view(-1, d) @ k.T * d**-0.5
    there = torch.ones(new, keys, dtype=torch.bool, device="cuda") if seen is None else seen.expand(new, keys)
    if causal:
        at = keys - new + torch.arange(new, device="cuda")
        there = there & (torch.arange(keys, device="cuda") <= at[:, None])
    there = there[:, None].expand(new, heads, keys).reshape(-1, keys)
    z = z.masked_fill(~there, -math.inf)
    none = ~there.any(1)
    p = torch.softmax(z, -1).nan_to_num(0.0)
    ref = p @ v
    got = out.double().view(-1, d)
    assert bool((got[none] == 0).all()) and bool((lse.view(-1)[none] == -math.inf).all())
    # Roundings. Of the result: half a bf16 step. Of a weight: half an fp16 step, 2^-11, or below 2^-14 half of fp16's
    # least step, 2^-25 of the reference 2^M. With W the largest weight among the keys taken together (at most 128
    # aligned ones) M is at most log2 W + 9: 2^-16 W, for weights below 2^-5 W. Where no key before has a larger
    # weight, M is at most log2 W - 5: 2^-30 W. Of the exponents: as in check_attention. Of n sums in binary32.
    page_of = torch.arange(keys, device="cuda") // layer.page
    s_v = layer.cache["v_scales"][torch.from_numpy(layer.order[0]).cuda().long()[page_of], 0].double()
    w = p * s_v
    pad = max(-keys % 128, 256 - keys)  # two blocks at least
    block = torch.nn.functional.pad(w, (0, pad)).view(w.shape[0], -1, 128).amax(2)
    first, second = block.topk(2, 1).values.T
    alone = (block == first[:, None]) & (first > 2.0**8 * second)[:, None]
    lost = (torch.where(alone, unit, 2.0**-16) * block).repeat_interleave(128, 1)[:, :keys]
    small = w < 2.0**-5 * block.repeat_interleave(128, 1)[:, :keys]
    floor = (lost * small) @ (v / s_v[:, None]).abs()
    big = (q.double().view(-1, d).abs() @ k.abs().T).amax(1, keepdim=True) * d**-0.5
    dz = (d + 8) * 2 * U32 * big + 8 * U32 * (big + 20.0) + 2.0**-21
    tol = UB * ref.abs() + (p @ v.abs()) * (2 * dz + U16 + 2 * keys * U32) + floor
    assert bool(((got - ref).abs() <= tol).all()), float(((got - ref).abs() / tol).max())
    lse_ref = torch.logsumexp(z, -1)
    off = (lse.double().view(-1) - lse_ref).abs() <= dz[:, 0] + 2 * keys * U32 + 4 * U32 * lse_ref.abs()
    assert bool(off[~none].all())
    # A result of many small terms of both signs: bf16's rounding is at most UB of the norm, the weights' roundings are
    # independent of each other and each at most U16 of its term, so that their sum's norm is about U16 / sqrt(3) of
    # the result's; four U16 leave room for the exponents' roundings.
    if channels is not None:
        channels = list(channels)
        got, ref = got[:, channels], ref[:, channels]
        assert float((got - ref).norm() / ref.norm()) <= UB + 4 * U16


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page,heads,new", FORMS)
@pytest.mark.parametrize("keys,mass", [(8192, 0.99), (8192, 0.999), (32768, 0.99), (5003, 0.9999)])
def test_a_sink_without_a_value(ss, fmt, d, page, heads, new, keys, mass):  # noqa: F811
    layer = flat_layer(ss, fmt, d, page, keys, 1)
    at, slot = key_at(layer, 0)
    layer.cache["k"][at, 0, slot] = 0
    layer.cache["k"][at, 0, slot, 0] = 127 if fmt == "int" else 0x7E  # the largest code: 127, 448
    layer.cache["v"][at, 0, slot] = 0
    q = torch.randn(new, heads, d, generator=gen(2), device="cuda") * 0.3
    q[..., 0] = math.log(keys * mass / (1 - mass)) * d**0.5 / (127 / 50 if fmt == "int" else 448 / 200)
    compare(ss, layer, q.bfloat16(), keys, 2.0**-30, range(d))
    layer.cache["v_scales"].fill_(2.0**-40)
    compare(ss, layer, q.bfloat16(), keys, 2.0**-30, range(d))


@pytest.mark.parametrize("d,page,heads,new", FORMS)
@pytest.mark.parametrize("place", [0, 700, 4095])
def test_equal_keys_beside_a_sink(ss, d, page, heads, new, place):  # noqa: F811
    """All other keys and values alike: a rounding of their common weight does not average out. The sink comes first, in
    the midst or last, 2^14 to 2^26 above them."""
    keys = 4096
    layer = flat_layer(ss, "int", d, page, keys, 3)
    layer.cache["k"].zero_()
    layer.cache["v"].copy_(torch.arange(d, device="cuda") - 40)
    at, slot = key_at(layer, place)
    layer.cache["k"][at, 0, slot, 0] = 127
    layer.cache["v"][at, 0, slot] = 0
    for bits in (14.45, 18.3, 23.6, 26.0):
        q = torch.zeros(new, heads, d, device="cuda")
        q[..., 0] = bits * math.log(2) * d**0.5 * 50 / 127
        compare(ss, layer, q.bfloat16(), keys, 2.0**-30, range(d))


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page,heads,new", FORMS)
@pytest.mark.parametrize("ratio", [2.0**9, 2.0**14, 2.0**20])
def test_one_channel_sets_a_page_s_scale(ss, fmt, d, page, heads, new, ratio):  # noqa: F811
    # the page's own keys are less than 4 bits apart: where some are taken after others, M is at most log2 W - 1: 2^-26 W
    keys = 8192
    layer = flat_layer(ss, fmt, d, page, keys, 4)
    at, slot = key_at(layer, 1024 + 7)
    layer.cache["v"][at] = 0
    layer.cache["v"][at, 0, slot, 5] = 127 if fmt == "int" else 0x7E
    layer.cache["v_scales"][at] *= ratio
    others = [c for c in range(d) if c != 5]
    q = torch.randn(new, heads, d, generator=gen(5), device="cuda") * 0.3
    compare(ss, layer, q.bfloat16(), keys, 2.0**-26, others)


@pytest.mark.parametrize("d,page,heads,new", FORMS)
def test_weights_that_rise_and_fall(ss, d, page, heads, new):  # noqa: F811
    """Logits in runs up to 60 bits apart, up and down, with page scales that undo or double the steps."""
    keys = 6000
    layer = flat_layer(ss, "int", d, page, keys, 6)
    g = gen(7)
    per = torch.randint(-100, 101, (layer.pages,), generator=g, device="cuda")
    layer.cache["k"][..., 0] = per[:, None, None].to(torch.int8)
    layer.cache["v_scales"].mul_(2.0 ** torch.randint(-20, 21, layer.cache["v_scales"].shape, generator=g, device="cuda"))
    for bits in (10.0, 30.0, -60.0):
        q = torch.randn(new, heads, d, generator=g, device="cuda") * 0.3
        q[..., 0] = bits * math.log(2) * d**0.5 * 50 / 100
        compare(ss, layer, q.bfloat16(), keys, 2.0**-16)


@pytest.mark.parametrize("d,page,heads,new", FORMS)
def test_tiny_and_huge_value_scales(ss, d, page, heads, new):  # noqa: F811
    """The sums stay in binary32's range: V scales of 2^-100 and 2^120, logits that fall by 35 bits behind a first key."""
    keys = 3000
    layer = flat_layer(ss, "int", d, page, keys, 8)
    at, slot = key_at(layer, 0)
    layer.cache["k"][at, 0, slot] = 0
    layer.cache["k"][at, 0, slot, 0] = 127
    q = torch.randn(new, heads, d, generator=gen(9), device="cuda") * 0.3
    q[..., 0] = 35 * math.log(2) * d**0.5 * 50 / 127
    q = q.bfloat16()
    for scale in (2.0**-100, 2.0**-60, 2.0**120):
        layer.cache["v_scales"].fill_(scale)
        # alike at every scale, as powers of two pass through the arithmetic
        out = ss.kv_attention(q, layer.cache, layer.table([keys]), i32([0, new]), i32([keys]), max_new=new, max_len=keys)
        layer.cache["v_scales"].fill_(1.0)
        one = ss.kv_attention(q, layer.cache, layer.table([keys]), i32([0, new]), i32([keys]), max_new=new, max_len=keys)
        assert bool(torch.isfinite(out.float()).all())
        assert float((out.double() / scale - one.double()).norm() / one.double().norm()) <= 2 * UB


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page,heads,new", FORMS)
@pytest.mark.parametrize("bits", [125, 118, 113, -113, -119])
def test_queries_of_any_magnitude(ss, fmt, d, page, heads, new, bits):  # noqa: F811
    """Finite queries up to bf16's largest and down to its smallest normal ones, on K scales that bring the logits back
    to order 1."""
    keys = 300
    layer = Layer(ss, fmt, d, page, 1, keys, 1, seed=10).fill([keys], 10)
    layer.cache["k_scales"].mul_(2.0**-bits)
    q = torch.randn(new, heads, d, generator=gen(11), device="cuda").clamp_(-7, 7)
    q = (q * 2.0**(bits - (bits == 125))).bfloat16()
    if bits == 125:
        q[0, 0, 0] = torch.finfo(torch.bfloat16).max
    assert bool(torch.isfinite(q).all())
    ws = ss.Workspace()
    out, lse = ss.kv_attention(q, layer.cache, layer.table([keys]), i32([0, new]), i32([keys]), max_new=new, max_len=keys,
                               lse=True, ws=ws)
    assert ws.error() == 0
    check_attention(layer, q, out, lse, [0, new], [keys], True, d**-0.5)


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page,heads,new", FORMS + [(128, 64, 7, 700)])
@pytest.mark.parametrize("keys", [200, 6000])
def test_a_query_of_nan_shows(ss, fmt, d, page, heads, new, keys):  # noqa: F811
    """In one part of the key axis and in several: the row's result and lse are NaN, not those of a row without keys,
    and no other row changes."""
    keys = max(keys, new)
    layer = Layer(ss, fmt, d, page, 1, keys, 1, seed=12).fill([keys], 12)
    q = torch.randn(new, heads, d, generator=gen(13), device="cuda").bfloat16()
    where = (layer.table([keys]), i32([0, new]), i32([keys]))
    good, good_lse = ss.kv_attention(q, layer.cache, *where, max_new=new, max_len=keys, lse=True)
    bad = q.clone()
    bad[new // 2, heads - 1] = math.nan
    out, lse = ss.kv_attention(bad, layer.cache, *where, max_new=new, max_len=keys, lse=True)
    assert bool(out[new // 2, heads - 1].isnan().all()) and bool(lse[new // 2, heads - 1].isnan())
    out[new // 2, heads - 1], lse[new // 2, heads - 1] = good[new // 2, heads - 1], good_lse[new // 2, heads - 1]
    # a CTA's other rows: their reference may move with a neighbour's vote, which scales by powers of two
    assert float((out.float() - good.float()).abs().max()) <= float(good.float().abs().max()) * UB
    assert torch.equal(lse.isfinite(), good_lse.isfinite())


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page,heads,new", FORMS + [(128, 16, 3, 1), (64, 32, 8, 1), (128, 128, 1, 600)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_page_outside_the_cache_counts_as_no_keys(ss, fmt, d, page, heads, new, causal):  # noqa: F811
    """First, last, neighbouring and all page numbers bad: as if their keys were masked, a row that sees no others like
    one without keys. The unused table entries stay out of range."""
    for keys in (max(new, 5 * page + 3), 3000):
        pages = -(-keys // page)
        layer = flat_layer(ss, fmt, d, page, keys, 14)
        q = (torch.randn(new, heads, d, generator=gen(15), device="cuda") * 0.3).bfloat16()
        for bad in ([0], [pages - 1], [1, 4], [2, 3], range(0, pages, 2), range(1, pages, 2), range(pages)):
            bad = list(bad)
            table = layer.table([keys])
            table[0, bad] = torch.tensor([(layer.pages, -1, 1 << 30)[i % 3] for i in bad], dtype=torch.int32, device="cuda")
            seen = torch.ones(pages, dtype=torch.bool, device="cuda")
            seen[bad] = False
            compare(ss, layer, q, keys, 2.0**-16, causal=causal, table=table, seen=seen.repeat_interleave(page)[:keys],
                    error=16)


@pytest.mark.parametrize("d,page,heads,new", FORMS)
@pytest.mark.parametrize("keys", [200, 3000])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_up_to_2_to_the_23(ss, d, page, heads, new, keys, sign):  # noqa: F811
    """Logits near +-2^23, some pages' up to 14 bits above the others', where binary32 has steps of 1: every weight stays
    finite, so that values that are alike within a column give themselves."""
    layer = flat_layer(ss, "int", d, page, keys, 17)
    layer.cache["k"].fill_(100)
    layer.cache["v"].copy_(torch.arange(d, device="cuda") - 40)
    more = torch.randint(0, 12, layer.cache["k_scales"].shape, generator=gen(18), device="cuda")
    layer.cache["k_scales"].copy_((1 / 50 + more.double() * (2.0**-23 / 50)).float())
    q = torch.full((new, heads, d), float(sign), device="cuda").bfloat16()
    z = float(d * 100 / 50 * (1 + 12 * 2.0**-23))
    out, lse = ss.kv_attention(q, layer.cache, layer.table([keys]), i32([0, new]), i32([keys]), scale=0.999 * 2**23 / z,
                               causal=False, max_new=new, max_len=keys, lse=True)
    ref = (torch.arange(d, device="cuda").double() - 40) / 50
    # the V scale 1 / 50 is rounded, a weight to 2^-11, the sums of n terms, the result
    assert bool(((out.double() - ref).abs() <= ref.abs() * (UB + U16 + 2 * keys * U32)).all())
    assert bool(((lse.double() / sign - 2**23).abs() <= 2**23 * 0.01).all())
