"""The 8-bit serving operators on the GPU against plain implementations in 64 bits: the INT8 product, new tokens into
the paged 8-bit cache, attention over it, and the three in a row as an attention layer uses them.

Tolerances count roundings: u32 = 2^-24 (binary32), u16 = 2^-11 (fp16), ub = 2^-8 (bf16)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U32, U16, UB = 2.0**-24, 2.0**-11, 2.0**-8


@pytest.fixture(scope="module")
def ss():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from semi_structured_sparsity_online_b200 import ss24
    ss24.lib()
    return ss24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# the INT8 product
# ---------------------------------------------------------------------------

def int8_operand(rows, k, seed):
    g = gen(seed)
    v = torch.randint(-127, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    return {"values": v, "scales": torch.rand(rows, 1, generator=g, device="cuda") * 0.01}


def check_product(y, a, b):
    ref = (a["values"].double() @ b["values"].double().T) * a["scales"].double() * b["scales"].double().T
    # the sum and the two scales each round once to binary32, bf16 once more
    tol = ref.abs() * (3.01 * U32 + (UB if y.dtype == torch.bfloat16 else 0.0))
    assert y.shape == ref.shape and bool(((y.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 128, 128), (2, 129, 144), (15, 40, 4096), (16, 257, 48),
                                   (17, 1000, 272), (33, 64, 1024), (64, 384, 112), (65, 127, 2064), (128, 128, 512),
                                   (129, 300, 96), (255, 513, 640), (256, 256, 256), (257, 1001, 1040),
                                   (700, 4100, 160), (3, 20000, 64), (5000, 3, 32), (513, 2049, 2000)])
def test_gemm_int8(ss, m, n, k, dtype):
    a, b = int8_operand(m, k, 1), int8_operand(n, k, 2)
    ws = ss.Workspace()
    check_product(ss.gemm_int8(a, b, dtype=dtype, ws=ws), a, b)
    assert ws.error() == 0


@pytest.mark.parametrize("m,n,k", [(4, 4, 131056), (300, 200, 131056)])
def test_gemm_int8_sum_is_exact_at_its_largest(ss, m, n, k):
    """Every product 127^2 (or 128^2): the sum is near 2^31 and any lost carry shows."""
    one = torch.ones(1, device="cuda")
    for code, sign in ((127, 1), (-128, 1), (127, -1)):
        a = {"values": torch.full((m, k), code, dtype=torch.int8, device="cuda"), "scales": one.expand(m, 1).contiguous()}
        b = {"values": torch.full((n, k), sign * code, dtype=torch.int8, device="cuda"),
             "scales": one.expand(n, 1).contiguous()}
        y = ss.gemm_int8(a, b, dtype=torch.float32)
        assert bool((y == float(np.float32(sign * code * code * k))).all())


@pytest.mark.parametrize("m,n", [(1, 70), (40, 130), (300, 515)])
def test_gemm_int8_fills_a_slice_and_nothing_else(ss, m, n):
    a, b = int8_operand(m, 64, 3), int8_operand(n, 64, 4)
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((m + 2, n + 9), 7.0, dtype=dtype, device="cuda")
        y = wide[1:m + 1, 5:5 + n]
        assert ss.gemm_int8(a, b, y=y) is y
        check_product(y, a, b)
        edge = wide.clone()
        edge[1:m + 1, 5:5 + n] = 7.0
        assert bool((edge == 7.0).all())


def test_gemm_int8_empty_and_zero(ss):
    a, b = int8_operand(0, 64, 5), int8_operand(10, 64, 6)
    assert ss.gemm_int8(a, b).shape == (0, 10) and ss.gemm_int8(b, a).shape == (10, 0)
    a = int8_operand(3, 64, 7)
    a["scales"].zero_()
    assert bool((ss.gemm_int8(a, b, dtype=torch.float32) == 0).all())


def test_gemm_int8_takes_the_quantizers_rows(ss):
    """Codes and scales as the INT8 pass with one scale per row writes them."""
    x = torch.randn(37, 1024, generator=gen(8), device="cuda").bfloat16()
    w = (torch.randn(200, 1024, generator=gen(9), device="cuda") * 0.02).bfloat16()
    a, b = (ss.run(t, pattern=ss.DENSE, fmt="int", bits=8) for t in (x, w))
    y = ss.gemm_int8(a, b, dtype=torch.float32)
    check_product(y, a, b)
    assert float((y - x.float() @ w.float().T).norm() / (x.float() @ w.float().T).norm()) < 0.02


def test_gemm_int8_allocates_for_the_stream_it_runs_on(ss):
    a, b = int8_operand(70, 4096, 12), int8_operand(4096, 4096, 13)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    ys = [ss.gemm_int8(a, b, dtype=torch.float32, stream=s) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(s)
    for y in ys:
        check_product(y, a, b)


def test_gemm_int8_on_another_stream_and_replayed(ss):
    a, b = int8_operand(20, 512, 10), int8_operand(300, 512, 11)
    ws = ss.Workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y1 = torch.empty(20, 300, device="cuda")
    ss.gemm_int8(a, b, y=y1, ws=ws, stream=s)
    y2 = torch.empty_like(y1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.gemm_int8(a, b, y=y2, ws=ws)
    a["values"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y1, -y2)
    check_product(y2, a, b)


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------

class Layer:
    """A paged cache and its sequences; pages in a shuffled order, unused slots and pages full of NaN or of the
    largest codes, unused table entries out of range."""

    def __init__(self, ss, fmt, d, page, kv_heads, most, seqs, seed):
        self.rng = np.random.default_rng(seed)
        per = max(1, -(-most // page))
        self.pages = per * seqs + 2
        self.fmt, self.d, self.page, self.heads = fmt, d, page, kv_heads
        self.cache = ss.kv_cache(self.pages, kv_heads, d, page=page, fmt=fmt)
        for n in ("k", "v"):
            self.cache[n].fill_(127 if fmt == "int" else 0x7F)  # E4M3 0x7F is NaN
            self.cache[n + "_scales"].fill_(math.nan)
        self.order = self.rng.permutation(self.pages)[:per * seqs].reshape(seqs, per).astype(np.int32)

    def table(self, lens):
        t = self.order.copy()
        for s, n in enumerate(lens):
            t[s, -(-n // self.page):] = 1 << 30
        return torch.from_numpy(t).cuda()

    def fill(self, lens, seed=0):
        """Codes and scales of cached tokens, written directly (E4M3: every finite code)."""
        g = gen(seed)
        for n in ("k", "v"):
            shape = self.cache[n].shape
            if self.fmt == "int":
                c = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
            else:
                c = torch.randint(0, 127, shape, generator=g, device="cuda").to(torch.uint8)
                c += (torch.randint(0, 2, shape, generator=g, device="cuda") * 128).to(torch.uint8)
            for s, length in enumerate(lens):
                for p in range(-(-length // self.page)):
                    live = min(self.page, length - p * self.page)
                    where = int(self.order[s, p])
                    self.cache[n][where, :, :live] = c[where, :, :live]
                    spread = 2.0 ** (torch.rand(self.heads, generator=g, device="cuda") * 6 - 3)
                    self.cache[n + "_scales"][where] = spread / (100 if self.fmt == "int" else 200)
        return self

    def values(self, name, s, length):
        """[length, heads, d] in binary64."""
        out = torch.empty(0, self.heads, self.d, dtype=torch.float64, device="cuda")
        parts = [out]
        for p in range(-(-length // self.page)):
            where = int(self.order[s, p])
            c = self.cache[name][where]
            c = c if self.fmt == "int" else c.view(torch.float8_e4m3fn).float()
            v = c.double() * self.cache[name + "_scales"][where].double()[:, None, None]
            parts.append(v.transpose(0, 1)[:length - p * self.page])
        return torch.cat(parts)


def quantize(x, s, fmt):
    """The library's codes, by IEEE binary32 divisions on the host."""
    q = np.divide(x, s, out=np.zeros_like(x), where=s > 0)
    if fmt == "int":
        return np.clip(np.rint(q), -127, 127).astype(np.int8)
    return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def decode(c, fmt):
    return c.astype(np.float32) if fmt == "int" else torch.from_numpy(c).view(torch.float8_e4m3fn).float().numpy()


def append_reference(layer, before, x, starts, lens, name):
    codes, scales = before[name].copy(), before[name + "_scales"].copy()
    top = np.float32(127 if layer.fmt == "int" else 448)
    for s, length in enumerate(lens):
        begin = length - (starts[s + 1] - starts[s])
        for p in range(max(begin, 0) // layer.page, -(-length // layer.page)):
            lo, hi = max(begin, p * layer.page), min(length, (p + 1) * layer.page)
            if lo >= hi:
                continue
            where, fill = layer.order[s, p], lo - p * layer.page
            t = x[starts[s] + lo - begin:starts[s] + hi - begin].transpose(1, 0, 2)
            new = np.abs(t).max((1, 2)) / top
            if fill:
                had = scales[where].copy()
                new = np.fmax(new, had)  # a NaN scale (no older token was written) counts as none
                grew = new > had
                old = decode(codes[where, :, :fill], layer.fmt) * had[:, None, None]
                codes[where, grew, :fill] = quantize(old, new[:, None, None], layer.fmt)[grew]
            codes[where, :, fill:fill + hi - lo] = quantize(t, new[:, None, None], layer.fmt)
            scales[where] = new
    return codes, scales


def host(cache):
    return {n: cache[n].cpu().numpy() for n in ("k", "v", "k_scales", "v_scales")}


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page,heads", [(128, 64, 2), (64, 16, 3), (128, 128, 1), (64, 128, 2), (128, 16, 8),
                                          (64, 32, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_bit_for_bit(ss, fmt, d, page, heads, dtype):
    """Calls one after the other: a prompt, single tokens (pages fill, scales grow), ragged pieces; every code and
    scale of the whole cache, the untouched ones too, equals the host's binary32 arithmetic."""
    seqs, most = 4, 3 * page + 5
    layer = Layer(ss, fmt, d, page, heads, most, seqs, seed=page)
    ws = ss.Workspace()
    lens = [0] * seqs
    g = gen(page + d)
    for step, news in enumerate([[page + 3, 1, 0, page], [1, 1, 1, 1], [1, 0, 1, 1], [page, 5, 2 * page, 0], [1, 1, 1, 1]]):
        lens = [a + b for a, b in zip(lens, news)]
        starts = np.concatenate([[0], np.cumsum(news)])
        x = {n: (torch.randn(int(starts[-1]) + 2, heads, d, generator=g, device="cuda") * (1 + 3 * step)).to(dtype)
             for n in ("k", "v")}
        x["v"][0] = 0.0
        before = host(layer.cache)
        ss.kv_append(layer.cache, x["k"], x["v"], layer.table(lens), i32(starts.tolist()), i32(lens), max_new=max(news),
                     ws=ws)
        after = host(layer.cache)
        for n in ("k", "v"):
            codes, scales = append_reference(layer, before, x[n].float().cpu().numpy(), starts, lens, n)
            assert np.array_equal(after[n].view(np.uint8), codes.view(np.uint8)), (step, n)
            assert np.array_equal(after[n + "_scales"].view(np.int32), scales.view(np.int32)), (step, n)
        # the same call once more changes nothing
        ss.kv_append(layer.cache, x["k"], x["v"], layer.table(lens), i32(starts.tolist()), i32(lens), ws=ws)
        again = host(layer.cache)
        assert all(np.array_equal(after[n].view(np.uint8), again[n].view(np.uint8)) for n in after)
    assert ws.error() == 0


def test_append_strided_slices_of_one_projection(ss):
    """k and v as slices of a fused projection's output, heads not packed."""
    layer, other = (Layer(ss, "int", 64, 16, 2, 40, 1, seed=1) for _ in range(2))
    qkv = torch.randn(37, 8, 64, generator=gen(2), device="cuda").bfloat16()
    where = (layer.table([37]), i32([0, 37]), i32([37]))
    ss.kv_append(layer.cache, qkv[:, 4:8:2], qkv[:, 5:8:2], *where)
    ss.kv_append(other.cache, qkv[:, 4:8:2].contiguous(), qkv[:, 5:8:2].contiguous(), *where)
    a, b = host(layer.cache), host(other.cache)
    assert all(np.array_equal(a[n].view(np.uint8), b[n].view(np.uint8)) for n in a)


def test_append_extreme_scales(ss):
    """Scales outside the corrected reciprocal's range, largest bf16 values, zeros."""
    for fmt in ("int", "fp8"):
        layer = Layer(ss, fmt, 64, 16, 1, 64, 1, seed=3)
        x = torch.randn(64, 1, 64, generator=gen(4), device="cuda")
        x[:16] *= 2.0**-110
        x[16:32] *= 2.0**100
        x[32:48] = 0.0
        x = x.bfloat16()
        before = host(layer.cache)
        ss.kv_append(layer.cache, x, -x, layer.table([64]), i32([0, 64]), i32([64]))
        after = host(layer.cache)
        for n, t in (("k", x), ("v", -x)):
            codes, scales = append_reference(layer, before, t.float().cpu().numpy(), [0, 64], [64], n)
            assert np.array_equal(after[n].view(np.uint8), codes.view(np.uint8))
            assert np.array_equal(after[n + "_scales"].view(np.int32), scales.view(np.int32))


def test_append_leaves_out_what_breaks_a_bound(ss):
    """Bad pages and bounds: recorded, and nothing else of the cache changes; more new tokens than the length drop the
    first ones."""
    x = torch.randn(12, 1, 64, generator=gen(5), device="cuda").bfloat16()
    for bad in ("page", "count", "length", "order"):
        layer = Layer(ss, "int", 64, 16, 1, 32, 2, seed=6)
        table, starts, lens, max_new = layer.table([20, 4]), [0, 8, 12], [20, 4], 8
        if bad == "page":
            table[0, 1] = layer.pages
        elif bad == "count":
            max_new = 7
        elif bad == "length":
            lens[0] = 33
        else:
            starts[0] = 9
        ws = ss.Workspace()
        before = host(layer.cache)
        ss.kv_append(layer.cache, x, x, table, i32(starts), i32(lens), max_new=max_new, ws=ws)
        assert ws.error() == (16 if bad == "page" else 17)
        after = host(layer.cache)
        for n in ("k", "v"):
            if bad == "page":  # the first page of sequence 0 got its tokens, the second had no place
                t = x.float().cpu().numpy()
                codes, scales = append_reference(layer, before, np.concatenate([t[:4], t[8:]]), [0, 4, 8], [16, 4], n)
            else:
                codes, scales = append_reference(layer, before, x[8:].float().cpu().numpy(), [0, 0, 4], [0, 4], n)
            if bad in ("page", "count", "length"):
                assert np.array_equal(after[n], codes)
                assert np.array_equal(after[n + "_scales"].view(np.int32), scales.view(np.int32))
    layer = Layer(ss, "int", 64, 16, 1, 32, 1, seed=7)
    ws = ss.Workspace()
    before = host(layer.cache)
    ss.kv_append(layer.cache, x, x, layer.table([5]), i32([0, 12]), i32([5]), ws=ws)
    codes, scales = append_reference(layer, before, x.float().cpu().numpy(), [0, 12], [5], "k")
    assert ws.error() == 0 and np.array_equal(host(layer.cache)["k"], codes)


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------

def check_attention(layer, q, out, lse, starts, lens, causal, scale):
    """Against binary64, with a bound from the roundings named in the header: q's and the codes' products are exact in
    binary32, D of them are summed; the exponent takes a few binary32 roundings of |z|, of log2 s_v and of the
    reference point; a weight rounds to fp16 (and below 2^-14 of the largest by 2^-25 of it); n products are summed in
    binary32; the result rounds to bf16."""
    d = layer.d
    group = q.shape[1] // layer.heads
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        if n == 0:
            continue
        t = slice(starts[s], starts[s + 1])
        k, v = layer.values("k", s, length), layer.values("v", s, length)
        x = q[t].double().view(n, layer.heads, group, d)
        z = torch.einsum("nhgd,lhd->nhgl", x, k) * scale
        mag = torch.einsum("nhgd,lhd->nhgl", x.abs(), k.abs()) * abs(scale)
        seen = torch.ones(n, length, dtype=torch.bool, device="cuda")
        if causal:
            seen = torch.arange(length, device="cuda") <= (length - n + torch.arange(n, device="cuda"))[:, None]
        z = z.masked_fill(~seen[:, None, None], -math.inf)
        none = ~seen.any(1)
        p = torch.softmax(z, -1).nan_to_num(0.0) if length else z
        ref = torch.einsum("nhgl,lhd->nhgd", p, v)
        ref_lse = torch.logsumexp(z, -1) if length else torch.full((n, layer.heads, group), -math.inf).cuda().double()
        got = out[t].double().view(n, layer.heads, group, d)
        got_lse = lse[t].double().view(n, layer.heads, group)
        assert bool((got[none] == 0).all()) and bool((got_lse[none] == -math.inf).all())
        if not length or bool(none.all()):
            continue
        live = ~none
        big = mag.masked_fill(~seen[:, None, None], 0.0).amax(-1)
        # absolute error of an exponent, in natural units
        dz = (d + 8) * 2 * U32 * big + 8 * U32 * (big + 20.0) + 2.0**-21
        spread = torch.einsum("nhgl,lhd->nhgd", p, v.abs())
        largest = v.abs().amax(0).amax(-1)[None, :, None, None]
        tol = UB * ref.abs() + spread * (2 * dz[..., None] + U16 + 2 * length * U32) + length * 2.0**-25 * largest
        assert bool(((got - ref).abs() <= tol)[live].all()), float(((got - ref).abs() / tol)[live].max())
        tol = dz + 2 * length * U32 + 4 * U32 * ref_lse.abs()
        assert bool(((got_lse - ref_lse).abs() <= tol)[live].all()), float(((got_lse - ref_lse).abs() / tol)[live].max())


def attend(ss, layer, lens, news, group, causal, seed=0, scale=None, spare=2, ws=None, **kw):
    starts = np.concatenate([[0], np.cumsum(news)]).tolist()
    heads = layer.heads * group
    q = torch.randn(starts[-1] + spare, heads, layer.d, generator=gen(seed), device="cuda").bfloat16()
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    ws = ws or ss.Workspace()
    ss.kv_attention(q, layer.cache, layer.table(lens), i32(starts), i32(lens), causal=causal, scale=scale, out=out,
                    lse=lse, ws=ws, **kw)
    assert ws.error() == 0
    assert bool((out[starts[-1]:] == 5.0).all()) and bool((lse[starts[-1]:] == 5.0).all())
    check_attention(layer, q, out, lse, starts, lens, causal, layer.d**-0.5 if scale is None else scale)
    return q, out, lse


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,heads,group", [(16, 1, 1), (64, 2, 4), (32, 3, 7), (128, 1, 8), (64, 2, 12), (16, 1, 32)])
@pytest.mark.parametrize("tight", [True, False])
def test_attention_single_tokens(ss, fmt, d, page, heads, group, tight):
    """One new token each over lengths around tiles, pages and parts; a sequence without keys, one without tokens."""
    lens = [1, 2, 15, 16, 17, page - 1, page, page + 1, 0, 300, 700, 129]
    news = [1] * 8 + [1, 0, 1, 1]
    layer = Layer(ss, fmt, d, page, heads, 1100, len(lens), seed=d + page).fill(lens)
    bounds = dict(max_new=1, max_len=max(lens)) if tight else {}
    for causal in (True, False):
        attend(ss, layer, lens, news, group, causal, **bounds)


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page,heads,group", [(128, 64, 2, 4), (64, 16, 1, 7), (64, 128, 2, 1), (128, 32, 1, 8),
                                                (128, 16, 1, 3), (64, 32, 1, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_many_tokens(ss, fmt, d, page, heads, group, causal):
    """Prompts and pieces of them, ragged; more new tokens than keys leave rows empty."""
    lens = [1, 5, 130, 128, 127, 400, 3, 0, 257, 640]
    news = [1, 5, 130, 100, 33, 1, 9, 4, 257, 70]
    layer = Layer(ss, fmt, d, page, heads, max(lens), len(lens), seed=d * page).fill(lens)
    attend(ss, layer, lens, news, group, causal, max_new=max(news), max_len=max(lens))


@pytest.mark.parametrize("fmt", ["int", "fp8"])
@pytest.mark.parametrize("d,page", [(128, 16), (128, 64), (64, 16), (64, 128)])
@pytest.mark.parametrize("rows", [9, 16, 17, 25, 32, 33, 127, 128, 129, 255, 256, 257, 511, 512, 513, 640])
def test_attention_row_counts_around_tiles(ss, fmt, d, page, rows):
    """One KV head, one query head: as many rows as new tokens, next to a single token, over a cached prefix."""
    lens, news = [rows + 45, 7, rows], [rows, 1, rows - 1]
    layer = Layer(ss, fmt, d, page, 1, max(lens), 3, seed=rows).fill(lens)
    attend(ss, layer, lens, news, 1, True, max_new=rows, max_len=max(lens))


@pytest.mark.parametrize("seqs", [257, 600])
def test_attention_more_sequences_than_threads(ss, seqs):
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 40, seqs).tolist()
    layer = Layer(ss, "int", 64, 16, 1, 40, seqs, seed=19).fill(lens)
    attend(ss, layer, lens, [1] * seqs, 2, True, max_new=1, max_len=40)


@pytest.mark.parametrize("new", [1, 50])
def test_a_slice_of_a_wider_page_table(ss, new):
    lens = [90, 120]
    layer = Layer(ss, "int", 64, 16, 1, 128, 2, seed=21).fill(lens)
    q = torch.randn(2 * new, 2, 64, generator=gen(1), device="cuda").bfloat16()
    starts, table = i32([0, new, 2 * new]), layer.table(lens)
    wide = torch.full((2, 3 * table.shape[1]), 1 << 30, dtype=torch.int32, device="cuda")
    part = wide[:, 5:5 + table.shape[1]]
    part.copy_(table)
    a = ss.kv_attention(q, layer.cache, table, starts, i32(lens))
    b = ss.kv_attention(q, layer.cache, part, starts, i32(lens))
    assert torch.equal(a, b)


@pytest.mark.parametrize("new", [1, 20, 40])
def test_attention_without_keys_or_pages(ss, new):
    """No sequence has a key; a cache without pages."""
    for pages in (3, 0):
        cache = ss.kv_cache(pages, 2, 64, page=16)
        q = torch.randn(2 * new, 4, 64, generator=gen(1), device="cuda").bfloat16()
        for width in (1, 0):
            table = torch.full((2, width), 99, dtype=torch.int32, device="cuda")
            out, lse = ss.kv_attention(q, cache, table, i32([0, new, 2 * new]), i32([0, 0]), lse=True)
            assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("fmt,d,group,new", [("int", 128, 4, 1), ("fp8", 64, 8, 1), ("fp8", 128, 4, 40), ("int", 64, 1, 17)])
def test_attention_long_context(ss, fmt, d, group, new):
    """Few rows over many keys: the key axis is split and joined; a short sequence beside a long one."""
    lens, news = [9001, 40, 5000], [new, min(new, 2), new]
    layer = Layer(ss, fmt, d, 64, 1, max(lens), 3, seed=11).fill(lens)
    attend(ss, layer, lens, news, group, True, max_new=new, max_len=max(lens))


@pytest.mark.parametrize("fmt,d,heads,group", [("int", 128, 3, 7), ("fp8", 64, 1, 20), ("int", 64, 5, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_chunks_in_parts(ss, fmt, d, heads, group, causal):
    """Thousands of rows and a split key axis; a sequence shorter than a part, one with rows that see no key."""
    lens, news = [2500, 130, 90], [151, 130, 100]
    layer = Layer(ss, fmt, d, 32, heads, max(lens), 3, seed=d + heads).fill(lens)
    attend(ss, layer, lens, news, group, causal, max_new=max(news), max_len=max(lens))


@pytest.mark.parametrize("new", [1, 50])
def test_attention_far_apart_values(ss, new):
    """Logits hundreds apart, page scales up to 2^40 apart, zero scales, a query row of zeros, a large scale."""
    lens = [300, 90]
    for fmt in ("int", "fp8"):
        layer = Layer(ss, fmt, 128, 16, 1, 300, 2, seed=12).fill(lens)
        for s, length in enumerate(lens):
            for p in range(-(-length // 16)):
                where = int(layer.order[s, p])
                layer.cache["v_scales"][where] *= 2.0 ** ((p * 7) % 41 - 20)
                if p % 5 == 4:
                    layer.cache["v"][where] = 0
                    layer.cache["v_scales"][where] = 0.0
        attend(ss, layer, lens, [new, new], 4, True, scale=0.5)
        attend(ss, layer, lens, [new, new], 4, True, scale=-0.25)
        attend(ss, layer, lens, [new, new], 4, True, scale=0.0)


@pytest.mark.parametrize("new", [1, 30])
def test_attention_strides_and_heads_major_output(ss, new):
    lens, news = [70, 33], [new, new]
    layer = Layer(ss, "int", 64, 16, 2, 70, 2, seed=13).fill(lens)
    q, out, lse = attend(ss, layer, lens, news, 3, True)
    wide = torch.zeros(q.shape[0], 12, 80, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2, 8:72] = q
    major = torch.zeros(6, q.shape[0], 64, dtype=torch.bfloat16, device="cuda")
    n = 2 * new
    got = ss.kv_attention(wide[:, ::2, 8:72], layer.cache, layer.table(lens), i32([0, new, n]), i32(lens),
                          out=major.transpose(0, 1))
    assert torch.equal(got[:n], out[:n]) and bool((major[:, n:] == 0).all())


@pytest.mark.parametrize("new", [1, 40])
def test_attention_records_bad_pages_and_bounds(ss, new):
    lens = [100, 60]
    layer = Layer(ss, "int", 64, 16, 1, 112, 2, seed=14).fill(lens)
    q = torch.randn(2 * new, 4, 64, generator=gen(1), device="cuda").bfloat16()
    starts = i32([0, new, 2 * new])
    good = ss.kv_attention(q, layer.cache, layer.table(lens), starts, i32(lens), max_new=new, max_len=112)
    for bad in ("page", "negative page", "length", "count"):
        table, l, st, most = layer.table(lens), i32(lens), starts, new
        if bad == "page":
            table[0, 2] = layer.pages
        elif bad == "negative page":
            table[0, 3] = -5
        elif bad == "length":
            l = i32([113, 60])
        else:
            st = i32([-1, new, 2 * new])
        ws = ss.Workspace()
        out = ss.kv_attention(q, layer.cache, table, st, l, max_new=most, max_len=112, ws=ws)
        assert ws.error() == (16 if "page" in bad else 17)
        assert torch.equal(out[new:], good[new:])  # the other sequence
    # a page that counts as no keys: as if those 16 keys were masked
    assert bool(torch.isfinite(out[new:].float()).all())


@pytest.mark.parametrize("new", [1, 40, 1200])
def test_attention_in_parts_leaves_out_a_sequence_that_breaks_a_bound(ss, new):
    """Where the key axis is split, the rows of a bad sequence are left as they were, too."""
    lens = [6000, 5000]
    layer = Layer(ss, "int", 64, 64, 1, 6000, 2, seed=20).fill(lens)
    q = torch.randn(2 * new + 3, 2, 64, generator=gen(2), device="cuda").bfloat16()
    table, starts = layer.table(lens), i32([0, new, 2 * new])
    good, good_lse = ss.kv_attention(q, layer.cache, table, starts, i32(lens), max_new=new, max_len=6000, lse=True)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    ws = ss.Workspace()
    ss.kv_attention(q, layer.cache, table, starts, i32([6001, 5000]), max_new=new, max_len=6000, out=out, lse=lse, ws=ws)
    assert ws.error() == 17
    assert bool((out[:new] == 5.0).all()) and bool((lse[:new] == 5.0).all())
    assert torch.equal(out[new:2 * new], good[new:2 * new]) and torch.equal(lse[new:2 * new], good_lse[new:2 * new])
    assert bool((out[2 * new:] == 5.0).all()) and bool((lse[2 * new:] == 5.0).all())


@pytest.mark.parametrize("fmt", ["int", "fp8"])
def test_a_cache_beyond_4_gib(ss, fmt):
    """Pages whose codes lie past 2^32 bytes: written, read by few rows, by many and in parts."""
    page, heads, d = 128, 8, 128
    pages = (1 << 32) // (page * heads * d) + 40
    dt = torch.int8 if fmt == "int" else torch.uint8
    cache = {n: torch.empty(pages, heads, page, d, dtype=dt, device="cuda") for n in ("k", "v")}
    cache.update({n: torch.zeros(pages, heads, device="cuda") for n in ("k_scales", "v_scales")})
    cache.update(page=page, fmt=fmt)
    small = ss.kv_cache(24, heads, d, page=page, fmt=fmt)
    length = 24 * page - 5
    x = torch.randn(length, 2 * heads, d, generator=gen(3), device="cuda").bfloat16()
    where = (i32([0, length]), i32([length]))
    far = torch.arange(pages - 24, pages, dtype=torch.int32, device="cuda").view(1, 24)
    near = torch.arange(24, dtype=torch.int32, device="cuda").view(1, 24)
    ss.kv_append(cache, x[:, :heads], x[:, heads:], far, *where)
    ss.kv_append(small, x[:, :heads], x[:, heads:], near, *where)
    for n in ("k_scales", "v_scales"):
        assert torch.equal(cache[n][pages - 24:], small[n])
    for new in (1, 20, 300):
        q = torch.randn(new, 2 * heads, d, generator=gen(4), device="cuda").bfloat16()
        st = i32([0, new])
        a = ss.kv_attention(q, cache, far, st, where[1], max_len=length, lse=True)
        b = ss.kv_attention(q, small, near, st, where[1], max_len=length, lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("new", [1, 20])
def test_attention_replayed_with_new_contents(ss, new):
    """A captured call follows the lengths, tables and cache it finds; two graphs share a workspace."""
    lens = [200, 90]
    layer = Layer(ss, "fp8", 128, 32, 1, 512, 2, seed=15).fill([512, 512])
    table = torch.from_numpy(layer.order).cuda()
    starts, l = i32([0, new, 2 * new]), i32(lens)
    q = torch.randn(2 * new, 4, 128, generator=gen(3), device="cuda").bfloat16()
    ws = ss.Workspace()
    outs, graphs = [], []
    for _ in range(2):
        ss.kv_attention(q, layer.cache, table, starts, l, max_new=new, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ss.kv_attention(q, layer.cache, table, starts, l, max_new=new, lse=True, ws=ws))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for step in range(3):
        lens = [200 + 101 * step, 90 + 7 * step]
        l.copy_(i32(lens))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for out, lse in outs:
            check_attention(layer, q, out, lse, [0, new, 2 * new], lens, True, 128**-0.5)
    assert ws.error() == 0


def test_attention_repeats_bit_for_bit(ss):
    for new, lens in ((1, [5000, 77]), (65, [1500, 200])):
        layer = Layer(ss, "int", 128, 64, 2, max(lens), 2, seed=16).fill(lens)
        runs = [attend(ss, layer, lens, [new, new], 4, True, max_new=new, max_len=max(lens))[1:] for _ in range(3)]
        assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


# ---------------------------------------------------------------------------
# the three in a row
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["int", "fp8"])
def test_an_attention_layer_in_8_bits(ss, fmt):
    """Prompt and then single tokens through: rows to INT8, one projection for q, k and v, k and v into the cache,
    attention, rows to INT8, output projection. Against the same layer in binary64 on the stored bf16 weights: each
    8-bit step is within its format's error, so the result is close, and single tokens give the rows that the whole
    prompt gives up to the cache's regrown scales."""
    d, heads, group, width = 64, 2, 4, 512
    hq = heads * group
    g = gen(17)
    w = (torch.randn((hq + 2 * heads) * d, width, generator=g, device="cuda") / width**0.5).bfloat16()
    wo = (torch.randn(width, hq * d, generator=g, device="cuda") / (hq * d)**0.5).bfloat16()
    w8, wo8 = (ss.run(t, pattern=ss.DENSE, fmt="int", bits=8) for t in (w, wo))
    x = torch.randn(200, width, generator=g, device="cuda").bfloat16()

    def run(layer, rows, length):
        a = ss.run(rows, pattern=ss.DENSE, fmt="int", bits=8)
        qkv = ss.gemm_int8(a, w8).view(rows.shape[0], hq + 2 * heads, d)
        where = (layer.table([length]), i32([0, rows.shape[0]]), i32([length]))
        ss.kv_append(layer.cache, qkv[:, hq:hq + heads], qkv[:, hq + heads:], *where)
        o = ss.kv_attention(qkv[:, :hq], layer.cache, *where)
        return ss.gemm_int8(ss.run(o.reshape(rows.shape[0], hq * d), pattern=ss.DENSE, fmt="int", bits=8), wo8,
                            dtype=torch.float32)

    whole = run(Layer(ss, fmt, d, 32, heads, 256, 1, seed=18), x, 200)
    layer = Layer(ss, fmt, d, 32, heads, 256, 1, seed=18)
    steps = [run(layer, x[:190], 190)] + [run(layer, x[i:i + 1], i + 1) for i in range(190, 200)]
    xd = x.double()
    q, k, v = (xd @ w.double().T).view(200, -1, d).split([hq, heads, heads], 1)
    k, v = (t.repeat_interleave(group, 1) for t in (k, v))
    z = torch.einsum("nhd,lhd->hnl", q, k) / d**0.5
    z = z.masked_fill(torch.ones(200, 200, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    ref = torch.einsum("hnl,lhd->nhd", torch.softmax(z, -1), v).reshape(200, hq * d) @ wo.double().T
    # INT8 rows are off by at most half a step of amax / 127, E4M3 by 2^-4 relative: a few such errors in a row
    limit = 0.05 if fmt == "int" else 0.1
    for y in (whole, torch.cat(steps)):
        assert float((y.double() - ref).norm() / ref.norm()) < limit
