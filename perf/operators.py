"""The 8-bit serving operators, in their plain form and through the library.

Three operators that consume what the quantizers write, one case each call:

  gemm    Y = diag(s_a) A B^T diag(s_b), A [m][k] and B [n][k] INT8 codes with one scale per row (a token of the
          activations, an output channel of the weight), Y bf16 or fp32.
  append  new tokens' K and V written into an 8-bit paged cache with one scale per (page, KV head).
  attend  attention of the new tokens over that cache: one new token per sequence (decode) or many (prefill).

Everything is made on the GPU from the seed. ``own`` selects the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INT8_MAX, E4M3_MAX = 127.0, 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _gemm(name, m, n, k, y):
    return {"name": name, "op": "gemm", "m": m, "n": n, "k": k, "y": y}


def _cache(name, op, seqs, new, ctx, kv_heads, group, d, page, fmt, causal=True, ragged=True):
    return {"name": name, "op": op, "seqs": seqs, "new": new, "ctx": ctx, "kv_heads": kv_heads, "group": group, "d": d,
            "page": page, "fmt": fmt, "causal": causal, "ragged": ragged}


def listed():
    return [
        # one token through a square projection: the weight is read once, latency counts
        _gemm("gemm_token", 1, 4096, 4096, "bf16"),
        # a decode batch through an up projection
        _gemm("gemm_decode_batch", 77, 14336, 4096, "bf16"),
        # odd row counts on both sides, k no multiple of a tile, fp32 result
        _gemm("gemm_ragged", 1001, 4099, 4112, "f32"),
        # the sweep's largest linear input, up projection: bound by the tensor cores
        _gemm("gemm_prefill", 16384, 14336, 4096, "bf16"),
        # one new token for each sequence of a decode batch
        _cache("append_decode", "append", 64, 1, 4096, 8, 1, 128, 64, "int"),
        # a long prompt's keys and values
        _cache("append_prefill", "append", 1, 8192, 8192, 8, 1, 128, 32, "fp8"),
        # one request, short context: latency counts
        _cache("decode_short", "attend", 1, 1, 500, 8, 4, 128, 64, "int"),
        # a decode batch of ragged contexts
        _cache("decode_batch", "attend", 64, 1, 8192, 8, 4, 128, 64, "int"),
        # one request over a long context: few rows, the work is along the keys
        _cache("decode_long", "attend", 1, 1, 131072, 8, 4, 128, 128, "fp8", ragged=False),
        # a prompt of 8192 tokens, 32 heads
        _cache("prefill_long", "attend", 1, 8192, 8192, 8, 4, 128, 64, "int", ragged=False),
        # pieces of prompts behind a cached prefix, small heads, small pages
        _cache("prefill_chunks", "attend", 4, 509, 4000, 4, 7, 64, 16, "fp8"),
        # queries that see every cached key, each query head its own KV head
        _cache("cross_all_keys", "attend", 6, 150, 1500, 16, 1, 64, 32, "int", causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "append", "attend", "attend", "attend"])
    if op == "gemm":
        m, n, k = _log(rng, 1, 16384), _log(rng, 64, 16384), 16 * _log(rng, 4, 896)
        m = max(1, min(m, 16384 * 14336 * 4096 // (n * k)))
        c = _gemm("", m, n, k, rng.choice(["bf16", "f32"]))
    else:
        d, page, fmt = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice(["int", "fp8"])
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
        seqs = _log(rng, 1, 64)
        if op == "append":
            ctx = _log(rng, 1, max(2, 65536 // seqs))
            new = rng.choice([1, min(ctx, _log(rng, 1, 8192))])
            new = max(1, min(new, 8192 // seqs))
            c = _cache("", op, seqs, new, ctx, kv_heads, 1, d, page, fmt)
        else:
            ctx = _log(rng, 1, min(131072, 524288 // seqs))
            new = 1
            if rng.random() < 0.5:
                new = min(ctx, _log(rng, 2, 4096))
                new = max(1, min(new, (1 << 30) // (seqs * ctx * kv_heads * group)))
            c = _cache("", op, seqs, new, ctx, kv_heads, group, d, page, fmt, causal=rng.random() < 0.75)
    del c["name"]
    return c


def _lengths(case):
    """Contexts (new tokens included) and new tokens of each sequence, the same for every seed. Ragged: contexts from
    1/8 of the longest up, the first one the longest; new tokens up to the most, the first one the most."""
    rng = np.random.default_rng([case["seqs"], case["ctx"], case["new"]])
    s, ctx, new = case["seqs"], case["ctx"], min(case["new"], case["ctx"])
    lens, news = np.full(s, ctx, dtype=np.int64), np.full(s, new, dtype=np.int64)
    if case["ragged"] and s > 1:
        lens[1:] = rng.integers(max(1, ctx // 8), ctx + 1, s - 1)
        if new > 1:
            news[1:] = rng.integers(1, new + 1, s - 1)
    return lens, np.minimum(news, lens)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _int8_rows(x):
    """Codes and scales of INT8 with one scale per row."""
    s = x.abs().amax(1, keepdim=True) / _top("int")
    q = torch.where(s > 0, x / s, 0).round_().clamp_(-INT8_MAX, INT8_MAX).to(torch.int8)
    return {"values": q, "scales": s}


def _activations(g, rows, cols, std):
    """Normal values with a few channels 20 times the others', in bf16 as a layer writes them."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * std
    hot = torch.randint(cols, (4,), generator=g, device="cuda")
    x[:, hot] *= 20.0
    return x.bfloat16().float()


def prepare(case, seed):
    g, rng = _generator(seed), np.random.default_rng(seed)
    if case["op"] == "gemm":
        a = _int8_rows(_activations(g, case["m"], case["k"], 1.0))
        b = _int8_rows((torch.randn(case["n"], case["k"], generator=g, device="cuda") * 0.02).bfloat16().float())
        return {"case": dict(case), "a": a, "b": b}
    h, d, page, fmt = case["kv_heads"], case["d"], case["page"], case["fmt"]
    lens, news = _lengths(case)
    per = -(-lens // page)
    pages = int(per.sum()) + 3  # a few that no sequence has
    order = rng.permutation(pages)
    table = np.full((case["seqs"], int(per.max())), -1, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(per)])
    for s in range(case["seqs"]):
        table[s, :per[s]] = order[at[s]:at[s + 1]]
    starts = np.concatenate([[0], np.cumsum(news)])
    tokens = int(starts[-1])

    def dev(v):
        return torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).cuda()

    # a cache in use: each page's codes reach its scale, as a page that was quantized by its largest value does
    channel = torch.ones(d, device="cuda")
    channel[torch.randint(d, (3,), generator=g, device="cuda")] = 4.0
    cache = {"fmt": fmt, "page": page}
    for name in ("k", "v"):
        x = torch.randn(pages, h, page, d, generator=g, device="cuda")
        if name == "k":
            x *= channel
        s = x.abs().amax((2, 3)) / _top(fmt)
        x /= s[:, :, None, None]
        cache[name] = x.round_().to(torch.int8) if fmt == "int" else x.to(torch.float8_e4m3fn).view(torch.uint8)
        cache[name + "_scales"] = s
        del x
    state = {"case": dict(case), "cache": cache, "table": dev(table), "starts": dev(starts), "lengths": dev(lens),
             "max_new": int(news.max()), "max_len": int(lens.max())}
    if case["op"] == "append":
        for name in ("k", "v"):
            x = torch.randn(tokens, h, d, generator=g, device="cuda")
            state[name] = (x * channel if name == "k" else x).bfloat16()
    else:
        state["q"] = torch.randn(tokens, h * case["group"], d, generator=g, device="cuda").bfloat16()
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        from semi_structured_sparsity_online_b200 import ss24
        if op == "gemm":
            return ss24.gemm_int8(state["a"], state["b"], dtype=DTYPES[state["case"]["y"]])
        where = (state["table"], state["starts"], state["lengths"])
        if op == "append":
            ss24.kv_append(state["cache"], state["k"], state["v"], *where, max_new=state["max_new"])
            return _cache_outputs(state["cache"])
        out, lse = ss24.kv_attention(state["q"], state["cache"], *where, causal=state["case"]["causal"],
                                     max_new=state["max_new"], max_len=state["max_len"], lse=True)
        return {"out": out, "lse": lse}
    return {"gemm": _plain_gemm, "append": _plain_append, "attend": _plain_attend}[op](state)


def _cache_outputs(cache):
    """The codes as what they stand for (INT8 numbers, E4M3 values) and their scales."""
    as_value = {"int": torch.int8, "fp8": torch.float8_e4m3fn}[cache["fmt"]]
    return {"k": cache["k"].view(as_value), "v": cache["v"].view(as_value), "k_scales": cache["k_scales"],
            "v_scales": cache["v_scales"]}


def _plain_gemm(state):
    a, b = state["a"], state["b"]
    y = (a["values"].float() @ b["values"].float().T) * a["scales"] * b["scales"].T
    return y.to(DTYPES[state["case"]["y"]])


def _top(fmt):
    """The largest code value, as a tensor: a division by a Python number is a product with its reciprocal."""
    return torch.tensor(INT8_MAX if fmt == "int" else E4M3_MAX, device="cuda")


def _quantize(x, s, fmt):
    q = torch.where(s > 0, x / s, 0)
    return q.round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8) if fmt == "int" else q.to(torch.float8_e4m3fn)


def _plain_append(state):
    cache, fmt, page = state["cache"], state["case"]["fmt"], state["case"]["page"]
    starts, lens, table = state["starts"].long(), state["lengths"].long(), state["table"].long()
    # sequence and position of every new token
    t = torch.arange(state["k"].shape[0], device="cuda")
    seq = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[seq] - (starts[seq + 1] - t)
    where, slot = table[seq, pos // page], pos % page
    touched = torch.zeros(cache["k"].shape[0], dtype=torch.bool, device="cuda")
    touched[where] = True
    # a sequence's first page with new tokens may hold older ones, in its first `fill` slots
    begin = lens - (starts[1:] - starts[:-1])
    first, fill = table.gather(1, (begin // page)[:, None])[:, 0], begin % page
    old = (torch.arange(page, device="cuda") < fill[:, None])[:, None, :, None]
    out = _cache_outputs(cache)
    for name in ("k", "v"):
        x, codes, scales = state[name].float(), out[name], out[name + "_scales"]
        amax = torch.zeros_like(scales).scatter_reduce(0, where[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
        s = amax / _top(fmt)
        s[first] = torch.maximum(s[first], torch.where(fill[:, None] > 0, scales[first], 0))
        raw = codes.view(torch.uint8)
        before = raw[first]
        again = _quantize(before.view(codes.dtype).float() * scales[first][..., None, None], s[first][..., None, None], fmt)
        raw[first] = torch.where(old, again.view(torch.uint8), before)
        raw[where, :, slot] = _quantize(x, s[where][:, :, None], fmt).view(torch.uint8)
        scales.copy_(torch.where(touched[:, None], s, scales))
    return out


def _plain_attend(state):
    case, cache, q = state["case"], state["cache"], state["q"]
    h, g, d, page = case["kv_heads"], case["group"], case["d"], case["page"]
    starts, lens, table = state["starts"].long(), state["lengths"].long(), state["table"].long()
    seqs, new = case["seqs"], state["max_new"]
    keys = table.shape[1] * page
    count = starts[1:] - starts[:-1]
    # padded queries [seqs, h, g * new, d]
    i = torch.arange(new, device="cuda")
    token = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[token].float().view(seqs, new, h, g, d).permute(0, 2, 3, 1, 4).reshape(seqs, h, g * new, d)
    # padded keys and values [seqs, h, keys, d]
    j = torch.arange(keys, device="cuda")
    there = j < lens[:, None]
    values = _cache_outputs(cache)

    def padded(name):
        p = table.clamp(min=0)
        v = values[name].view(torch.uint8)[p].view(values[name].dtype).float()
        v *= values[name + "_scales"][p][..., None, None]
        v = v.transpose(1, 2).reshape(seqs, h, keys, d)
        return v.masked_fill_(~there[:, None, :, None], 0.0)

    logits = torch.matmul(x, padded("k").transpose(2, 3))
    logits *= 1.0 / math.sqrt(d)
    seen = there[:, None, :].expand(seqs, new, keys)
    if case["causal"]:
        seen = seen & (j <= (lens - count)[:, None, None] + i[:, None])
    logits.view(seqs, h, g, new, keys).masked_fill_(~seen[:, None, None], -math.inf)
    m = logits.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = logits.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, padded("v")) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + m
    live = i < count[:, None]
    o = o.view(seqs, h, g, new, d).permute(0, 3, 1, 2, 4).reshape(seqs, new, h * g, d)
    lse = lse.view(seqs, h, g, new).permute(0, 3, 1, 2).reshape(seqs, new, h * g)
    return {"out": o[live].bfloat16(), "lse": lse[live]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    return {"gemm": _exact_gemm, "append": _exact_append, "attend": _exact_attend}[case["op"]](state)


def _exact_gemm(state):
    a, b = state["a"], state["b"]
    y = torch.empty(a["values"].shape[0], b["values"].shape[0], dtype=torch.float64, device="cuda")
    bt = b["values"].double().t()
    for r in range(0, y.shape[0], 2048):
        y[r:r + 2048] = torch.mm(a["values"][r:r + 2048].double(), bt)
    y.mul_(a["scales"].double()).mul_(b["scales"].double().view(1, -1))
    return y


def _exact_append(state):
    """Codes and scales are defined with binary32 quotients: a binary64 quotient of binary32 numbers rounded to
    binary32 is that quotient."""
    case, cache = state["case"], state["cache"]
    page, fmt = case["page"], case["fmt"]
    top = INT8_MAX if fmt == "int" else E4M3_MAX
    f32 = np.float32
    table, starts, lens = (state[n].cpu().numpy() for n in ("table", "starts", "lengths"))
    out = {}

    def codes_of(v, s):
        q = np.divide(v.astype(np.float64), s.astype(np.float64)[..., None, None], where=(s > 0)[..., None, None],
                      out=np.zeros(v.shape)).astype(f32)
        if fmt == "int":
            return np.clip(np.rint(q), -127, 127).astype(f32)
        return torch.from_numpy(q).to(torch.float8_e4m3fn).float().numpy()

    for name in ("k", "v"):
        raw = cache[name] if fmt == "int" else cache[name].view(torch.float8_e4m3fn)
        codes, scales = raw.float().cpu().numpy(), cache[name + "_scales"].cpu().numpy()
        x = state[name].float().cpu().numpy()
        for s in range(case["seqs"]):
            begin, end = int(lens[s] - (starts[s + 1] - starts[s])), int(lens[s])
            for p in range(begin // page, -(-end // page)):
                lo, hi = max(begin, p * page), min(end, (p + 1) * page)
                where, fill = table[s, p], lo - p * page
                t = x[starts[s] + lo - begin:starts[s] + hi - begin].transpose(1, 0, 2)
                scale = (np.abs(t).max((1, 2)).astype(np.float64) / top).astype(f32)
                if fill:
                    scale = np.maximum(scale, scales[where])
                    old = (codes[where, :, :fill].astype(np.float64) * scales[where][:, None, None]).astype(f32)
                    codes[where, :, :fill] = codes_of(old, scale)
                codes[where, :, fill:fill + hi - lo] = codes_of(t, scale)
                scales[where] = scale
        t = torch.from_numpy(codes).cuda()
        out[name] = t.to(torch.int8) if fmt == "int" else t.to(torch.float8_e4m3fn)
        out[name + "_scales"] = torch.from_numpy(scales).cuda()
    return out


def _exact_attend(state):
    case, cache, q = state["case"], state["cache"], state["q"]
    page, group, d = case["page"], case["group"], case["d"]
    table, starts, lens = (state[n].cpu().numpy() for n in ("table", "starts", "lengths"))
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")

    def whole(name, s, head):
        ids = torch.from_numpy(table[s, :-(-int(lens[s]) // page)].astype(np.int64)).cuda()
        c = cache[name][ids, head]
        c = c if case["fmt"] == "int" else c.view(torch.float8_e4m3fn)
        x = c.to(torch.float32).double() * cache[name + "_scales"][ids, head].double().view(-1, 1, 1)
        return x.reshape(-1, d)[:int(lens[s])]

    for s in range(case["seqs"]):
        n, length = int(starts[s + 1] - starts[s]), int(lens[s])
        visible = torch.arange(length, device="cuda")
        for head in range(case["kv_heads"]):
            k, v = whole("k", s, head), whole("v", s, head)
            for lo in range(0, n, 2048):
                t = slice(int(starts[s]) + lo, int(starts[s]) + min(lo + 2048, n))
                x = q[t, head * group:(head + 1) * group].double()
                z = torch.einsum("tgd,ld->tgl", x, k) / math.sqrt(d)
                if case["causal"]:
                    at = length - n + lo + torch.arange(x.shape[0], device="cuda")
                    z.masked_fill_((visible > at[:, None])[:, None], -math.inf)
                lse[t, head * group:(head + 1) * group] = torch.logsumexp(z, 2)
                out[t, head * group:(head + 1) * group] = torch.einsum("tgl,ld->tgd", torch.softmax(z, 2), v)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["y"] == "bf16" else 4
        return {"bytes": m * k + n * k + 4 * (m + n) + size * m * n, "flops": 2 * m * n * k}
    h, g, d, page = case["kv_heads"], case["group"], case["d"], case["page"]
    lens, news = _lengths(case)
    tokens = int(news.sum())
    if case["op"] == "append":
        # bf16 in, codes out, scales of the pages that get tokens
        pages = int(((lens - 1) // page - (lens - news) // page + 1).sum())
        return {"bytes": tokens * h * d * 2 * (2 + 1) + 2 * 4 * h * pages, "flops": 4 * tokens * h * d}
    cache = h * (2 * d * int(lens.sum()) + 8 * int((-(-lens // page)).sum()))
    pairs = int((news * lens).sum())
    if case["causal"]:
        pairs -= int((news * (news - 1) // 2).sum())
    return {"bytes": cache + tokens * h * g * (4 * d + 4), "flops": 4 * d * h * g * pairs}
