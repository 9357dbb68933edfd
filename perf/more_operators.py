"""More operators of a decoder block, as measurable cases: a paged key/value cache whose values are held
in 4 bits, written as positions are turned (`to_pages`, with the written rows read back), read back alone
(`to_rows`) and attended over (`attention`), and the norm after a block, its gate, the scaled residual add
and the norm before the next block in one pass (`block_norms`).

The cache. A head's row of `dim` values is cut into groups of 16. A group is held as 16 codes of 4 bits,
sign and the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 (value 2i in the low half of byte i), and one scale of
8 bits (float8 e4m3). With the pool's own factor g and a group's largest magnitude A:

    s = A / (6 g) rounded to e4m3, at most 448;   u = s g, in 32 bits;   code = x / u rounded, at most 6

both to the nearest, ties to the even code; a group whose s is 0 has codes 0, one that holds a NaN a
NaN as s. What is held is u code. A pool is (codes [pages, page_size, kv_heads, dim / 2], scales [pages,
page_size, kv_heads, dim / 16]), here laid out head by head within a page or token by token.

Tokens of all sequences are packed: q [tokens, heads, dim]; a sequence's row of the page table lists its
pages in order; query heads share key/value heads in groups of heads / kv_heads.

Every case has an operator name ("op"), sizes and a dtype. `run` is the plain form, elementary torch
operations, unless `own` is set; then it is the library's calls.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def _norms(name, seqs, tokens, hidden, dtype, post, gate, residual_scale, block_scale):
    return dict(name=name, op="block_norms", seqs=seqs, tokens=tokens, hidden=hidden, dtype=dtype, post=post,
                gate=gate, residual_scale=residual_scale, block_scale=block_scale, eps=1e-6)


def _write(name, tokens, heads, kv_heads, dim, rot, interleaved, dtype, page, pages, by_head, far, factor):
    return dict(name=name, op="to_pages", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved, dtype=dtype, page=page, pages=pages, by_head=by_head, far=far,
                factor=factor)


def _read(name, tokens, kv_heads, dim, dtype, page, pages, by_head, ordered, factor):
    return dict(name=name, op="to_rows", tokens=tokens, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page,
                pages=pages, by_head=by_head, ordered=ordered, factor=factor)


def _attn(name, seqs, q_low, q_high, past_low, past_high, heads, kv_heads, dim, dtype, page, by_head, factor):
    return dict(name=name, op="attention", seqs=seqs, q_low=q_low, q_high=q_high, past_low=past_low,
                past_high=past_high, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page,
                by_head=by_head, factor=factor)


def listed():
    return [
        # the end of a block in a decode step: norm, a gate per channel, add, norm; latency
        _norms("norms_step", 4, 1, 1536, "bf16", True, "channel", 1.0, 1.0),
        # a prompt's batch through the same, gated per sequence; streams two tensors in and out
        _norms("norms_prompt", 3, 5461, 8192, "bf16", True, "sequence", 1.0, 0.5),
        # a decode step: one token per sequence, turned and put into the cache in 4 bits, and read back
        _write("pages_step", 64, 32, 8, 128, 128, False, "bf16", 16, 4096, True, 131072, 1.0),
        # a prompt into the cache
        _write("pages_prompt", 8192, 56, 8, 128, 128, False, "fp16", 64, 256, True, 4096, 0.5),
        # odd sizes: part of a head turned in pairs of neighbours, token by token pools, 32 bits
        _write("pages_odd", 1333, 7, 1, 80, 30, True, "fp32", 16, 100, False, 8192, 0.375),
        # a sequence's keys and values out of the cache, to be sent elsewhere: streams
        _read("rows_long", 131001, 8, 128, "bf16", 64, 2100, True, True, 1.0),
        # some tokens of many, from anywhere
        _read("rows_few", 777, 8, 128, "fp16", 16, 4096, False, False, 0.5),
        # one new token of one sequence: latency
        _attn("attn_one", 1, 1, 1, 1000, 1000, 32, 8, 128, "bf16", 16, True, 1.0),
        # a decode step of a serving batch with ragged contexts: the cache's bytes
        _attn("attn_step", 64, 1, 1, 700, 8100, 64, 8, 128, "bf16", 16, True, 1.0),
        # few sequences with long contexts, token by token pools: the long axis has to be split
        _attn("attn_step_long", 4, 1, 1, 120000, 131000, 32, 8, 128, "fp16", 64, False, 0.5),
        # a mixed batch: chunks of prompts beside single tokens
        _attn("attn_mixed", 16, 1, 517, 0, 4200, 32, 8, 128, "bf16", 32, True, 1.0),
        # a long prompt's chunk over as much context again: the matrix products
        _attn("attn_prompt", 1, 8192, 8192, 8192, 8192, 32, 8, 128, "bf16", 64, True, 1.0),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(("block_norms", "block_norms", "to_pages", "to_rows", "attention", "attention", "attention"))
    dtype = rng.choice(("bf16", "fp16", "bf16", "fp16" if op == "attention" else "fp32"))
    by_head, factor = rng.random() < 0.6, rng.choice((1.0, 1.0, 0.5, 0.375, 251 / 4096))
    if op == "block_norms":
        hidden = 8 * _log_int(rng, 16, 2048) + rng.choice((0, 0, 0, 1, 4))
        rows = _log_int(rng, 1, min(65536, (48 << 20) // hidden))
        seqs = max(1, min(rows, rng.choice((1, 2, 7, 64))))
        return dict(op=op, seqs=seqs, tokens=rows // seqs, hidden=hidden, dtype=dtype, post=rng.random() < 0.7,
                    gate=rng.choice(("none", "channel", "sequence", "token")),
                    residual_scale=rng.choice((1.0, 1.0, 0.75)), block_scale=rng.choice((1.0, 0.22, 0.5)),
                    eps=rng.choice((1e-6, 1e-5)))
    page = rng.choice((8, 16, 32, 64, 128))
    if op == "to_pages":
        dim = rng.choice((64, 80, 96, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8, 12))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8))
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        tokens = _log_int(rng, 1, max(1, min(16384, (130 << 20) // ((heads + 2 * kv_heads) * dim * 2))))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                    interleaved=rng.random() < 0.4, dtype=dtype, page=page, pages=-(-tokens // page) + rng.randint(1, 64),
                    by_head=by_head, far=_log_int(rng, 64, 262144), factor=factor)
    if op == "to_rows":
        dim, kv_heads = rng.choice((64, 80, 96, 128, 128, 256)), rng.choice((1, 2, 4, 8, 12))
        tokens = _log_int(rng, 1, (96 << 20) // (kv_heads * dim))
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page,
                    pages=-(-tokens // page) + rng.randint(1, 64), by_head=by_head, ordered=rng.random() < 0.5,
                    factor=factor)
    if rng.random() < 0.5:  # single tokens, now and then a few (drafts that are checked together)
        dim = rng.choice((64, 96, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 4, 5, 8, 16))
        seqs = _log_int(rng, 1, 256)
        most = max(64, min(131072, (1 << 30) // (seqs * kv_heads * dim * 4)))
        high = _log_int(rng, 1, most)
        return dict(op=op, seqs=seqs, q_low=1, q_high=rng.choice((1, 1, 1, 2, 5)), past_low=rng.randint(0, high),
                    past_high=high, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page,
                    by_head=by_head, factor=factor)
    dim = rng.choice((64, 80, 96, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 4, 7, 8))
    seqs = _log_int(rng, 1, 16)
    q = _log_int(rng, 2, max(2, 2048 // seqs))
    high = _log_int(rng, 1, 8192)
    return dict(op=op, seqs=seqs, q_low=rng.randint(0, q), q_high=q, past_low=rng.randint(0, high), past_high=high,
                heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page, by_head=by_head, factor=factor)


# ------------------------------------------------------------------------------------- the 4-bit groups

def _magnitudes(device, dtype):
    return torch.tensor((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0), device=device, dtype=dtype)


def _steps(device, dtype):
    """The values of e4m3's codes 0 .. 126."""
    return torch.arange(127, device=device, dtype=torch.uint8).view(torch.float8_e4m3fn).to(dtype)


def _nearest(x, values):
    """The index of the value nearest to each x >= 0, ties to the even index."""
    borders = (values[1:] + values[:-1]) / 2
    i = torch.bucketize(x, borders, out_int32=True)
    tie = x == borders[i.clamp(max=borders.numel() - 1).long()]
    return i + (tie & (i % 2 == 1) & (i < borders.numel())).to(torch.int32)


def _quantise(x, factor):
    """x [..., dim] in 64 bits: codes [..., dim / 2] and scales [..., dim / 16]."""
    groups = x.unflatten(-1, (-1, 16))
    size = groups.abs()
    top = size.amax(-1)
    steps = _steps(x.device, torch.float64)
    scale = steps[_nearest(top / (6.0 * factor), steps).long()].float()
    unit = (scale * torch.tensor(factor, device=x.device)).double()[..., None]  # rounded to 32 bits
    code = _nearest(torch.where(unit > 0, size / unit, 0.0), _magnitudes(x.device, torch.float64))
    nan = torch.isnan(top)
    code = torch.where(nan[..., None], 0, code + 8 * (groups < 0).to(torch.int32)).flatten(-2)
    scale = torch.where(nan, math.nan, scale).to(torch.float8_e4m3fn)
    return (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8), scale


def _held(codes, scales, factor):
    """The values of codes [..., dim / 2] and scales [..., dim / 16], in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    value = _magnitudes(codes.device, torch.float32)[c & 7] * torch.where(c > 7, -1.0, 1.0)
    unit = scales.float() * torch.tensor(factor, device=codes.device)
    return (value.unflatten(-1, (-1, 16)) * unit[..., None]).flatten(-2)


def _taken(pool, page, place):
    """A pool's codes and scales at some places."""
    codes, scales = pool
    return codes[page, place], scales.view(torch.uint8)[page, place].view(torch.float8_e4m3fn)


# ------------------------------------------------------------------------------------- inputs

def _frequencies(case, device):
    """Angle per position of each rotated pair, in 64 bits."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=device)
    return 10000.0 ** (-i / case["rot"])


def _lengths(case):
    """New tokens and past tokens per sequence: the highest of each range is in the batch."""
    rng = random.Random(case["seqs"] * 7919 + case["q_high"] * 31 + case["past_high"])
    q = [rng.randint(case["q_low"], case["q_high"]) for _ in range(case["seqs"])]
    past = [rng.randint(case["past_low"], case["past_high"]) for _ in range(case["seqs"])]
    q[0], past[-1] = case["q_high"], case["past_high"]
    return q, past


def _pool(case, pages, g, device):
    """A pool that holds what became of normal values, as a cache in use does."""
    kv, page, dim, factor = case["kv_heads"], case["page"], case["dim"], case["factor"]
    order = (pages, kv, page) if case["by_head"] else (pages, page, kv)
    x = torch.randn(*order, dim // 16, 16, generator=g, device=device)
    scales = (x.abs().amax(-1) / (6.0 * factor)).clamp(max=448.0).to(torch.float8_e4m3fn)
    x /= scales.float().clamp(min=2.0 ** -9).mul_(factor)[..., None]
    borders = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=device)
    c = (torch.bucketize(x.abs(), borders, out_int32=True).to(torch.uint8) + (x < 0).to(torch.uint8) * 8).flatten(-2)
    codes = c[..., 0::2] | c[..., 1::2] << 4
    return (codes.transpose(1, 2), scales.transpose(1, 2)) if case["by_head"] else (codes, scales)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    st = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    if case["op"] == "block_norms":
        shape = (case["seqs"], case["tokens"], case["hidden"])
        st["x"] = (normal(*shape) * 3).to(dt)
        st["residual"] = (normal(*shape) * 2).to(dt)
        st["weight"] = (1 + 0.1 * normal(case["hidden"])).to(dt)
        st["post_weight"] = (0.5 + 0.1 * normal(case["hidden"])).to(dt) if case["post"] else None
        gates = {"none": None, "channel": (case["hidden"],), "sequence": (case["seqs"], 1, case["hidden"]), "token": shape}
        st["gate"] = (0.3 + 0.2 * normal(*gates[case["gate"]])).to(dt) if gates[case["gate"]] else None
        return st

    hk, d = case["kv_heads"], case["dim"]
    if case["op"] == "to_pages":
        t, hq = case["tokens"], case["heads"]
        qkv = normal(t, (hq + 2 * hk) * d).to(dt)  # the fused projection's output, which q, k and v are views of
        st["q"] = qkv[:, :hq * d].view(t, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        st["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        st["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=dev)
        st["freq"] = _frequencies(case, dev)
        # the same frequencies as fractions of a turn in 64-bit fixed point, a plan that a program keeps
        st["steps"] = torch.round(st["freq"] / (2 * math.pi) * 2.0 ** 63).to(torch.int64) * 2
        st["k_pages"], st["v_pages"] = _pool(case, case["pages"], g, dev), _pool(case, case["pages"], g, dev)
        st["slots"] = torch.randperm(case["pages"] * case["page"], generator=g, device=dev)[:t].contiguous()
        return st
    if case["op"] == "to_rows":
        t = case["tokens"]
        st["k_pages"], st["v_pages"] = _pool(case, case["pages"], g, dev), _pool(case, case["pages"], g, dev)
        if case["ordered"]:  # a sequence's places, page by page
            order = torch.randperm(case["pages"], generator=g, device=dev)
            st["slots"] = (order[:, None] * case["page"] + torch.arange(case["page"], device=dev)).flatten()[:t].contiguous()
        else:
            st["slots"] = torch.randint(0, case["pages"] * case["page"], (t,), generator=g, device=dev)
        return st

    q_lens, past = _lengths(case)
    kv = [a + b for a, b in zip(q_lens, past)]
    need = [-(-n // case["page"]) for n in kv]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(case["seqs"], max(1, max(need)), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    st["q"] = normal(max(1, starts[-1]), case["heads"], d).to(dt)
    st["k_pages"], st["v_pages"] = _pool(case, pool, g, dev), _pool(case, pool, g, dev)
    st["table"] = table
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    st["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["max_q"] = max(q_lens)
    st["max_kv"] = max(kv)
    return st


# ------------------------------------------------------------------------------------- run

def _plain_norms(st):
    x, r, eps = st["x"].float(), st["residual"].float(), st["eps"]
    if st["post_weight"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * st["post_weight"].float()
    if st["gate"] is not None:
        x = x * st["gate"].float()
    s = r * st["residual_scale"] + x * st["block_scale"]
    st["residual"].copy_(s)
    st["x"].copy_(s * torch.rsqrt((s * s).mean(-1, keepdim=True) + eps) * st["weight"].float())
    return st["x"], st["residual"]


def _rotate(x, cos, sin, rot, interleaved):
    """x [tokens, heads, dim] in 32 or 64 bits with its first `rot` values of each head rotated by cos, sin
    [tokens, rot / 2]."""
    part = x[..., :rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
    c, s = cos[:, None, :], sin[:, None, :]
    u, w = a * c - b * s, b * c + a * s
    y = torch.stack((u, w), dim=-1).flatten(-2) if interleaved else torch.cat((u, w), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _plain_rows(st):
    page, place = st["slots"] // st["page"], st["slots"] % st["page"]
    dt = _DTYPES[st["dtype"]]
    return tuple(_held(*_taken(p, page, place), st["factor"]).to(dt) for p in (st["k_pages"], st["v_pages"]))


def _plain_to_pages(st):
    angle = st["positions"].double()[:, None] * st["freq"]
    cos, sin = torch.cos(angle), torch.sin(angle)
    q = _rotate(st["q"].float(), cos.float(), sin.float(), st["rot"], st["interleaved"]).to(st["q"].dtype)
    k = _rotate(st["k"].double(), cos, sin, st["rot"], st["interleaved"])
    page, place = st["slots"] // st["page"], st["slots"] % st["page"]
    for pool, x in ((st["k_pages"], k), (st["v_pages"], st["v"].double())):
        codes, scales = _quantise(x, st["factor"])
        pool[0][page, place] = codes
        pool[1].view(torch.uint8)[page, place] = scales.view(torch.uint8)
    return (q,) + _plain_rows(st)


def _plain_attention(st):
    q, table, starts = st["q"], st["table"].long(), st["q_starts"].long()
    page, group, dev = st["page"], st["heads"] // st["kv_heads"], st["q"].device
    kv_lens, q_lens = st["kv_lens"].long(), starts[1:] - starts[:-1]
    # every sequence's keys and values in order, padded to the longest: [seqs, kv_heads, keys, dim]
    at = torch.arange(st["max_kv"], device=dev)
    pages, place = table[:, at // page], at % page
    keys, values = (_held(*_taken(p, pages, place), st["factor"]).transpose(1, 2) for p in (st["k_pages"], st["v_pages"]))
    # every sequence's queries, padded: [seqs, kv_heads, max_q * group, dim]
    i = torch.arange(st["max_q"], device=dev)
    token = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    rows = q[token].float().unflatten(2, (st["kv_heads"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(rows, keys.transpose(-1, -2)) * (1.0 / math.sqrt(st["dim"]))
    sees = at < (kv_lens - q_lens)[:, None, None] + i[:, None] + 1  # [seqs, max_q, keys]
    sees = (sees & (at < kv_lens[:, None, None])).repeat_interleave(group, dim=1)[:, None]
    s = torch.where(sees, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, values) / torch.where(total == 0, 1.0, total)
    o = o.unflatten(2, (st["max_q"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[i < q_lens[:, None]].to(q.dtype)  # back to packed tokens


def run(st):
    op = st["op"]
    if not own:
        return {"block_norms": _plain_norms, "to_pages": _plain_to_pages, "to_rows": _plain_rows,
                "attention": _plain_attention}[op](st)
    import row_wise_rmsnorm_ks_gb300 as ks
    if op == "block_norms":
        ks.gated_add_rms_norm(st["x"], st["residual"], st["weight"], post_weight=st["post_weight"], gate=st["gate"],
                              residual_scale=st["residual_scale"], block_scale=st["block_scale"], eps=st["eps"])
        return st["x"], st["residual"]
    factors = dict(k_scale=st["factor"], v_scale=st["factor"])
    if op == "attention":
        return ks.paged_attention_4bit(st["q"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"], st["q_starts"],
                                       max_q_len=st["max_q"], **factors)
    dt = _DTYPES[st["dtype"]]
    if op == "to_rows":
        return ks.pages_4bit_to_rows(st["k_pages"], st["v_pages"], st["slots"], dtype=dt, **factors)
    q = ks.rotary_to_pages_4bit(st["q"], st["k"], st["v"], st["positions"], st["steps"], st["k_pages"], st["v_pages"],
                                st["slots"], interleaved=st["interleaved"], **factors)
    return (q,) + ks.pages_4bit_to_rows(st["k_pages"], st["v_pages"], st["slots"], dtype=dt, **factors)


# ------------------------------------------------------------------------------------- work, exact

def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "block_norms":
        h, rows = case["hidden"], case["seqs"] * case["tokens"]
        gate = {"none": 0, "channel": h, "sequence": case["seqs"] * h, "token": rows * h}[case["gate"]]
        return {"bytes": e * (4 * rows * h + h * (2 if case["post"] else 1) + gate),
                "flops": rows * h * (7 + (4 if case["post"] else 0) + (1 if gate else 0))}
    hk, d = case["kv_heads"], case["dim"]
    held = hk * (d // 2 + d // 16)  # a token's keys, or values, in the cache
    if case["op"] == "to_rows":
        return {"bytes": case["tokens"] * (2 * held + 2 * hk * d * e + 8), "flops": 2 * case["tokens"] * hk * d}
    if case["op"] == "to_pages":
        t, hq = case["tokens"], case["heads"]
        return {"bytes": t * ((2 * hq + 4 * hk) * d * e + 2 * held + 16) + case["rot"] * 4,
                "flops": 3 * t * (hq + hk) * case["rot"] + 6 * t * hk * d}
    q_lens, past = _lengths(case)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(q_lens, past))
    keys = sum(n + p for n, p in zip(q_lens, past) if n)
    return {"bytes": 2 * sum(q_lens) * case["heads"] * d * e + 2 * keys * held
            + 4 * sum(-(-(n + p) // case["page"]) for n, p in zip(q_lens, past)) + 8 * case["seqs"],
            "flops": 4 * pairs * case["heads"] * d}


def _exact_held(codes, scales, factor):
    """What a pool's rows hold, in 64 bits: the sign's bit, two of exponent and one of fraction."""
    n = torch.stack((codes.bitwise_and(15), codes.bitwise_right_shift(4)), dim=-1).reshape(*codes.shape[:-1], -1).double()
    sign = 1 - 2 * torch.floor(n / 8)
    n = n - 8 * torch.floor(n / 8)
    power, fraction = torch.floor(n / 2), n - 2 * torch.floor(n / 2)
    size = torch.where(power == 0, fraction / 2, (2 + fraction) * (power + (power == 3)) / 2)  # 1, 2, 4 times
    unit = scales.to(torch.float32).mul(factor).double()
    return sign * size * unit.repeat_interleave(16, dim=-1)


def _exact_stored(x, factor):
    """x in 64 bits as the cache holds it: rounded to multiples of the step at each value's size."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    powers = torch.tensor([2.0 ** k for k in range(-30, 31)], dtype=torch.float64, device=x.device)  # exact ones

    def rounded(v, bits, lowest, most):  # to `bits` bits of fraction, exponents from `lowest` on; ties to even
        exponent = torch.frexp(v).exponent.clamp(min=lowest + 1, max=30) - 1
        step = powers[(exponent - bits + 30).long()]
        return (torch.round(v / step) * step).clamp(max=most)

    scale = rounded(torch.max(y.abs(), dim=-1).values / (6.0 * factor), 3, -6, 448.0)
    unit = scale.float().mul(factor).double().unsqueeze(-1)
    size = rounded(y.abs() / torch.where(unit == 0, math.inf, unit), 1, 0, 6.0)
    return (torch.sign(y) * size * unit).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "block_norms":
        n = st["x"].double()
        if st["post_weight"] is not None:
            n = n / torch.sqrt(n.square().sum(-1, keepdim=True) / case["hidden"] + case["eps"]) * st["post_weight"].double()
        n = n if st["gate"] is None else st["gate"].double() * n
        s = case["residual_scale"] * st["residual"].double() + case["block_scale"] * n
        return s / torch.sqrt(s.square().sum(-1, keepdim=True) / case["hidden"] + case["eps"]) * st["weight"].double(), s
    if case["op"] == "to_rows":
        out = []
        for codes, scales in (st["k_pages"], st["v_pages"]):
            of = lambda t: t.view(torch.uint8).reshape(-1, *t.shape[2:]).index_select(0, st["slots"])  # noqa: E731
            out.append(_exact_held(of(codes), of(scales).view(torch.float8_e4m3fn), case["factor"]))
        return tuple(out)
    if case["op"] == "to_pages":
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=st["q"].device),
                           st["positions"].to(torch.float64).unsqueeze(1) * st["freq"].unsqueeze(0))
        half = case["rot"] // 2

        def rotated(x):
            y = x.double()
            if case["interleaved"]:
                z = torch.complex(y[:, :, 0:2 * half:2].contiguous(), y[:, :, 1:2 * half:2].contiguous())
            else:
                z = torch.complex(y[:, :, :half].contiguous(), y[:, :, half:2 * half].contiguous())
            z = z * turn.unsqueeze(1)
            if case["interleaved"]:
                y[:, :, 0:2 * half:2], y[:, :, 1:2 * half:2] = z.real, z.imag
            else:
                y[:, :, :half], y[:, :, half:2 * half] = z.real, z.imag
            return y

        return (rotated(st["q"]), _exact_stored(rotated(st["k"]), case["factor"]),
                _exact_stored(st["v"].double(), case["factor"]))
    q_lens, past = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    out = torch.empty(sum(q_lens), case["heads"], case["dim"], dtype=torch.float64, device=st["q"].device)
    at = 0
    for b, (n, before) in enumerate(zip(q_lens, past)):
        pages = st["table"][b, :-(-(n + before) // case["page"])].long()
        k, v = (_exact_held(pool[0].index_select(0, pages).flatten(0, 1)[:n + before],
                            pool[1].view(torch.uint8).index_select(0, pages).flatten(0, 1)[:n + before]
                            .view(torch.float8_e4m3fn), case["factor"]) for pool in (st["k_pages"], st["v_pages"]))
        q = st["q"][at:at + n].double()
        for first in range(0, n, 1024):  # some rows at a time, to hold one block of scores
            rows = min(1024, n - first)
            hidden = torch.ones(rows, n + before, dtype=torch.bool, device=q.device).triu(before + first + 1)
            for h in range(case["heads"]):
                s = q[first:first + rows, h] @ k[:, h // group].T / case["dim"] ** 0.5
                out[at + first:at + first + rows, h] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
        at += n
    return out
