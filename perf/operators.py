"""The decode-step operators around the norms, as measurable cases: rotary positions (`rotary`),
rotary positions written into a paged key/value cache (`rotary_to_pages`), and attention of a chunk
of new tokens over that cache (`paged_attention`).

Layouts. Tokens of all sequences of a batch are packed: q [tokens, heads, dim]. The cache is a pool
of pages, [pages, page_size, kv_heads, dim]; a sequence's row of the page table lists its pages in
order. Query heads share key/value heads in groups of heads / kv_heads.

Every case has an operator name ("op"), sizes and a dtype. `run` is the plain form, elementary torch
operations in 32 bits (the angles in 64), unless `own` is set; then it is the library's call.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def _rot(name, tokens, heads, kv_heads, dim, rot, interleaved, dtype, scaling="none", base=10000.0,
         far=4096):
    return dict(name=name, op="rotary", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                rot=rot, interleaved=interleaved, dtype=dtype, scaling=scaling, base=base, far=far)


def _write(name, tokens, heads, kv_heads, dim, rot, interleaved, dtype, page, pages,
           scaling="none", base=10000.0, far=4096):
    return dict(name=name, op="rotary_to_pages", tokens=tokens, heads=heads, kv_heads=kv_heads,
                dim=dim, rot=rot, interleaved=interleaved, dtype=dtype, scaling=scaling, base=base,
                far=far, page=page, pages=pages)


def _attn(name, seqs, q_low, q_high, past_low, past_high, heads, kv_heads, dim, dtype, page):
    return dict(name=name, op="paged_attention", seqs=seqs, q_low=q_low, q_high=q_high,
                past_low=past_low, past_high=past_high, heads=heads, kv_heads=kv_heads, dim=dim,
                dtype=dtype, page=page)


def listed():
    return [
        # one decode step of a small batch, far positions, frequencies scaled in bands
        _rot("rotary_step", 16, 32, 8, 128, 128, False, "bf16", "bands", 500000.0, 131072),
        # the prompt of a batch in one pass: streams q and k once
        _rot("rotary_prompt", 16384, 64, 8, 128, 128, False, "bf16"),
        # part of each head rotated in pairs of neighbours, an odd token count
        _rot("rotary_part_pairs", 4099, 40, 40, 128, 64, True, "fp16", "linear", 10000.0, 32768),
        # odd sizes in 32 bits: a rotated part that no 16-byte vector divides
        _rot("rotary_odd", 1333, 7, 1, 80, 30, False, "fp32", "none", 10000.0, 8192),
        # a decode step that appends one token per sequence to its cache
        _write("pages_step", 64, 32, 8, 128, 128, False, "bf16", 16, 4096, "bands", 500000.0, 131072),
        # a prompt appended to the cache
        _write("pages_prompt", 8192, 56, 8, 128, 128, False, "fp16", 64, 256),
        # one new token of one sequence: latency
        _attn("attn_one", 1, 1, 1, 1000, 1000, 32, 8, 128, "bf16", 16),
        # a decode step of a serving batch with ragged contexts: cache bandwidth
        _attn("attn_step", 64, 1, 1, 700, 8100, 64, 8, 128, "bf16", 16),
        # few sequences with long contexts: the long axis has to be split
        _attn("attn_step_long", 4, 1, 1, 120000, 131000, 32, 8, 128, "fp16", 64),
        # a mixed batch: chunks of prompts beside single tokens
        _attn("attn_mixed", 16, 1, 517, 0, 4200, 32, 8, 128, "bf16", 32),
        # heads of 64 without sharing, odd lengths
        _attn("attn_heads64", 3, 301, 1025, 17, 2100, 12, 12, 64, "fp16", 16),
        # a long prompt's chunk over as much context again: tensor-core bound
        _attn("attn_prompt", 1, 8192, 8192, 8192, 8192, 32, 8, 128, "bf16", 64),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(("rotary", "rotary_to_pages", "paged_attention", "paged_attention"))
    dtype = rng.choice(("bf16", "fp16", "bf16", "fp32" if op != "paged_attention" else "fp16"))
    if op != "paged_attention":
        dim = rng.choice((64, 80, 96, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8, 12))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8))
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        tokens = _log_int(rng, 1, max(1, min(16384, (150 << 20) // ((heads + 2 * kv_heads) * dim * 2))))
        more = dict(interleaved=rng.random() < 0.4, scaling=rng.choice(("none", "linear", "bands")),
                    base=rng.choice((10000.0, 500000.0)), far=_log_int(rng, 64, 262144))
        if op == "rotary":
            return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                        dtype=dtype, **more)
        page = rng.choice((8, 16, 32, 64, 128))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                    dtype=dtype, page=page, pages=-(-tokens // page) + rng.randint(1, 64), **more)
    page = rng.choice((8, 16, 32, 64, 128))
    kind = rng.choice(("step", "step", "chunk", "chunk"))
    if kind == "step":  # single tokens, now and then a few (drafts that are checked together)
        dim = rng.choice((64, 96, 128, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 4, 5, 8, 16))
        seqs = _log_int(rng, 1, 256)
        most = max(64, min(131072, (1 << 30) // (seqs * kv_heads * dim * 4)))
        high = _log_int(rng, 1, most)
        q = rng.choice((1, 1, 1, 2, 5))
        return dict(op=op, seqs=seqs, q_low=1, q_high=q, past_low=rng.randint(0, high),
                    past_high=high, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page)
    dim = rng.choice((64, 80, 96, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 4, 7, 8))
    seqs = _log_int(rng, 1, 16)
    q = _log_int(rng, 2, max(2, 2048 // seqs))
    high = _log_int(rng, 1, 8192)
    return dict(op=op, seqs=seqs, q_low=rng.randint(0, q), q_high=q, past_low=rng.randint(0, high),
                past_high=high, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page)


# ------------------------------------------------------------------------------------- inputs

def _scaling(case):
    """The keyword arguments of the frequencies' scaling."""
    if case["scaling"] == "linear":
        return dict(scaling="linear", factor=4.0)
    if case["scaling"] == "bands":
        return dict(scaling="bands", factor=8.0, original_length=8192, low=1.0, high=4.0)
    return {}


def _frequencies(case, device):
    """Angle per position of each rotated pair, in 64 bits."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=device)
    f = case["base"] ** (-i / case["rot"])
    s = _scaling(case)
    if case["scaling"] == "linear":
        return f / s["factor"]
    if case["scaling"] == "bands":  # few turns over the old length: slowed; many: kept; between: blended
        turns = s["original_length"] * f / (2 * math.pi)
        keep = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        return f * keep + f / s["factor"] * (1 - keep)
    return f


def _lengths(case):
    """New tokens and past tokens per sequence: the highest of each range is in the batch."""
    import random
    rng = random.Random(case["seqs"] * 7919 + case["q_high"] * 31 + case["past_high"])
    q = [rng.randint(case["q_low"], case["q_high"]) for _ in range(case["seqs"])]
    past = [rng.randint(case["past_low"], case["past_high"]) for _ in range(case["seqs"])]
    q[0], past[-1] = case["q_high"], case["past_high"]
    return q, past


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    st = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    if case["op"] != "paged_attention":
        t = case["tokens"]
        qkv = normal(t, (hq + 2 * hk) * d)  # the fused projection's output, which q, k and v are views of
        st["q"] = qkv[:, :hq * d].view(t, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        st["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        st["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=dev)
        f = _frequencies(case, dev)
        st["freq"] = f
        # the same frequencies as fractions of a turn in 64-bit fixed point, a plan that a program keeps
        st["steps"] = torch.round(f / (2 * math.pi) * 2.0 ** 63).to(torch.int64) * 2
        if case["op"] == "rotary_to_pages":
            st["k_pages"] = normal(case["pages"], case["page"], hk, d)
            st["v_pages"] = normal(case["pages"], case["page"], hk, d)
            st["slots"] = torch.randperm(case["pages"] * case["page"], generator=g, device=dev)[:t].contiguous()
        return st

    q_lens, past = _lengths(case)
    kv = [a + b for a, b in zip(q_lens, past)]
    page = case["page"]
    need = [-(-n // page) for n in kv]
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
    st["q"] = normal(max(1, starts[-1]), hq, d)
    st["k_pages"] = normal(pool, page, hk, d)
    st["v_pages"] = normal(pool, page, hk, d)
    st["table"] = table
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    st["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["max_q"] = max(q_lens)
    st["max_kv"] = max(kv)
    return st


# ------------------------------------------------------------------------------------- run

def _rotate(x, cos, sin, rot, interleaved):
    """x [tokens, heads, dim] with its first `rot` values of each head rotated by cos, sin
    [tokens, rot / 2]; in 32 bits, rounded once."""
    part = x[..., :rot].float()
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
    c, s = cos[:, None, :], sin[:, None, :]
    u, w = a * c - b * s, b * c + a * s
    if interleaved:
        y = torch.stack((u, w), dim=-1).flatten(-2)
    else:
        y = torch.cat((u, w), dim=-1)
    return torch.cat((y.to(x.dtype), x[..., rot:]), dim=-1)


def _plain_rotary(st):
    angle = st["positions"].double()[:, None] * st["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate(st["q"], cos, sin, st["rot"], st["interleaved"])
    k = _rotate(st["k"], cos, sin, st["rot"], st["interleaved"])
    if st["op"] == "rotary":
        return q, k
    st["k_pages"].view(-1, *k.shape[1:])[st["slots"]] = k
    st["v_pages"].view(-1, *k.shape[1:])[st["slots"]] = st["v"]
    return q, st["k_pages"], st["v_pages"]


def _plain_attention(st):
    q, table, starts = st["q"], st["table"].long(), st["q_starts"].long()
    page, group = st["page"], st["heads"] // st["kv_heads"]
    dev = q.device
    kv_lens, q_lens = st["kv_lens"].long(), starts[1:] - starts[:-1]
    # every sequence's keys and values in order, padded to the longest: [seqs, kv_heads, keys, dim]
    at = torch.arange(st["max_kv"], device=dev)
    slot = table[:, at // page] * page + at % page
    keys = st["k_pages"].view(-1, *st["k_pages"].shape[2:])[slot].float().transpose(1, 2)
    values = st["v_pages"].view(-1, *st["v_pages"].shape[2:])[slot].float().transpose(1, 2)
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
    if own:
        import row_wise_rmsnorm_ks_gb300 as ks
        if st["op"] == "rotary":
            return ks.rotary(st["q"], st["k"], st["positions"], st["steps"],
                             interleaved=st["interleaved"])
        if st["op"] == "rotary_to_pages":
            q = ks.rotary_to_pages(st["q"], st["k"], st["v"], st["positions"], st["steps"],
                                   st["k_pages"], st["v_pages"], st["slots"],
                                   interleaved=st["interleaved"])
            return q, st["k_pages"], st["v_pages"]
        return ks.paged_attention(st["q"], st["k_pages"], st["v_pages"], st["table"],
                                  st["kv_lens"], st["q_starts"], max_q_len=st["max_q"])
    return _plain_attention(st) if st["op"] == "paged_attention" else _plain_rotary(st)


# ------------------------------------------------------------------------------------- work, exact

def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] != "paged_attention":
        t, rot = case["tokens"], case["rot"]
        moved = (hq + hk) + (hk if case["op"] == "rotary_to_pages" else 0)
        index = 8 + (8 if case["op"] == "rotary_to_pages" else 0)
        return {"bytes": 2 * t * moved * d * e + t * index + rot * 4,
                "flops": 3 * t * (hq + hk) * rot}
    q_lens, past = _lengths(case)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(q_lens, past))
    keys = sum(n + p for n, p in zip(q_lens, past) if n)
    return {"bytes": 2 * sum(q_lens) * hq * d * e + 2 * keys * hk * d * e
            + 4 * sum(-(-(n + p) // case["page"]) for n, p in zip(q_lens, past)) + 8 * case["seqs"],
            "flops": 4 * pairs * hq * d}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "paged_attention":
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

        q, k = rotated(st["q"]), rotated(st["k"])
        if case["op"] == "rotary":
            return q, k
        kp, vp = st["k_pages"].double(), st["v_pages"].double()
        page, offset = st["slots"] // case["page"], st["slots"] % case["page"]
        kp[page, offset], vp[page, offset] = k, st["v"].double()
        return q, kp, vp
    q_lens, past = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    out = torch.empty(sum(q_lens), case["heads"], case["dim"], dtype=torch.float64, device=st["q"].device)
    at = 0
    for b, (n, before) in enumerate(zip(q_lens, past)):
        pages = st["table"][b, :-(-(n + before) // case["page"])].long()
        k = st["k_pages"][pages].flatten(0, 1)[:n + before].double()
        v = st["v_pages"][pages].flatten(0, 1)[:n + before].double()
        q = st["q"][at:at + n].double()
        for first in range(0, n, 1024):  # some rows at a time, to hold one block of scores
            rows = min(1024, n - first)
            hidden = torch.ones(rows, n + before, dtype=torch.bool, device=q.device).triu(before + first + 1)
            for h in range(case["heads"]):
                s = q[first:first + rows, h] @ k[:, h // group].T / case["dim"] ** 0.5
                out[at + first:at + first + rows, h] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
        at += n
    return out
