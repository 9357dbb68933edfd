"""The 4-bit cache on the GPU against plain 64-bit implementations: writing with rotary positions, reading
back, attention over it, and a run of a block's operators together.

Codes and scales are compared for equality: they are defined on the real values, and 64-bit arithmetic errs by about
10^-11 of a step, which none of these inputs come near to a border. Rotated queries have the tolerance of rotary.

Tolerance of attention, per element: half a step of the output type relative to the value; the probabilities'
rounding to fp16, 2^-11 relative to each (the largest is held as 2^8 or more, so those below 2^-14 / 2^8 = 2^-22 of it are
off by half of fp16's last step, 2^-25 / 2^8 = 2^-33 of it each); the FP32 scores,
off by (dim + 8) 2^-23 of sum |q k| |scale| at most (products of 11 and 6 bits are exact, dim sums that may truncate,
the scale), and for bf16 queries 2^-25 of the row's largest times sum |k| |scale| for what fp16 drops, which is the
relative error of p, and of l again; 2 n 2^-23 for n summed keys in l and in the output, 2^-21 for each exponential.
"""
import math

import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from row_wise_rmsnorm_ks_gb300 import _abi
from test_gpu_decode_ops import close, faults, freqs, no_faults, normal, rotated  # noqa: F401

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn
MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
SCALES = torch.arange(127, dtype=torch.uint8).view(F8).double()


# ------------------------------------------------------------------------------------- reference

def nearest(x, values):
    """Index of the value nearest to each x >= 0 (64 bits), ties to the even index, by counting the borders below."""
    borders = (values[1:] + values[:-1]) / 2
    out = torch.zeros(x.shape, dtype=torch.int64)
    for i, b in enumerate(borders.tolist()):
        out += ((x > b) | ((x == b) & (i % 2 == 1))).long()
    return out


def stored(x, factor):
    """(codes, scales) of x [..., dim] in 64 bits, on the CPU, as whole numbers."""
    x = x.double().cpu().unflatten(-1, (-1, 16))
    factor = float(torch.tensor(factor, dtype=F32))
    top = x.abs().amax(-1)
    scale = nearest(torch.nan_to_num(top, nan=0.0, posinf=1e300) / (6 * factor), SCALES)
    unit = (SCALES[scale].float() * torch.tensor(factor, dtype=F32)).double()[..., None]
    size = torch.where(unit > 0, torch.nan_to_num(x.abs(), nan=0.0, posinf=1e300) / unit.clamp(min=1e-300), 0.0)
    code = nearest(size, MAGNITUDES) + 8 * (x < 0).long()
    nan = top.isnan()
    return torch.where(nan[..., None], 0, code).flatten(-2), torch.where(nan, 127, scale)


def unpacked(codes):
    c = codes.cpu().long()
    return torch.stack((c & 15, c >> 4), -1).flatten(-2)


def held(pool, factor):
    """What a pool holds, in 64 bits, on the pool's device."""
    codes, scales = pool
    c = unpacked(codes)
    value = MAGNITUDES[c & 7] * torch.where(c > 7, -1.0, 1.0)
    unit = (scales.contiguous().cpu().float() * torch.tensor(factor, dtype=F32)).double()
    return (value.unflatten(-1, (-1, 16)) * unit[..., None]).flatten(-2).to(codes.device)


def bits(scales):
    return scales.contiguous().view(torch.uint8).cpu().long()


def same_codes(got, want, scale, name):
    """Codes equal, a zero of either sign counting as one."""
    got, want = (torch.where(c == 8, 0, c) for c in (got, want))
    bad = got != want
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} codes differ"


def pools(pages, page_size, heads, dim, device, order="heads_outer", seed=0):
    """A pool with other contents than zeros, in one of the layouts."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def part(size):
        shape = (pages, heads, page_size, size) if order == "heads_outer" else (pages, page_size, heads, size)
        t = torch.randint(0, 100, shape, generator=g, device=device, dtype=torch.uint8)
        return t.transpose(1, 2) if order == "heads_outer" else t
    codes, scales = part(dim // 2), part(dim // 16)
    if order == "unaligned":  # scales that begin at an odd byte, codes at 8 bytes that are not 16
        buf = torch.randint(0, 100, (codes.numel() + 8,), generator=g, device=device, dtype=torch.uint8)
        codes = buf[8:].view(codes.shape)
        buf = torch.randint(0, 100, (scales.numel() + 1,), generator=g, device=device, dtype=torch.uint8)
        scales = buf[1:].view(scales.shape)
    elif order == "one_buffer":  # a page's head: its codes, then its scales
        row = page_size * (dim // 2 + dim // 16)
        row += -row % 8
        buf = torch.randint(0, 100, (pages, heads, row), generator=g, device=device, dtype=torch.uint8)
        codes = buf[..., :page_size * dim // 2].unflatten(-1, (page_size, dim // 2)).transpose(1, 2)
        scales = buf[..., page_size * dim // 2:page_size * (dim // 2 + dim // 16)].unflatten(-1, (page_size, dim // 16)).transpose(1, 2)
    return codes, scales.view(F8)


# ------------------------------------------------------------------------------------- writing

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("order", ["heads_outer", "slots_outer", "unaligned", "one_buffer"])
@pytest.mark.parametrize("tokens, hq, hk, dim, rot, page_size, interleaved, factor", [
    (1, 4, 1, 64, 64, 16, False, 1.0), (45, 8, 2, 128, 64, 7, True, 0.375), (200, 6, 6, 48, 20, 1, False, 1.0),
    (64, 0, 3, 96, 0, 32, False, 0.5), (5, 3, 1, 16, 4, 3, True, 2.0), (33, 2, 2, 80, 30, 16, True, 251 / 4096),
    (33, 2, 2, 80, 34, 16, False, 0.3), (1100, 4, 2, 128, 128, 64, False, 1.0), (9, 1, 1, 1024, 1024, 4, False, 1.0),
    (17, 8, 4, 256, 96, 8, False, 3e-5),
])
def test_written_codes_are_those_of_the_real_values(cuda_device, dtype, order, tokens, hq, hk, dim, rot, page_size,
                                                    interleaved, factor):
    pages = -(-2 * tokens // page_size) + 2
    q = normal((tokens, hq, dim), dtype, 1, cuda_device) if hq else None
    k, v = normal((tokens, hk, dim), dtype, 2, cuda_device), normal((tokens, hk, dim), dtype, 3, cuda_device)
    kp, vp = pools(pages, page_size, hk, dim, cuda_device, order, 4), pools(pages, page_size, hk, dim, cuda_device, order, 5)
    before = [t.clone() for t in (kp[0], bits(kp[1]), vp[0], bits(vp[1]))]
    g = torch.Generator().manual_seed(6)
    slots = torch.randperm(pages * page_size, generator=g)[:tokens]
    slots[tokens // 2::5] = -1 if tokens > 1 else slots[0]  # padding tokens
    pos = torch.randint(0, 1 << 18, (tokens,), generator=g)
    steps = ks.rotary_steps(rot, device=cuda_device) if rot else None
    out = ks.rotary_to_pages_4bit(q, k, v, pos.to(cuda_device) if rot else None, steps, kp, vp, slots.to(cuda_device),
                                  interleaved=interleaved, k_scale=factor, v_scale=2 * factor)
    f = freqs(rot) if rot else torch.zeros(0, dtype=torch.float64)
    if hq:
        close(out, *rotated(q, pos, f, interleaved), "q")
    else:
        assert out is None
    live = [t for t in range(tokens) if slots[t] >= 0]
    at = slots[live] // page_size, slots[live] % page_size
    there = tuple(i.to(cuda_device) for i in at)
    for pool, x, g_, name in ((kp, rotated(k, pos, f, interleaved)[0], factor, "k"), (vp, v, 2 * factor, "v")):
        codes, scales = stored(x[live], g_)
        assert torch.equal(bits(pool[1])[at], scales), f"{name}'s scales"
        same_codes(unpacked(pool[0][there]), codes, scales, name)
    untouched = torch.ones(pages, page_size, dtype=torch.bool)
    untouched[at] = False
    for now, then in zip((kp[0].cpu(), bits(kp[1]), vp[0].cpu(), bits(vp[1])), before):
        assert torch.equal(now[untouched], then.cpu()[untouched])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("factor", [1.0, 0.5, 0.3, 1.7e-3])
def test_borders_and_ties(cuda_device, dtype, factor):
    """Values on the borders between codes and groups on the borders between scales, and their neighbours."""
    g = torch.Generator().manual_seed(11)
    f = float(torch.tensor(factor, dtype=F32))
    tops = (SCALES[1:] + SCALES[:-1]) / 2 * 6 * f  # groups whose largest value lies on a border of the scale
    rows = []
    for top in torch.cat((tops, SCALES[1:] * 6 * f, SCALES[40:60] * 6.3 * f)).tolist():
        s = float(SCALES[nearest(torch.tensor([top / (6 * f)], dtype=torch.float64), SCALES)[0]])
        u = float(torch.tensor(s, dtype=F32) * torch.tensor(f, dtype=F32))
        edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0, 6.0, 4.0, 0.3, 1.0, 2.0, 3.0, 0.5]) * u
        sign = torch.randint(0, 2, (15,), generator=g) * 2 - 1
        rows.append(torch.cat((torch.tensor([top], dtype=torch.float64), edge.double() * sign)))
    x = torch.stack(rows)
    x = torch.cat((x, x * (1 + 2.0 ** -7), x * (1 - 2.0 ** -7), x * (1 + 2.0 ** -22), x * (1 - 2.0 ** -22))).to(dtype)
    k = x.view(-1, 1, 16).to(cuda_device)
    n = k.shape[0]
    slots = torch.arange(n, device=cuda_device)
    zero = torch.zeros(n, dtype=torch.int64, device=cuda_device)
    for steps in (None, ks.rotary_steps(16, device=cuda_device)):  # as they are, and turned by nothing
        kp, vp = ks.empty_pages_4bit(n, 1, 1, 16, device=cuda_device), ks.empty_pages_4bit(n, 1, 1, 16, device=cuda_device)
        ks.rotary_to_pages_4bit(None, k, k, None if steps is None else zero, steps, kp, vp, slots, k_scale=factor, v_scale=factor)
        codes, scales = stored(k.float(), factor)
        for pool in (kp, vp):
            assert torch.equal(bits(pool[1])[:, 0], scales)
            same_codes(unpacked(pool[0])[:, 0], codes, scales, "ties")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("turned", [False, True])
def test_written_values_that_are_not_ordinary(cuda_device, dtype, turned):
    k = normal((12, 2, 32), dtype, 1, cuda_device)
    k[0, 0, 3] = math.nan
    k[1, 1, 20], k[2, 0, 0] = math.inf, -math.inf
    k[3] = 0.0
    k[4], k[5] = k[4] * 1e-3, k[5] * torch.finfo(dtype).tiny
    k[6] = torch.finfo(dtype).max
    k[7] = -0.0
    k[8] = (k[8] * 3000).to(dtype)  # past the largest scale
    k[9, 0, :16] = 0.0
    slots = torch.arange(12, device=cuda_device)
    kp, vp = ks.empty_pages_4bit(3, 4, 2, 32, device=cuda_device), ks.empty_pages_4bit(3, 4, 2, 32, device=cuda_device)
    zero = torch.zeros(12, dtype=torch.int64, device=cuda_device)
    steps = ks.rotary_steps(32, device=cuda_device) if turned else None
    ks.rotary_to_pages_4bit(None, k, k, zero if turned else None, steps, kp, vp, slots)
    for pool, rotates in ((kp, turned), (vp, False)):
        x = k.double()
        if rotates:  # a turn by nothing: an infinity or NaN spoils its partner, by way of 0 times infinity
            for t, h, d in ((0, 0, 3), (1, 1, 20), (2, 0, 0)):
                x[t, h, d ^ 16] = math.nan
        codes, scales = stored(x, 1.0)
        assert torch.equal(bits(pool[1]).view(12, 2, 2), scales)
        live = (scales < 127).repeat_interleave(16, -1)
        same_codes(unpacked(pool[0]).view(12, 2, 32)[live], codes[live], scales, "values")
    back, _ = ks.pages_4bit_to_rows(vp, vp, slots, dtype=F32)
    assert bool(back[0, 0, :16].isnan().all()) and bool(back[0, 0, 16:].isfinite().all())
    assert float(back[1, 1, 20]) == 2688.0 and float(back[2, 0, 0]) == -2688.0
    assert not bool(back[3].any()) and not bool(back[7].any()) and not bool(back[9, 0, :16].any())


def test_written_slots_beyond_the_pool_are_left_out_and_reported(cuda_device):
    k = normal((3, 2, 64), BF16, 1, cuda_device)
    kp, vp = pools(2, 8, 2, 64, cuda_device, seed=2), pools(2, 8, 2, 64, cuda_device, seed=3)
    before = [kp[0].clone(), bits(kp[1]), vp[0].clone(), bits(vp[1])]
    ks.rotary_to_pages_4bit(None, k, k, None, None, kp, vp, torch.tensor([16, -1, 1 << 40], device=cuda_device))
    assert faults() == _abi.KS_FAULT_BAD_INDEX
    for now, then in zip((kp[0], bits(kp[1]), vp[0], bits(vp[1])), before):
        assert torch.equal(now, then)
    rows, _ = ks.pages_4bit_to_rows(kp, vp, torch.tensor([16, 3, -1, 1 << 40], device=cuda_device))
    assert faults() == _abi.KS_FAULT_BAD_INDEX
    assert not bool(rows[0].any()) and not bool(rows[2:].any()) and bool(rows[1].any())


def test_projection_views_and_scale(cuda_device):
    """q, k and v as parts of one projection, q turned in place, a factor on the rotated values."""
    tokens, hq, hk, dim = 33, 8, 2, 128
    qkv = normal((tokens, (hq + 2 * hk) * dim), BF16, 9, cuda_device)
    q, k, v = (t.view(tokens, -1, dim) for t in qkv.split([hq * dim, hk * dim, hk * dim], 1))
    pos = torch.arange(tokens)
    (wq, tq), (wk, _) = rotated(q, pos, freqs(dim), False, scale=1.25), rotated(k, pos, freqs(dim), False, scale=1.25)
    kp, vp = ks.empty_pages_4bit(3, 16, hk, dim, device=cuda_device), ks.empty_pages_4bit(3, 16, hk, dim, device=cuda_device)
    wv = v.clone()
    out = ks.rotary_to_pages_4bit(q, k, v, pos.to(cuda_device), ks.rotary_steps(dim, device=cuda_device), kp, vp,
                                  torch.arange(tokens, device=cuda_device), scale=1.25, out=q)
    assert out is q
    close(q, wq, tq, "q")
    for pool, x in ((kp, wk), (vp, wv)):
        codes, scales = stored(x, 1.0)
        assert torch.equal(bits(pool[1]).flatten(0, 1)[:tokens], scales)
        same_codes(unpacked(pool[0]).flatten(0, 1)[:tokens], codes, scales, "parts")


# ------------------------------------------------------------------------------------- reading back

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("order", ["heads_outer", "slots_outer", "unaligned", "one_buffer"])
@pytest.mark.parametrize("tokens, hk, dim, page_size, factor", [
    (1, 1, 16, 1, 1.0), (300, 2, 128, 16, 0.5), (77, 3, 80, 7, 0.3), (1025, 8, 64, 64, 1.0), (5, 70, 256, 4, 1e-4),
    (3, 2, 1024, 8, 2.0),
])
def test_rows_are_what_is_held(cuda_device, dtype, order, tokens, hk, dim, page_size, factor):
    pages = -(-tokens // page_size) + 1
    kp, vp = pools(pages, page_size, hk, dim, cuda_device, order, 1), pools(pages, page_size, hk, dim, cuda_device, order, 2)
    slots = torch.randint(0, pages * page_size, (tokens,), generator=torch.Generator().manual_seed(3))  # some twice
    slots[1::7] = -1
    live = slots >= 0
    at = (slots[live] // page_size, slots[live] % page_size)
    for layout in ("new", "head_major", "unaligned", "parts"):
        out = None
        if layout == "head_major":
            out = tuple(torch.full((hk, tokens, dim), 7.0, dtype=dtype, device=cuda_device).transpose(0, 1) for _ in range(2))
        elif layout == "unaligned":
            out = tuple(torch.zeros(tokens * hk * dim + 1, dtype=dtype, device=cuda_device)[1:].view(tokens, hk, dim) for _ in range(2))
        elif layout == "parts":
            both = torch.zeros(tokens, hk, 2, dim, dtype=dtype, device=cuda_device)
            out = both[:, :, 0], both[:, :, 1]
        got = ks.pages_4bit_to_rows(kp, vp, slots.to(cuda_device), k_scale=factor, v_scale=3 * factor, dtype=dtype, out=out)
        assert out is None or (got[0] is out[0] and got[1] is out[1])
        for rows, pool, f in zip(got, (kp, vp), (factor, 3 * factor)):
            want = held(pool, f)[tuple(i.to(cuda_device) for i in at)]
            # u * code is rounded to FP32, then to the type
            tol = want.abs() * (2.0 ** -24 + (torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -23) if dtype != F32 else 0.0))
            tol = tol + (2.0 ** -25 if dtype == F16 else 0.0)
            close(rows[live.to(cuda_device)], want, tol, layout)
            assert not bool(rows[~live.to(cuda_device)].any())


# ------------------------------------------------------------------------------------- attention

def check_rows(out, q, k, v, keys, causal, scale, name):
    """One sequence's rows: q [n, Hq, D] against k, v [keys, Hk, D] in 64 bits."""
    n, hq, dim = q.shape
    if n == 0:
        return
    if keys == 0:
        assert not bool(out.any()), name
        return
    group = hq // k.shape[1]
    kk, vv = (t.double().repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))
    qq = q.double().transpose(0, 1)
    s = qq @ kk.transpose(1, 2) * scale
    mag = (qq.abs() @ kk.abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(scale) * (dim + 8) * 2.0 ** -23
    if q.dtype == BF16:
        mag = mag + qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).amax(-1)[:, None, None] * abs(scale) * 2.0 ** -25
    j, i = torch.arange(keys, device=q.device), torch.arange(n, device=q.device)
    sees = (j < keys - n + i[:, None] + 1) if causal else torch.ones(n, keys, dtype=torch.bool, device=q.device)
    s = s.masked_fill(~sees, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
    l = p.sum(-1, keepdim=True)
    inv = torch.where(l > 0, 1 / l, 0.0)
    want, share = (p @ vv) * inv, (p @ vv.abs()) * inv
    tol = share * (2.0 ** -11 + 2 * (mag + 2.0 ** -21) + 4 * keys * 2.0 ** -23)
    tol = tol + keys * 2.0 ** -33 * vv.abs().amax() * inv
    tol = tol + torch.finfo(q.dtype).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if q.dtype == F16 else 0.0)
    close(out.transpose(0, 1), want, tol, name)
    assert not bool(out[(~sees.any(-1))].any()), f"{name}: rows that see nothing must be 0"


def build(q_lens, kv_lens, hq, hk, dim, dtype, page_size, device, seed=0, order="heads_outer", extra_rows=0,
          k_scale=1.0, v_scale=1.0, spoil=True, ordinary=True):
    """Sequences in a shuffled pool. What no sequence owns holds codes and NaN scales, and table entries past a
    sequence's pages are out of range."""
    pool = sum(-(-n // page_size) for n in kv_lens) + 2
    kp, vp = (pools(pool, page_size, hk, dim, device, order, seed + i) for i in (1, 2))
    if spoil:
        for p in (kp, vp):
            p[1].view(torch.uint8).fill_(127)
    width = max(1, max(-(-n // page_size) for n in kv_lens))
    table = torch.full((len(kv_lens), width), -7, dtype=torch.int32)
    perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    ks_, vs_, at = [], [], 0
    for b, n in enumerate(kv_lens):
        need = -(-n // page_size)
        mine = perm[at:at + need]
        at += need
        table[b, :need] = torch.tensor(mine, dtype=torch.int32)
        rows = torch.arange(n)
        pg, pl = torch.tensor(mine, dtype=torch.int64)[rows // page_size].to(device), (rows % page_size).to(device)
        for p, f, into, s0 in ((kp, k_scale, ks_, 10), (vp, v_scale, vs_, 50)):
            x = normal((n, hk, dim), F32, seed + s0 + b, device)
            c, s = stored(x, f)
            p[0][pg, pl] = (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8).to(device)
            p[1].view(torch.uint8)[pg, pl] = s.to(torch.uint8).to(device)
            into.append(held((p[0][pg, pl], p[1].view(torch.uint8)[pg, pl].view(F8)), f))
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    q = normal((starts[-1] + extra_rows, hq, dim), dtype, seed + 3, device)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(q=q, kp=kp, vp=vp, table=table.to(device), kv=torch.tensor(kv_lens, **i32), starts=torch.tensor(starts, **i32),
                k=ks_, v=vs_, q_lens=q_lens, kv_lens=kv_lens, s=starts, f=dict(k_scale=k_scale, v_scale=v_scale))


def check_all(out, st, causal=True, scale=None, name=""):
    scale = st["q"].shape[2] ** -0.5 if scale is None else scale
    for b, n in enumerate(st["q_lens"]):
        lo = st["s"][b]
        check_rows(out[lo:lo + n], st["q"][lo:lo + n], st["k"][b], st["v"][b], st["kv_lens"][b], causal, scale,
                   f"{name} sequence {b} ({n} over {st['kv_lens'][b]})")


def attend(st, **kw):
    return ks.paged_attention_4bit(st["q"], st["kp"], st["vp"], st["table"], st["kv"], st["starts"], **st["f"], **kw)


STEP = ([1] * 7, [1, 2, 63, 64, 65, 200, 1111])
CHUNK = ([5, 0, 130, 1, 33, 300], [5, 77, 130, 400, 65, 801])
BLIND = ([3, 4, 2, 40, 1], [0, 2, 2, 17, 0])       # fewer keys than new tokens, and none
PROMPT = ([257, 700], [257, 1500])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens", [STEP, CHUNK, BLIND, PROMPT], ids=["step", "chunk", "blind", "prompt"])
@pytest.mark.parametrize("hq, hk, dim, page_size", [
    (8, 1, 128, 16), (4, 4, 64, 32), (10, 2, 128, 128), (6, 2, 96, 7), (3, 3, 256, 16), (40, 2, 64, 8), (7, 1, 80, 64),
    (32, 8, 128, 1), (2, 1, 16, 256), (160, 1, 128, 48), (4, 2, 192, 16), (6, 3, 176, 32), (5, 1, 48, 16), (2, 2, 240, 24),
])
def test_attention_matches_64_bits(cuda_device, dtype, lens, hq, hk, dim, page_size):
    st = build(*lens, hq, hk, dim, dtype, page_size, cuda_device, seed=hq + dim, k_scale=0.5, v_scale=0.3)
    check_all(attend(st), st)
    # the hint only picks the kernel
    for hint in (1, max(lens[0])):
        check_all(attend(st, max_q_len=hint), st, name=f"hint {hint}")


@pytest.mark.parametrize("lens", [STEP, CHUNK, BLIND], ids=["step", "chunk", "blind"])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_without_causal_and_with_scale(cuda_device, lens, dim):
    st = build(*lens, 8, 2, dim, BF16, 16, cuda_device, seed=3)
    for scale in (0.3, -0.05, 0.0):
        check_all(attend(st, causal=False, scale=scale), st, causal=False, scale=scale)


@pytest.mark.parametrize("order", ["heads_outer", "slots_outer", "unaligned", "one_buffer"])
@pytest.mark.parametrize("q_layout", ["packed", "head_major", "projection"])
@pytest.mark.parametrize("dim, page_size, hint", [(64, 16, None), (128, 16, None), (128, 5, None), (256, 32, None), (128, 16, 1)])
def test_attention_strides_and_rows_left_alone(cuda_device, order, q_layout, dim, page_size, hint):
    st = build([3, 20, 1], [50, 300, 129], 8, 4, dim, F16, page_size, cuda_device, order=order, extra_rows=5)
    total = st["q"].shape[0]
    if q_layout == "head_major":
        st["q"] = st["q"].transpose(0, 1).contiguous().transpose(0, 1)
    elif q_layout == "projection":
        wide = torch.zeros(total, 16 * dim, dtype=F16, device=cuda_device)
        wide[:, 128:128 + 8 * dim] = st["q"].reshape(total, -1)
        st["q"] = wide[:, 128:128 + 8 * dim].view(total, 8, dim)
    out = torch.full((8, total, dim), 7.0, dtype=F16, device=cuda_device).transpose(0, 1)
    assert attend(st, out=out, max_q_len=hint) is out
    check_all(out, st)
    assert bool((out[-5:] == 7.0).all()), "rows behind the last sequence are left as they were"


@pytest.mark.parametrize("order", ["heads_outer", "slots_outer", "one_buffer"])
@pytest.mark.parametrize("dim", [32, 64, 96, 112, 128])
@pytest.mark.parametrize("page_size", [8, 16, 24, 64, 128, 200, 256])
def test_attention_pages_within_and_beyond_a_step(cuda_device, order, dim, page_size):
    """Many rows over pages that a step of 128 keys is made of, or that it is part of, and that it is neither."""
    st = build([90, 0, 40, 3], [700, 64, 41, 300], 8, 2, dim, BF16, page_size, cuda_device, seed=dim + page_size, order=order,
               k_scale=2.0, v_scale=0.7)
    for causal in (True, False):
        check_all(attend(st, causal=causal), st, causal=causal, name=f"causal {causal}")


@pytest.mark.parametrize("dim", [64, 80, 96, 128])
@pytest.mark.parametrize("group", [1, 4, 5])
def test_attention_of_drafts(cuda_device, dim, group):
    """A few tokens a sequence, on either side of the numbers of rows at which another kernel is taken."""
    for n in (2, 3, 4, 5, 8, 9, 12, 13, 17, 33, 49):
        st = build([n, 1, n - 1, n], [n, 130, 1000, 257], 2 * group, 2, dim, BF16, 16, cuda_device, seed=n)
        check_all(attend(st, max_q_len=n), st, name=f"{n} tokens")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hint", [1, 200])
def test_attention_large_and_small_queries(cuda_device, dtype, hint):
    """Rows of queries whose sizes differ by many powers of two, and within a row; the scores are brought back."""
    st = build([1, 200], [777, 777], 4, 2, 128, dtype, 16, cuda_device, seed=8)
    size = torch.exp2(torch.linspace(-14, 8, 201 * 4, device=cuda_device)).view(201, 4, 1)
    within = torch.exp2(torch.linspace(0, -20 if dtype == BF16 else -8, 128, device=cuda_device))
    st["q"] = (st["q"].float() * size * within).to(dtype)
    check_all(attend(st, max_q_len=hint), st)
    st["q"] = (st["q"].float() * -0.01).to(dtype)
    st["q"][3, 1] = 0.0
    check_all(attend(st, scale=1.0, max_q_len=hint), st, scale=1.0)


def test_attention_of_far_queries_in_bf16(cuda_device):
    """Queries near the ends of bf16's range, scores brought back by the scale."""
    for power, scale in ((1e30, 1e-31), (1e-30, 1e29), (3e38, 1e-39), (1e-38, 1e37)):
        for hint, n in ((1, 1), (40, 40)):
            st = build([n], [100], 4, 2, 64, BF16, 16, cuda_device, seed=5)
            st["q"] = (st["q"].double() / st["q"].double().abs().max() * power).to(BF16)
            check_all(attend(st, scale=scale, max_q_len=hint), st, scale=scale)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 7, 90]])
def test_attention_non_finite_keys_stay_in_their_sequence(cuda_device, q_lens):
    st = build(q_lens, [150, 100, 200], 8, 2, 128, BF16, 16, cuda_device, seed=2)
    st["kp"][1].view(torch.uint8)[int(st["table"][1, 2]), 3] = 127
    st["vp"][1].view(torch.uint8)[int(st["table"][1, 2]), 3] = 127
    lo, hi = st["s"][1], st["s"][2]
    st["q"][lo:hi, 3] = math.nan
    out = attend(st, max_q_len=max(q_lens))
    assert bool(out[lo:hi].isnan().all())
    for b in (0, 2):
        at, n = st["s"][b], st["q_lens"][b]
        check_rows(out[at:at + n], st["q"][at:at + n], st["k"][b], st["v"][b], st["kv_lens"][b], True, 128 ** -0.5, "neighbour")


@pytest.mark.parametrize("q_lens, kv_lens, hq, hk, dim, page_size", [
    ([2000], [2000], 4, 1, 128, 128),          # many row tiles of one sequence, split among the CTAs
    ([40, 3], [700, 2900], 320, 1, 64, 32),    # a group of more heads than a row tile has rows
    ([1] * 40 + [600], [3000] * 40 + [900], 8, 4, 128, 64),
    ([33], [33], 1, 1, 96, 8), ([17, 18, 19], [128, 256, 384], 2, 2, 112, 384), ([1, 2], [9000, 5000], 64, 4, 128, 16),
    ([2, 1], [5000, 9000], 16, 2, 128, 16),
])
def test_attention_shapes_of_work(cuda_device, q_lens, kv_lens, hq, hk, dim, page_size):
    st = build(q_lens, kv_lens, hq, hk, dim, BF16, page_size, cuda_device, seed=30)
    check_all(attend(st, max_q_len=max(q_lens)), st)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hint, n", [(1, 1), (64, 64)])
@pytest.mark.parametrize("powers", [5, 7.9, 8.1, 13.9, 15.9, 16.1, 24, 60])
@pytest.mark.parametrize("negative", [False, True])
def test_scores_that_outgrow_the_first_keys(cuda_device, dtype, dim, hint, n, powers, negative):
    """A key late in the sequence scores 2^powers times what the others do, in the exponent's base."""
    st = build([n], [1500], 2, 1, dim, dtype, 16, cuda_device, seed=40)
    st["q"] = torch.zeros_like(st["q"])
    st["q"][..., 0] = 1.0
    one = torch.zeros(1500, 1, dim, device=cuda_device)
    one[700, 0, 0], one[1400, 0, 0] = 3.0, 6.0
    rows = torch.arange(1500, device=cuda_device)
    pg, pl = st["table"][0].long()[rows // 16], rows % 16
    c, s = stored(one, 1.0)
    st["kp"][0][pg, pl] = (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8).to(cuda_device)
    st["kp"][1].view(torch.uint8)[pg, pl] = s.to(torch.uint8).to(cuda_device)
    st["k"][0] = held((st["kp"][0][pg, pl], st["kp"][1].view(torch.uint8)[pg, pl].view(F8)), 1.0)
    scale = powers * math.log(2.0) / 6.0
    if negative:
        st["q"], scale = -st["q"], -scale
    check_all(attend(st, scale=scale, max_q_len=hint, causal=False), st, causal=False, scale=scale)


def test_attention_bad_indices_are_reported(cuda_device):
    """A page outside the pool reads as zeros; lengths and starts are brought into range."""
    for n in (2, 40):
        st = build([1, n], [40, 30], 2, 1, 64, BF16, 16, cuda_device, seed=4, spoil=False)
        good = attend(st)
        st["table"][0, 1] = 10 ** 6
        out = attend(st)
        assert faults() == _abi.KS_FAULT_BAD_INDEX
        k, v = st["k"][0].clone(), st["v"][0].clone()
        k[16:32], v[16:32] = 0, 0
        check_rows(out[:1], st["q"][:1], k, v, 40, True, 64 ** -0.5, "zeros")
        assert torch.equal(out[1:], good[1:])
        st["table"][0, 1] = -1
        attend(st)
        assert faults() == _abi.KS_FAULT_BAD_INDEX
        st = build([1, n], [48, 30], 2, 1, 64, BF16, 16, cuda_device, seed=4, spoil=False)
        st["kv"][0] = 10 ** 6  # more keys than the table has room for
        check_rows(attend(st)[:1], st["q"][:1], st["k"][0], st["v"][0], 48, True, 64 ** -0.5, "room")
        assert faults() == _abi.KS_FAULT_BAD_INDEX
        st["kv"][0], st["starts"][2] = -5, 100
        out = attend(st)
        assert faults() == _abi.KS_FAULT_BAD_INDEX and not bool(out[0].any())


def test_empty_calls(cuda_device):
    st = build([2, 1], [20, 30], 2, 1, 64, BF16, 16, cuda_device)
    assert attend({**st, "q": st["q"][:0], "starts": st["starts"] * 0}).shape == (0, 2, 64)
    out = torch.full_like(st["q"], 3.0)
    none = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    ks.paged_attention_4bit(st["q"], st["kp"], st["vp"], st["table"][:0], none,
                            torch.zeros(1, dtype=torch.int32, device=cuda_device), out=out)
    attend({**st, "starts": st["starts"] * 0}, out=out)
    assert bool((out == 3.0).all())
    empty = ks.empty_pages_4bit(0, 16, 1, 64, device=cuda_device)
    out = ks.paged_attention_4bit(st["q"], empty, empty, st["table"][:, :0], st["kv"] * 0, st["starts"])
    assert not bool(out.any())
    k = torch.zeros(0, 1, 64, dtype=BF16, device=cuda_device)
    i = torch.zeros(0, dtype=torch.int64, device=cuda_device)
    assert ks.rotary_to_pages_4bit(None, k, k, None, None, st["kp"], st["vp"], i) is None
    rows, _ = ks.pages_4bit_to_rows(st["kp"], st["vp"], i)
    assert rows.shape == (0, 1, 64)
    rows, _ = ks.pages_4bit_to_rows(empty, empty, torch.full((3,), -1, device=cuda_device))
    assert rows.shape == (3, 1, 64) and not bool(rows.any())


def test_attention_many_sequences(cuda_device):
    """More sequences than threads of a block, most of them without new tokens."""
    seqs, page = 1500, 8
    g = torch.Generator().manual_seed(1)
    kv = torch.randint(0, 40, (seqs,), generator=g).tolist()
    ql = [(1 if i % 7 == 0 else 3 if i % 11 == 0 else 0) for i in range(seqs)]
    need = [-(-n // page) for n in kv]
    kp, vp = (pools(sum(need), page, 2, 64, cuda_device, "slots_outer", i) for i in (1, 2))
    table = torch.zeros(seqs, 5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    starts = torch.tensor([0] + ql).cumsum(0).int()
    q = normal((int(starts[-1]), 4, 64), BF16, 3, cuda_device)
    kk, vv = (held(p, 1.0).view(-1, 2, 64) for p in (kp, vp))
    for hint in (None, 3):
        out = ks.paged_attention_4bit(q, kp, vp, table.to(cuda_device), torch.tensor(kv, dtype=torch.int32, device=cuda_device),
                                      starts.to(cuda_device), max_q_len=hint, scale=0.001)
        for b in range(0, seqs, 77):
            lo, hi = int(starts[b]), int(starts[b + 1])
            first = int(table[b, 0]) * page if need[b] else 0
            check_rows(out[lo:hi], q[lo:hi], kk[first:first + kv[b]], vv[first:first + kv[b]], kv[b], True, 0.001, f"sequence {b}")


def test_pool_beyond_31_bit_offsets(cuda_device):
    """Pools of more than 2^32 bytes: slots, pages and attention address them in 64 bits."""
    page_size, hk, dim = 64, 8, 128
    pages = (1 << 32) // (page_size * hk * dim // 2) + 40
    kp, vp = ks.empty_pages_4bit(pages, page_size, hk, dim, device=cuda_device), ks.empty_pages_4bit(pages, page_size, hk, dim, device=cuda_device)
    n = 100
    k, v = normal((n, hk, dim), BF16, 1, cuda_device), normal((n, hk, dim), BF16, 2, cuda_device)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=cuda_device)
    t = torch.arange(n, device=cuda_device)
    slots = table[0].long()[t // page_size] * page_size + t % page_size
    ks.rotary_to_pages_4bit(None, k, v, None, None, kp, vp, slots)
    kk, vv = (t.double() for t in ks.pages_4bit_to_rows(kp, vp, slots, dtype=F32))
    for x, pool, back in ((k, kp, kk), (v, vp, vv)):
        c, s = stored(x, 1.0)
        assert torch.equal(back.cpu(), (MAGNITUDES[c & 7] * torch.where(c > 7, -1.0, 1.0)) * SCALES[s].repeat_interleave(16, -1))
    q = normal((n, hk, dim), BF16, 3, cuda_device)
    for few in (1, n):
        out = ks.paged_attention_4bit(q[-few:].contiguous(), kp, vp, table, torch.tensor([n], dtype=torch.int32, device=cuda_device),
                                      torch.tensor([0, few], dtype=torch.int32, device=cuda_device), max_q_len=few)
        check_rows(out, q[-few:], kk, vv, n, True, dim ** -0.5, "far pages")


def test_longest_context(cuda_device):
    """As many keys as a sequence may have, 2^31 - 1024: places ahead of the last key do not wrap. One page of 2^20 keys
    lies behind every table entry, so that a key counts 2048 times, the last 1024 of the page 2047 times.

    Some of the sums have 2^31 / 128 / 608 < 28000 steps, of two matrix instructions each for an output, whose FP32 sums
    may truncate (2^-23 of a running sum, which is below l max|v|) and of one addition for l (2^-24): 0.0085 max|v| at most,
    and 2^-8 + 2^-11 max|v| for the output's and the probabilities' roundings."""
    page_size, dim, hq, keys = 1 << 20, 64, 8, 0x7ffffc00
    kp, vp = (ks.empty_pages_4bit(1, page_size, 1, dim, device=cuda_device) for _ in range(2))
    g = torch.Generator(device=cuda_device).manual_seed(4)
    kp[0].copy_(torch.randint(0, 256, kp[0].shape, dtype=torch.uint8, device=cuda_device, generator=g))
    # values of 6 and of 0.5, the first more often the higher the dim
    large = torch.rand(page_size, dim, device=cuda_device, generator=g) < torch.arange(dim, device=cuda_device) / dim
    codes = torch.where(large, 7, 1).to(torch.uint8)
    vp[0].copy_((codes[:, 0::2] | codes[:, 1::2] << 4)[None, :, None])
    for p in (kp, vp):
        p[1].view(torch.uint8).fill_(0x38)  # 1
    q = normal((1, hq, dim), BF16, 6, cuda_device)
    i32 = dict(dtype=torch.int32, device=cuda_device)
    out = ks.paged_attention_4bit(q, kp, vp, torch.zeros(1, 2048, **i32), torch.tensor([keys], **i32), torch.tensor([0, 1], **i32),
                                  scale=0.03, max_q_len=1)
    count = torch.full((page_size,), 2048.0, dtype=torch.float64, device=cuda_device)
    count[-1024:] = 2047
    k = held((kp[0][0, :, 0], kp[1][0, :, 0]), 1.0)
    p = torch.exp(q[0].double() @ k.T * 0.03) * count
    want = p @ torch.where(large, 6.0, 0.5).double() / p.sum(-1, keepdim=True)
    close(out[0], want, torch.full_like(want, 6 * (0.0085 + 2.0 ** -8 + 2.0 ** -11)), "the longest context")


@pytest.mark.parametrize("lens", [STEP, PROMPT], ids=["step", "prompt"])
def test_attention_is_reproducible_and_takes_a_workspace(cuda_device, lens):
    st = build(*lens, 8, 2, 128, BF16, 16, cuda_device, seed=5)
    most = max(lens[0])
    first = attend(st, max_q_len=most)
    need = ks.paged_attention_4bit_workspace(st["q"].shape[0], len(lens[0]), 8, 2, 128, 16, st["table"].shape[1], BF16,
                                             max_q_len=most, device=cuda_device)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=cuda_device)
    for _ in range(3):
        assert torch.equal(attend(st, workspace=ws, max_q_len=most), first)
    with pytest.raises(_abi.KsError):
        attend(st, workspace=ws[:64], max_q_len=most)
    with pytest.raises(_abi.KsError):
        attend(st, workspace=st["kp"][0].transpose(1, 2).flatten(), max_q_len=most)


@pytest.mark.parametrize("dim", [64, 80, 128, 192, 256])
def test_workspace_never_grows_with_less(cuda_device, dim):
    def need(tokens, seqs, width, most):
        return ks.paged_attention_4bit_workspace(tokens, seqs, 8, 2, dim, 16, width, BF16, max_q_len=most, device=cuda_device)
    sizes = [need(t, s, w, m) for t, s, w, m in ((4096, 64, 512, 4096), (1000, 64, 512, 1000), (1000, 8, 512, 1000),
                                                 (1000, 8, 5, 1000), (20, 8, 5, 20), (8, 8, 5, 1), (1, 1, 1, 1))]
    assert sizes == sorted(sizes, reverse=True) and sizes[-1] > 0


# ------------------------------------------------------------------------------------- refusals

def test_refusals(cuda_device):
    k = normal((3, 2, 64), BF16, 1, cuda_device)
    kp, vp = ks.empty_pages_4bit(4, 8, 2, 64, device=cuda_device), ks.empty_pages_4bit(4, 8, 2, 64, device=cuda_device)
    slots = torch.arange(3, device=cuda_device)
    pos, steps = slots, ks.rotary_steps(64, device=cuda_device)
    with pytest.raises(ValueError):
        ks.empty_pages_4bit(4, 8, 2, 40, device=cuda_device)

    def write(q=k, k=k, v=k, positions=pos, steps=steps, kp=kp, vp=vp, slots=slots, **kw):
        return ks.rotary_to_pages_4bit(q, k, v, positions, steps, kp, vp, slots, **kw)
    for bad in (lambda: write(kp=kp[0]), lambda: write(kp=(kp[0], kp[1].view(torch.uint8))), lambda: write(v=k.half()),
                lambda: write(slots=slots.int()), lambda: write(kp=(kp[0].to(torch.int8), kp[1])), lambda: write(k=k.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: write(kp=(kp[0][:, :, :1], kp[1][:, :, :1])), lambda: write(kp=(kp[0][:2], kp[1])), lambda: write(k_scale=0.0),
                lambda: write(v_scale=math.inf), lambda: write(k_scale=1e30), lambda: write(scale=math.nan), lambda: write(slots=slots[:2]),
                lambda: write(q=k[..., :48], k=k[..., :48], v=k[..., :48]), lambda: write(vp=ks.empty_pages_4bit(5, 8, 2, 64, device=cuda_device)),
                lambda: write(kp=(kp[0].cpu(), kp[1].cpu())), lambda: write(q=None, out=k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        write(k=k.clone().requires_grad_())
    half = torch.zeros(4, 2, 8, 36, dtype=torch.uint8, device=cuda_device)
    for bad in (lambda: write(vp=kp), lambda: write(vp=(vp[0], kp[1])), lambda: write(out=kp[0].view(BF16).flatten()[:3 * 2 * 64].view(3, 2, 64)
                                                                                    if kp[0].is_contiguous() else
                                                                                    kp[0].transpose(1, 2).flatten().view(BF16)[:3 * 2 * 64].view(3, 2, 64)),
                # codes whose rows begin at odd multiples of 4 bytes
                lambda: write(kp=(half[..., :32].transpose(1, 2), kp[1])), lambda: write(kp=(kp[0][:, :1].expand(4, 8, 2, 32), kp[1]))):
        with pytest.raises(_abi.KsError):
            bad()
    for bad in (lambda: ks.pages_4bit_to_rows(kp[0], vp, slots), lambda: ks.pages_4bit_to_rows(kp, vp, slots, dtype=torch.float64),
                lambda: ks.pages_4bit_to_rows(kp, vp, slots.int()), lambda: ks.pages_4bit_to_rows(kp, vp, slots, out=(k.half(), k))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ks.pages_4bit_to_rows(kp, vp, slots, k_scale=-1.0), lambda: ks.pages_4bit_to_rows(kp, vp, slots, out=(k[:2], k[:2])),
                lambda: ks.pages_4bit_to_rows(kp, vp, slots.cpu()), lambda: ks.pages_4bit_to_rows(kp, vp, slots, out=k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_abi.KsError):
        ks.pages_4bit_to_rows(kp, vp, slots, out=(k, k))
    with pytest.raises(RuntimeError):
        ks.pages_4bit_to_rows(kp, vp, slots, out=(k.clone().requires_grad_(), k))
    st = build([1, 2], [40, 30], 4, 2, 64, BF16, 16, cuda_device)
    for bad in (lambda: attend({**st, "q": st["q"].float()}), lambda: attend({**st, "kp": st["kp"][0]}),
                lambda: attend({**st, "table": st["table"].long()}), lambda: attend({**st, "kv": st["kv"].long()})):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: attend({**st, "q": st["q"][:, :3]}), lambda: attend({**st, "starts": st["starts"][:2]}),
                lambda: attend(st, scale=math.inf), lambda: attend(st, max_q_len=-1), lambda: attend({**st, "q": st["q"][..., :48]}),
                lambda: attend(st, out=st["q"][:1]), lambda: attend({**st, "f": dict(k_scale=0)})):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: attend(st, out=st["q"]), lambda: attend(st, scale=3e38)):
        with pytest.raises((_abi.KsError, ValueError)):
            bad()
    with pytest.raises(RuntimeError):
        attend({**st, "q": st["q"].clone().requires_grad_()})


# ------------------------------------------------------------------------------------- together

def test_graph_replays_with_other_lengths(cuda_device):
    """One captured step, replayed with other contents of the lengths, the table and the queries; two graphs at
    once on two streams."""
    st = [build([1, 3, 1], [60, 300, 500], 8, 2, 128, BF16, 16, cuda_device, seed=20 * i) for i in (1, 2)]
    fresh = [build([2, 2, 1], [300, 60, 490], 8, 2, 128, BF16, 16, cuda_device, seed=20 * i) for i in (3, 4)]
    graphs, outs = [], []
    for s in st:
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            attend(s, max_q_len=3)
        torch.cuda.current_stream().wait_stream(warm)
        g = torch.cuda.CUDAGraph()
        # room for the other lengths' pages
        s["kp"], s["vp"] = (ks.empty_pages_4bit(100, 16, 2, 128, device=cuda_device) for _ in range(2))
        with torch.cuda.graph(g):
            outs.append(attend(s, max_q_len=3))
        graphs.append(g)
    for s, f in zip(st, fresh):
        for name in ("q", "table", "kv", "starts"):
            into = s[name][:, :f[name].shape[1]] if name == "table" else s[name]
            into.copy_(f[name])
        for pool in ("kp", "vp"):
            for i in range(2):
                s[pool][i].view(torch.uint8)[:f[pool][i].shape[0]] = f[pool][i].view(torch.uint8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for o, f in zip(outs, fresh):
        check_all(o, f)


@pytest.mark.parametrize("tokens", [3, 1500])
def test_captured_writes_and_norms_replay_with_other_contents(cuda_device, tokens):
    """A norm, a write and a read-back in one graph, replayed with other rows, positions and slots: what eager calls give."""
    hq, hk, dim, page = 6, 2, 128, 32
    steps, w = ks.rotary_steps(dim, device=cuda_device), normal(((hq + 2 * hk) * dim,), BF16, 1, cuda_device)

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        return [normal((tokens, (hq + 2 * hk) * dim), BF16, seed, cuda_device), normal((tokens, (hq + 2 * hk) * dim), BF16, seed + 1, cuda_device),
                torch.randint(0, 1 << 40, (tokens,), generator=g).to(cuda_device), (torch.randperm(64 * page, generator=g)[:tokens] - 1).to(cuda_device)]

    def run(x, r, pos, slots, kp, vp):
        ks.gated_add_rms_norm(x, r, w, block_scale=0.5)
        q, k, v = (t.view(tokens, -1, dim) for t in x.split([hq * dim, hk * dim, hk * dim], 1))
        return [ks.rotary_to_pages_4bit(q, k, v, pos, steps, kp, vp, slots, k_scale=0.5), *ks.pages_4bit_to_rows(kp, vp, slots, k_scale=0.5)]

    def fresh():
        return [ks.empty_pages_4bit(64, page, hk, dim, device=cuda_device) for _ in range(2)]
    held_in, pools_in = inputs(20), fresh()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        run(*inputs(30), *fresh())
    torch.cuda.current_stream().wait_stream(warm)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run(*held_in, *pools_in)
    for seed in (40, 50):
        new, pools_new = inputs(seed), fresh()
        for a, b in zip(held_in, new):
            a.copy_(b)
        for pool in pools_in:
            for t in pool:
                t.view(torch.uint8).zero_()
        g.replay()
        want = run(*new, *pools_new)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([*outs, *held_in[:2]], [*want, *new[:2]]))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for p, n in zip(pools_in, pools_new) for a, b in zip(p, n))


def test_calls_on_another_stream(cuda_device):
    st = build(*CHUNK, 8, 2, 128, BF16, 16, cuda_device, seed=6)
    want = attend(st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [attend(st) for _ in range(4)]
    more = [attend(st) for _ in range(4)]  # at the same time on this one
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got + more)


def test_with_programmatic_dependent_launch(cuda_device):
    """A chain of steps with every launch scheduled early: each kernel waits for the one before."""
    st = build([1, 30, 2], [300, 200, 80], 8, 2, 128, BF16, 16, cuda_device, seed=9)
    pos = torch.arange(33, device=cuda_device)
    steps = ks.rotary_steps(128, device=cuda_device)
    w = normal((128,), BF16, 5, cuda_device)
    seq = torch.tensor([0] * 1 + [1] * 30 + [2] * 2, device=cuda_device)
    rows = st["table"].long()[seq, pos // 16] * 16 + pos % 16

    def chain():
        kp, vp = ([t.clone() for t in p] for p in (st["kp"], st["vp"]))
        x, r, got = st["q"].clone(), st["q"].clone(), []
        for _ in range(6):
            x = ks.rotary_to_pages_4bit(x, x[:, :2].contiguous(), x[:, 2:4].contiguous(), pos, steps, kp, vp, rows)
            x = attend({**st, "q": x, "kp": kp, "vp": vp}, max_q_len=30)
            ks.gated_add_rms_norm(x, r, w, post_weight=w)
            got += [x.clone(), r.clone(), *ks.pages_4bit_to_rows(kp, vp, rows)]
        return got
    want = chain()
    assert _abi.ks_set_launch_options(_abi.KS_LAUNCH_PDL) == _abi.KS_SUCCESS
    try:
        got = chain()
        torch.cuda.synchronize()
    finally:
        _abi.ks_set_launch_options(0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("early", [False, True])
def test_many_tokens_behind_their_producer(cuda_device, early):
    """Queries and pages in kernels of their own (from 1024 tokens on), keys and values written just before them and
    read back just behind them, with and without every launch scheduled early."""
    tokens, hq, hk, dim, page = 3000, 16, 4, 128, 64
    x0 = normal((tokens, (hq + 2 * hk) * dim), BF16, 11, cuda_device)
    w = normal((x0.shape[1],), BF16, 12, cuda_device)
    pos = torch.arange(tokens, device=cuda_device)
    steps = ks.rotary_steps(dim, device=cuda_device)
    slots = torch.randperm(64 * page, generator=torch.Generator().manual_seed(13))[:tokens].to(cuda_device)

    def step(x, kp, vp):
        q, k, v = (t.view(tokens, -1, dim) for t in x.split([hq * dim, hk * dim, hk * dim], 1))
        ks.rotary_to_pages_4bit(q, k, v, pos, steps, kp, vp, slots, out=q)
        return ks.pages_4bit_to_rows(kp, vp, slots)

    def chain(wait):
        x, r, got = x0.clone(), x0.clone(), []
        kp, vp = (ks.empty_pages_4bit(64, page, hk, dim, device=cuda_device) for _ in range(2))
        for _ in range(5):
            ks.gated_add_rms_norm(x, r, w, residual_scale=0.5)
            wait()
            got += step(x, kp, vp)
            wait()
        return [*got, x, r]
    want = chain(torch.cuda.synchronize)
    if early:
        assert _abi.ks_set_launch_options(_abi.KS_LAUNCH_PDL) == _abi.KS_SUCCESS
    try:
        got = chain(lambda: None)
        torch.cuda.synchronize()
    finally:
        _abi.ks_set_launch_options(0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_block_run(cuda_device):
    """A prompt in two chunks and three single tokens of two sequences through a block: norm, projection, rotary
    positions into the 4-bit cache, attention over it, projection, and the norms, gate and add behind it."""
    hidden, hq, hk, dim, page = 512, 8, 2, 64, 16
    g = torch.Generator().manual_seed(7)
    lens = [45, 70]
    x = [torch.randn(n, hidden, generator=g).to(BF16).to(cuda_device) for n in lens]
    w, post, gate = ((1 + 0.1 * torch.randn(hidden, generator=g)).to(BF16).to(cuda_device) for _ in range(3))
    proj = (torch.randn(hidden, (hq + 2 * hk) * dim, generator=g) / hidden ** 0.5).to(BF16).to(cuda_device)
    back = (torch.randn(hq * dim, hidden, generator=g) / hidden ** 0.5).to(BF16).to(cuda_device)
    steps = ks.rotary_steps(dim, device=cuda_device)
    kp, vp = ks.empty_pages_4bit(12, page, hk, dim, device=cuda_device), ks.empty_pages_4bit(12, page, hk, dim, device=cuda_device)
    table = torch.tensor([[4, 1, 9, 0, 0], [2, 3, 5, 7, 11]], dtype=torch.int32, device=cuda_device)
    done, outs, qs, all_k, ends = [0, 0], [[], []], [[], []], [[], []], []
    for n in ([20, 41], [22, 26], [1, 1], [1, 1], [1, 1]):
        rows = torch.cat([x[b][done[b]:done[b] + n[b]] for b in range(2)])
        pos = torch.cat([torch.arange(done[b], done[b] + n[b]) for b in range(2)]).to(cuda_device)
        seq = torch.tensor([0] * n[0] + [1] * n[1], device=cuda_device)
        slots = table.long()[seq, pos // page] * page + pos % page
        qkv = ks.rms_norm(rows, w) @ proj
        q, k, v = (t.view(sum(n), -1, dim) for t in qkv.split([hq * dim, hk * dim, hk * dim], 1))
        for b, part in enumerate(k.split(n)):
            all_k[b].append(part)
        q = ks.rotary_to_pages_4bit(q, k, v, pos, steps, kp, vp, slots)
        done = [done[b] + n[b] for b in range(2)]
        o = ks.paged_attention_4bit(q, kp, vp, table, torch.tensor(done, dtype=torch.int32, device=cuda_device),
                                    torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=cuda_device), max_q_len=max(n))
        y, r = o.flatten(1) @ back, rows.clone()
        ends.append((y.clone(), rows, y, r))
        ks.gated_add_rms_norm(y, r, w, post_weight=post, gate=gate, block_scale=0.5)
        for b in range(2):
            outs[b].append(o.split(n)[b])
            qs[b].append(q.split(n)[b])
    for b in range(2):
        n = lens[b]
        at = torch.arange(n, device=cuda_device)
        slots = table.long()[b, at // page] * page + at % page
        kk, vv = (t.double() for t in ks.pages_4bit_to_rows(kp, vp, slots, dtype=F32))
        codes, scales = stored(rotated(torch.cat(all_k[b]), at.cpu(), freqs(dim), False)[0], 1.0)
        assert torch.equal(bits(kp[1])[(slots // page).cpu(), (slots % page).cpu()], scales)
        same_codes(unpacked(kp[0][slots // page, slots % page]), codes, scales, "keys")
        check_rows(torch.cat(outs[b]), torch.cat(qs[b]), kk, vv, n, True, dim ** -0.5, f"sequence {b}")
    from test_gpu_gated_norm import check
    for y0, r0, y, r in ends:
        check(y, r, y0, r0, w, post, gate, 1.0, 0.5, 1e-6, "end of the block")
