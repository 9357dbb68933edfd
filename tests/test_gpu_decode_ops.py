"""The decode operators on the GPU against plain 64-bit implementations: rotary positions, the
paged cache's writes, attention over it, and a run of them together.

Tolerances, per element:
  rotary     half a step of the output type relative to the value, plus the FP32 evaluation: sine and
             cosine within 2 ulp of 1 and an argument off by 2^-25, the scale's and two products'
             roundings: at most 8 * 2^-24 (|x| + |y|) |scale|; fp16 outputs below 2^-14 have steps
             of 2^-24, half of it is added.
  attention  half a step of the output type relative to the value; the probabilities' rounding, half
             a step relative to each, so that share of sum p |v| / l (fp16 probabilities below 2^-14:
             2^-25 each); the FP32 scores, off by (dim + 8) 2^-23 of sum |q k| |scale| at most
             (products are exact, dim sums that may truncate, the scale), which is the relative
             error of p, and of l again; 2 n 2^-23 for n summed keys in l and in the output, 2^-21
             for each exponential.
"""
import math

import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from row_wise_rmsnorm_ks_gb300 import _abi

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def faults(clear=True):
    st, flags = _abi.ks_device_faults(clear=clear)
    assert st == _abi.KS_SUCCESS
    return flags


@pytest.fixture(autouse=True)
def no_faults(cuda_device):
    assert faults() == 0
    yield
    assert faults() == 0


def normal(shape, dtype, seed, device, scale=1.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)


# ------------------------------------------------------------------------------------- rotary

def rotated(x, positions, freq, interleaved, scale=1.0, inverse=False):
    """(value, tolerance) of the rotation in 64 bits."""
    dt = x.dtype
    y = x.double()
    rot = 2 * freq.numel()
    # the angle's turns reduced exactly: position * round(f / 2 pi 2^64) mod 2^64, in integers
    step = torch.tensor([round(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in freq.tolist()], dtype=torch.float64)
    turns = [[((p * int(s)) % 2 ** 64) / 2.0 ** 64 for s in step.tolist()] for p in positions.tolist()]
    angle = (torch.tensor(turns, dtype=torch.float64) * (2 * math.pi)).to(x.device).reshape(len(turns), freq.numel())
    c, s = (torch.cos(angle) * scale)[:, None], (torch.sin(angle) * (-scale if inverse else scale))[:, None]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, w = a * c - b * s, b * c + a * s
    err = 8 * 2.0 ** -24 * (a.abs() + b.abs()) * abs(scale)
    out, tol = y.clone(), torch.zeros_like(y)
    if interleaved:
        out[..., 0:rot:2], out[..., 1:rot:2] = u, w
        tol[..., 0:rot:2], tol[..., 1:rot:2] = err, err
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = u, w
        tol[..., :rot // 2], tol[..., rot // 2:rot] = err, err
    tol[..., :rot] += torch.finfo(dt).eps / 2 * (out[..., :rot].abs() + tol[..., :rot])
    if dt == F16:
        tol[..., :rot] += 2.0 ** -25
    return out, tol


def close(got, want, tol, name):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), f"{name}: off by {float(d[bad].max())} where {float(tol[bad].max())} is allowed, {int(bad.sum())} of {bad.numel()}"


def freqs(rot, base=10000.0):
    return torch.tensor([base ** (-2 * j / rot) for j in range(rot // 2)], dtype=torch.float64)


def view3(tokens, heads, dim, dtype, seed, device, layout):
    """[tokens, heads, dim] in one of the layouts a program has it in."""
    if layout == "head_major":
        return normal((heads, tokens, dim), dtype, seed, device).transpose(0, 1)
    if layout == "unaligned":  # rows begin one element after a 16-byte boundary
        return normal((tokens, heads * dim + 1), dtype, seed, device)[:, 1:].view(tokens, heads, dim) \
            if tokens == 1 else normal((tokens * heads * dim + 1,), dtype, seed, device)[1:].view(tokens, heads, dim)
    return normal((tokens, heads, dim), dtype, seed, device)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim, rot, interleaved", [
    (128, 128, False), (128, 64, True), (64, 64, True), (80, 30, False), (80, 30, True), (256, 96, False),
    (96, 32, True), (5, 4, False), (2, 2, True), (1024, 1024, False), (1024, 1024, True), (8, 2, True),
])
@pytest.mark.parametrize("tokens, heads, kv_heads", [(1, 4, 1), (7, 5, 5), (311, 9, 3)])
def test_rotary_matches_64_bits(cuda_device, dtype, dim, rot, interleaved, tokens, heads, kv_heads):
    if dim == 1024 and tokens > 7:
        tokens = 40
    q = normal((tokens, heads, dim), dtype, 1, cuda_device)
    k = normal((tokens, kv_heads, dim), dtype, 2, cuda_device)
    f = freqs(rot)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=torch.Generator().manual_seed(3))
    qo, ko = ks.rotary(q, k, pos.to(cuda_device), ks.rotary_steps(rot, device=cuda_device), interleaved=interleaved)
    close(qo, *rotated(q, pos, f, interleaved), "q")
    close(ko, *rotated(k, pos, f, interleaved), "k")
    # what is not rotated is copied bit by bit
    assert torch.equal(qo[..., rot:], q[..., rot:]) and torch.equal(ko[..., rot:], k[..., rot:])


@pytest.mark.parametrize("layout", ["packed", "head_major", "unaligned"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rotary_layouts_and_in_place(cuda_device, layout, dtype):
    tokens, heads, dim = 19, 6, 64
    q = view3(tokens, heads, dim, dtype, 5, cuda_device, layout)
    k = view3(tokens, 2, dim, dtype, 6, cuda_device, layout)
    pos = torch.arange(tokens) * 1000 - 3000  # negative positions turn the other way
    steps = ks.rotary_steps(dim, device=cuda_device)
    f = freqs(dim)
    wants = [rotated(t, pos, f, False, scale=1.25) for t in (q, k)]
    got = ks.rotary(q, k, pos.to(cuda_device), steps, scale=1.25)
    again = ks.rotary(q, k, pos.to(cuda_device), steps, scale=1.25, out=(q, k))
    assert again[0] is q and again[1] is k
    for g, a, (w, tol) in zip(got, again, wants):
        close(g, w, tol, layout)
        assert torch.equal(g, a)


def test_rotary_parts_of_one_projection_in_place(cuda_device):
    tokens, hq, hk, dim = 33, 8, 2, 128
    qkv = normal((tokens, (hq + 2 * hk) * dim), BF16, 9, cuda_device)
    before = qkv.clone()
    q = qkv[:, :hq * dim].view(tokens, hq, dim)
    k = qkv[:, hq * dim:(hq + hk) * dim].view(tokens, hk, dim)
    pos = torch.arange(tokens)
    f = freqs(dim)
    (wq, tq), (wk, tk) = rotated(q, pos, f, False), rotated(k, pos, f, False)
    ks.rotary(q, k, pos.to(cuda_device), ks.rotary_steps(dim, device=cuda_device), out=(q, k))
    close(q, wq, tq, "q")
    close(k, wk, tk, "k")
    assert torch.equal(qkv[:, (hq + hk) * dim:], before[:, (hq + hk) * dim:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_turns_back_and_is_the_gradient(cuda_device, interleaved):
    tokens, heads, dim, rot = 9, 3, 32, 24
    q = normal((tokens, heads, dim), F32, 11, cuda_device)
    g = normal((tokens, heads, dim), F32, 12, cuda_device)
    pos = torch.randint(0, 1 << 30, (tokens,), generator=torch.Generator().manual_seed(1))
    steps = ks.rotary_steps(rot, device=cuda_device)
    p = pos.to(cuda_device)
    y, none = ks.rotary(q, None, p, steps, interleaved=interleaved)
    assert none is None
    back, _ = ks.rotary(y, None, p, steps, interleaved=interleaved, inverse=True)
    want, tol = rotated(y, pos, freqs(rot), interleaved, inverse=True)
    close(back, want, tol, "inverse")
    # two turns, each within its bound of the exact one; lengths are kept
    close(back, q.double(), 4 * tol.max() + torch.zeros_like(want), "round trip")
    # <rotary(q), g> = <q, gradient>: the turn is linear
    dq, _ = ks.rotary(g, None, p, steps, interleaved=interleaved, scale=0.5, inverse=True)
    y, _ = ks.rotary(q, None, p, steps, interleaved=interleaved, scale=0.5)
    rest = (y[..., rot:].double() * g[..., rot:].double()).sum(), (q[..., rot:].double() * dq[..., rot:].double()).sum()
    a = (y[..., :rot].double() * g[..., :rot].double()).sum()
    b = (q[..., :rot].double() * dq[..., :rot].double()).sum()
    n = tokens * heads * rot
    bound = 12 * 2.0 ** -24 * float(q.abs().max() * g.abs().max()) * n
    assert abs(float(a - b)) <= bound and abs(float(rest[0] - rest[1])) <= bound


def test_rotary_far_positions(cuda_device):
    """Positions whose FP32 angle would be meaningless, up to the ends of 64 bits."""
    pos = torch.tensor([2 ** 24 + 1, 2 ** 31 - 1, 2 ** 40 + 7, 2 ** 62 + 12345, -2 ** 63, 2 ** 63 - 1, 0, -1])
    q = normal((8, 2, 16), F32, 4, cuda_device)
    y, _ = ks.rotary(q, None, pos.to(cuda_device), ks.rotary_steps(16, device=cuda_device))
    close(y, *rotated(q, pos, freqs(16), False), "far")


def test_rotary_empty_and_refusals(cuda_device):
    steps = ks.rotary_steps(8, device=cuda_device)
    q = torch.zeros(0, 4, 8, device=cuda_device)
    i = torch.zeros(0, dtype=torch.int64, device=cuda_device)
    y, k = ks.rotary(q, q, i, steps)
    assert y.shape == k.shape == (0, 4, 8)
    q = torch.zeros(3, 4, 8, device=cuda_device)
    i = torch.zeros(3, dtype=torch.int64, device=cuda_device)
    for bad in (lambda: ks.rotary(q, q.half(), i, steps), lambda: ks.rotary(q, q, i.int(), steps),
                lambda: ks.rotary(q.double(), None, i, steps), lambda: ks.rotary(q, q, i, steps.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ks.rotary(q, q[:2], i, steps), lambda: ks.rotary(q, q, i[:2], steps),
                lambda: ks.rotary(q, q, i, ks.rotary_steps(10, device=cuda_device)),
                lambda: ks.rotary(q[0], None, i, steps), lambda: ks.rotary(q, None, i.cpu(), steps),
                lambda: ks.rotary(q.transpose(1, 2), None, i, steps),
                lambda: ks.rotary(q, None, i, steps, scale=math.inf), lambda: ks.rotary(q, None, i, steps, scale=1e39),
                lambda: ks.rotary(q, None, i, steps, out=(q, q)), lambda: ks.rotary(q, None, i, steps, out=q)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_abi.KsError):  # partial overlap
        big = torch.zeros(5, 4, 8, device=cuda_device)
        ks.rotary(big[:3], None, i, steps, out=(big[1:4], None))
    with pytest.raises(RuntimeError):
        ks.rotary(q.clone().requires_grad_(), None, i, steps)


# ------------------------------------------------------------------------------------- cache

def pool_of(pages, page_size, heads, dim, dtype, seed, device, order):
    if order == "heads_outer":
        return normal((pages, heads, page_size, dim), dtype, seed, device).transpose(1, 2)
    return normal((pages, page_size, heads, dim), dtype, seed, device)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("order", ["slots_outer", "heads_outer"])
@pytest.mark.parametrize("tokens, hq, hk, dim, rot, page_size, interleaved", [
    (1, 4, 1, 64, 64, 16, False), (45, 8, 2, 128, 64, 7, True), (200, 6, 6, 40, 20, 1, False),
    (64, 0, 3, 96, 0, 32, False), (5, 3, 1, 6, 4, 3, True),
])
def test_rotary_to_pages(cuda_device, dtype, order, tokens, hq, hk, dim, rot, page_size, interleaved):
    pages = -(-2 * tokens // page_size) + 2
    q = normal((tokens, hq, dim), dtype, 1, cuda_device) if hq else None
    k, v = normal((tokens, hk, dim), dtype, 2, cuda_device), normal((tokens, hk, dim), dtype, 3, cuda_device)
    kp = pool_of(pages, page_size, hk, dim, dtype, 4, cuda_device, order)
    vp = pool_of(pages, page_size, hk, dim, dtype, 5, cuda_device, order)
    kp0, vp0 = kp.clone(), vp.clone()
    g = torch.Generator().manual_seed(6)
    slots = torch.randperm(pages * page_size, generator=g)[:tokens]
    slots[tokens // 2::5] = -1 if tokens > 1 else slots[0]  # padding tokens
    pos = torch.randint(0, 1 << 18, (tokens,), generator=g)
    steps = ks.rotary_steps(rot, device=cuda_device) if rot else None
    out = ks.rotary_to_pages(q, k, v, pos.to(cuda_device) if rot else None, steps, kp, vp,
                             slots.to(cuda_device), interleaved=interleaved)
    f = freqs(rot) if rot else torch.zeros(0, dtype=torch.float64)
    if hq:
        close(out, *rotated(q, pos, f, interleaved), "q")
    else:
        assert out is None
    want, tol = rotated(k, pos, f, interleaved)
    live = [t for t in range(tokens) if slots[t] >= 0]
    at = [(int(slots[t]) // page_size, int(slots[t]) % page_size) for t in live]
    pg, pl = torch.tensor([a for a, _ in at], device=cuda_device), torch.tensor([b for _, b in at], device=cuda_device)
    close(kp[pg, pl], want[live], tol[live], "k")
    assert torch.equal(vp[pg, pl], v[live])
    untouched = torch.ones(pages, page_size, dtype=torch.bool, device=cuda_device)
    untouched[pg, pl] = False
    assert torch.equal(kp[untouched], kp0[untouched]) and torch.equal(vp[untouched], vp0[untouched])


def test_pages_beyond_the_pool_are_left_out_and_reported(cuda_device):
    k = normal((3, 2, 64), BF16, 1, cuda_device)
    kp, vp = pool_of(2, 8, 2, 64, BF16, 2, cuda_device, ""), pool_of(2, 8, 2, 64, BF16, 3, cuda_device, "")
    kp0, vp0 = kp.clone(), vp.clone()
    ks.rotary_to_pages(None, k, k, None, None, kp, vp, torch.tensor([16, 5, 1 << 40], device=cuda_device))
    assert faults() == _abi.KS_FAULT_BAD_INDEX
    kp0.view(16, 2, 64)[5], vp0.view(16, 2, 64)[5] = k[1], k[1]
    assert torch.equal(kp, kp0) and torch.equal(vp, vp0)


def test_keys_and_values_of_a_page_side_by_side(cuda_device):
    both = normal((4, 2, 8, 2, 32), F16, 1, cuda_device)  # [pages, key or value, page_size, heads, dim]
    kp, vp = both[:, 0], both[:, 1]
    k, v = normal((6, 2, 32), F16, 2, cuda_device), normal((6, 2, 32), F16, 3, cuda_device)
    slots = torch.tensor([31, 0, 8, 9, 17, 2], device=cuda_device)
    ks.rotary_to_pages(None, k, v, None, None, kp, vp, slots)
    assert torch.equal(kp[slots // 8, slots % 8], k) and torch.equal(vp[slots // 8, slots % 8], v)


def test_cache_beyond_31_bit_offsets(cuda_device):
    """A pool of more than 2^32 elements: slots, pages and attention address it in 64 bits."""
    page_size, hk, dim = 64, 8, 128
    pages = (1 << 32) // (page_size * hk * dim) + 40
    kp = torch.zeros(pages, page_size, hk, dim, dtype=BF16, device=cuda_device)
    vp = torch.zeros_like(kp)
    n = 100
    k, v = normal((n, hk, dim), BF16, 1, cuda_device), normal((n, hk, dim), BF16, 2, cuda_device)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=cuda_device)
    t = torch.arange(n, device=cuda_device)
    slots = table[0].long()[t // page_size] * page_size + t % page_size
    ks.rotary_to_pages(None, k, v, None, None, kp, vp, slots)
    assert torch.equal(kp[pages - 1], k[:64]) and torch.equal(vp[pages - 3, :36], v[64:])
    q = normal((n, hk, dim), BF16, 3, cuda_device)
    for few in (1, n):
        out = ks.paged_attention(q[-few:].contiguous(), kp, vp, table,
                                 torch.tensor([n], dtype=torch.int32, device=cuda_device),
                                 torch.tensor([0, few], dtype=torch.int32, device=cuda_device), max_q_len=few)
        check_rows(out, q[-few:], k, v, n, True, dim ** -0.5, "far pages")


# ------------------------------------------------------------------------------------- attention

def check_rows(out, q, k, v, keys, causal, scale, name):
    """One sequence's rows: q [n, Hq, D] against k, v [keys, Hk, D]."""
    n, hq, dim = q.shape
    group = hq // k.shape[1]
    u = torch.finfo(q.dtype).eps / 2
    if n == 0:
        return
    if keys == 0:
        assert not bool(out.any()), name
        return
    kk, vv = (t.double().repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))
    qq = q.double().transpose(0, 1)
    s = qq @ kk.transpose(1, 2) * scale
    mag = (qq.abs() @ kk.abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(scale)
    j, i = torch.arange(keys, device=q.device), torch.arange(n, device=q.device)
    sees = (j < keys - n + i[:, None] + 1) if causal else torch.ones(n, keys, dtype=torch.bool, device=q.device)
    s = s.masked_fill(~sees, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
    l = p.sum(-1, keepdim=True)
    inv = torch.where(l > 0, 1 / l, 0.0)
    want = (p @ vv) * inv
    share = (p @ vv.abs()) * inv
    fp32 = 2 * ((dim + 8) * 2.0 ** -23 * mag + 2.0 ** -21) + 4 * keys * 2.0 ** -23
    tol = share * (u + fp32)
    if q.dtype == F16:
        tol = tol + keys * 2.0 ** -25 * vv.abs().amax() * inv + 2.0 ** -25
    tol = tol + u * (want.abs() + tol)
    close(out.transpose(0, 1), want, tol, name)
    blind = ~sees.any(-1)
    assert not bool(out[blind].any()), f"{name}: rows that see nothing must be 0"


def build(q_lens, kv_lens, hq, hk, dim, dtype, page_size, device, seed=0, order="", spoil=True, extra_rows=0):
    """Sequences in a shuffled pool. Everything that no sequence owns holds NaN, and table entries
    past a sequence's pages are out of range."""
    pool = sum(-(-n // page_size) for n in kv_lens) + 2
    kp, vp = (pool_of(pool, page_size, hk, dim, dtype, seed + i, device, order) for i in (1, 2))
    if spoil:
        kp.fill_(math.nan)
        vp.fill_(math.nan)
    width = max(1, max(-(-n // page_size) for n in kv_lens))
    table = torch.full((len(kv_lens), width), -7, dtype=torch.int32)
    perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    ks_, vs_, at = [], [], 0
    for b, n in enumerate(kv_lens):
        k, v = normal((n, hk, dim), dtype, seed + 10 + b, device), normal((n, hk, dim), dtype, seed + 50 + b, device)
        need = -(-n // page_size)
        mine = perm[at:at + need]
        at += need
        table[b, :need] = torch.tensor(mine, dtype=torch.int32)
        for c, page in enumerate(mine):
            rows = min(page_size, n - c * page_size)
            kp[page, :rows], vp[page, :rows] = k[c * page_size:c * page_size + rows], v[c * page_size:c * page_size + rows]
        ks_.append(k)
        vs_.append(v)
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    q = normal((starts[-1] + extra_rows, hq, dim), dtype, seed + 3, device)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(q=q, kp=kp, vp=vp, table=table.to(device), kv=torch.tensor(kv_lens, **i32),
                starts=torch.tensor(starts, **i32), k=ks_, v=vs_, q_lens=q_lens, kv_lens=kv_lens, s=starts)


def check_all(out, st, causal=True, scale=None, name=""):
    scale = st["q"].shape[2] ** -0.5 if scale is None else scale
    for b, n in enumerate(st["q_lens"]):
        lo = st["s"][b]
        check_rows(out[lo:lo + n], st["q"][lo:lo + n], st["k"][b], st["v"][b], st["kv_lens"][b], causal, scale,
                   f"{name} sequence {b} ({n} over {st['kv_lens'][b]})")


def attend(st, **kw):
    return ks.paged_attention(st["q"], st["kp"], st["vp"], st["table"], st["kv"], st["starts"], **kw)


STEP = ([1] * 7, [1, 2, 63, 64, 65, 200, 1111])
CHUNK = ([5, 0, 130, 1, 33, 300], [5, 77, 130, 400, 65, 801])
BLIND = ([3, 4, 2, 40, 1], [0, 2, 2, 17, 0])       # fewer keys than new tokens, and none
PROMPT = ([257, 700], [257, 1500])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens", [STEP, CHUNK, BLIND, PROMPT], ids=["step", "chunk", "blind", "prompt"])
@pytest.mark.parametrize("hq, hk, dim, page_size", [
    (8, 1, 128, 16), (4, 4, 64, 32), (10, 2, 128, 128), (6, 2, 96, 7), (3, 3, 256, 16), (40, 2, 64, 8),
    (7, 1, 80, 64), (32, 8, 128, 1), (2, 1, 8, 256), (160, 1, 128, 48),
])
def test_paged_attention_matches_64_bits(cuda_device, dtype, lens, hq, hk, dim, page_size):
    st = build(*lens, hq, hk, dim, dtype, page_size, cuda_device, seed=hq + dim)
    out = attend(st)
    check_all(out, st)
    # the hint only picks the kernel
    for hint in (1, max(lens[0])):
        check_all(attend(st, max_q_len=hint), st, name=f"hint {hint}")


@pytest.mark.parametrize("lens", [STEP, CHUNK, BLIND], ids=["step", "chunk", "blind"])
@pytest.mark.parametrize("dim", [64, 128])
def test_paged_attention_without_causal_and_with_scale(cuda_device, lens, dim):
    st = build(*lens, 8, 2, dim, BF16, 16, cuda_device, seed=3)
    for scale in (0.3, -0.05, 0.0):
        check_all(attend(st, causal=False, scale=scale), st, causal=False, scale=scale)


@pytest.mark.parametrize("order", ["slots_outer", "heads_outer"])
@pytest.mark.parametrize("q_layout", ["packed", "head_major", "projection"])
def test_paged_attention_strides_and_rows_left_alone(cuda_device, order, q_layout):
    st = build([3, 20, 1], [50, 300, 129], 8, 4, 64, F16, 16, cuda_device, order=order, extra_rows=5)
    total = st["q"].shape[0]
    if q_layout == "head_major":
        st["q"] = st["q"].transpose(0, 1).contiguous().transpose(0, 1)
    elif q_layout == "projection":
        wide = torch.zeros(total, 16 * 64, dtype=F16, device=cuda_device)
        wide[:, 128:128 + 512] = st["q"].reshape(total, -1)
        st["q"] = wide[:, 128:128 + 512].view(total, 8, 64)
    out = torch.full((8, total, 64), 7.0, dtype=F16, device=cuda_device).transpose(0, 1)
    assert attend(st, out=out) is out
    check_all(out, st)
    assert bool((out[-5:] == 7.0).all()), "rows behind the last sequence are left as they were"


def test_paged_attention_large_scores(cuda_device):
    """Scores of several hundreds in rising order: the running maximum moves at every step."""
    st = build([1, 200], [777, 777], 4, 2, 128, BF16, 16, cuda_device, seed=8, spoil=False)
    ramp = torch.linspace(0.1, 6.0, 777, device=cuda_device)[:, None, None]
    base = normal((2, 128), BF16, 99, cuda_device).float()
    for b in range(2):
        st["k"][b] = (base[None] * ramp).to(BF16)
        for c in range(-(-777 // 16)):
            page, rows = int(st["table"][b, c]), min(16, 777 - 16 * c)
            st["kp"][page, :rows] = st["k"][b][16 * c:16 * c + rows]
    st["q"] = (base.repeat_interleave(2, 0)[None] * 2.0).to(BF16).expand(201, 4, 128).contiguous()
    check_all(attend(st, scale=0.5), st, scale=0.5)


def test_paged_attention_non_finite_keys_stay_in_their_sequence(cuda_device):
    st = build([1, 1, 1], [100, 100, 100], 4, 2, 64, BF16, 16, cuda_device, seed=2)
    st["kp"][int(st["table"][1, 2]), 3] = math.inf
    st["vp"][int(st["table"][1, 2]), 3] = math.nan
    out = attend(st)
    assert bool(out[1].isnan().all())
    for b in (0, 2):
        check_rows(out[b:b + 1], st["q"][b:b + 1], st["k"][b], st["v"][b], 100, True, 64 ** -0.5, "neighbour")


def test_chunks_beside_non_finite_neighbours(cuda_device):
    """Row tiles reach into the next sequence's queries, and steps past a sequence's keys: what is not
    finite there stays there."""
    st = build([40, 7, 90], [150, 100, 200], 8, 2, 128, BF16, 16, cuda_device, seed=12)
    st["q"][40:47] = math.nan
    st["kp"][int(st["table"][1, 2]), 3] = math.inf
    st["vp"][int(st["table"][1, 2]), 3] = math.nan
    out = attend(st, max_q_len=90)
    assert bool(out[40:47].isnan().all())
    for b in (0, 2):
        lo, n = st["s"][b], st["q_lens"][b]
        check_rows(out[lo:lo + n], st["q"][lo:lo + n], st["k"][b], st["v"][b], st["kv_lens"][b], True,
                   128 ** -0.5, "neighbour")


@pytest.mark.parametrize("q_lens, kv_lens, hq, hk, dim, page_size", [
    ([2000], [2000], 4, 1, 128, 128),          # many row tiles of one sequence, split among the CTAs
    ([40, 3], [700, 2900], 320, 1, 64, 32),    # a group of more heads than a row tile has rows
    ([1] * 40 + [600], [3000] * 40 + [900], 8, 4, 128, 64),
    ([33], [33], 1, 1, 96, 8), ([17, 18, 19], [128, 256, 384], 2, 2, 112, 384),
])
def test_paged_attention_shapes_of_work(cuda_device, q_lens, kv_lens, hq, hk, dim, page_size):
    st = build(q_lens, kv_lens, hq, hk, dim, BF16, page_size, cuda_device, seed=30)
    check_all(attend(st, max_q_len=max(q_lens)), st)


def test_broadcast_queries(cuda_device):
    """A head stride of 0: one row for every head of the group."""
    st = build([1, 30], [100, 200], 4, 2, 64, BF16, 16, cuda_device, seed=13)
    row = st["q"][:, :1].clone()
    st["q"] = row.expand(31, 4, 64)
    check_all(attend(st), st)
    pos = torch.arange(31)
    y, _ = ks.rotary(st["q"], None, pos.to(cuda_device), ks.rotary_steps(64, device=cuda_device))
    close(y, *rotated(st["q"], pos, freqs(64), False), "expanded")


def test_workspace_never_grows_with_less(cuda_device):
    def need(tokens, seqs, width, most):
        return ks.paged_attention_workspace(tokens, seqs, 8, 2, 128, 16, width, BF16, max_q_len=most, device=cuda_device)
    sizes = [need(t, s, w, m) for t, s, w, m in ((4096, 64, 512, 4096), (1000, 64, 512, 1000), (1000, 8, 512, 1000),
                                                 (1000, 8, 5, 1000), (20, 8, 5, 20), (8, 8, 5, 1), (1, 1, 1, 1))]
    assert sizes == sorted(sizes, reverse=True) and sizes[-1] > 0


def test_paged_attention_bad_indices_are_reported(cuda_device):
    """A page outside the pool reads as zeros; lengths and starts are brought into range."""
    st = build([1, 2], [40, 30], 2, 1, 64, BF16, 16, cuda_device, seed=4, spoil=False)
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
    st = build([1, 2], [48, 30], 2, 1, 64, BF16, 16, cuda_device, seed=4, spoil=False)
    st["kv"][0] = 10 ** 6  # more keys than the table has room for
    check_rows(attend(st)[:1], st["q"][:1], st["k"][0], st["v"][0], 48, True, 64 ** -0.5, "room")
    assert faults() == _abi.KS_FAULT_BAD_INDEX
    st["kv"][0], st["starts"][2] = -5, 100
    out = attend(st)
    assert faults() == _abi.KS_FAULT_BAD_INDEX and not bool(out[0].any())


def test_paged_attention_empty_calls(cuda_device):
    st = build([2, 1], [20, 30], 2, 1, 64, BF16, 16, cuda_device)
    assert attend({**st, "q": st["q"][:0], "starts": st["starts"] * 0}).shape == (0, 2, 64)
    out = torch.full_like(st["q"], 3.0)
    none = torch.zeros(0, dtype=torch.int32, device=cuda_device)
    ks.paged_attention(st["q"], st["kp"], st["vp"], st["table"][:0], none, torch.zeros(1, dtype=torch.int32, device=cuda_device), out=out)
    attend({**st, "starts": st["starts"] * 0}, out=out)
    assert bool((out == 3.0).all())
    # an empty pool with sequences that have no keys
    empty = st["kp"][:0]
    out = ks.paged_attention(st["q"], empty, empty, st["table"][:, :0], st["kv"] * 0, st["starts"])
    assert not bool(out.any())


def test_paged_attention_many_sequences(cuda_device):
    """More sequences than threads of a block, most of them without new tokens."""
    seqs = 1500
    g = torch.Generator().manual_seed(1)
    kv = torch.randint(0, 40, (seqs,), generator=g).tolist()
    ql = [(1 if i % 7 == 0 else 3 if i % 11 == 0 else 0) for i in range(seqs)]
    page = 8
    need = [-(-n // page) for n in kv]
    pool = sum(need)
    kp, vp = (normal((pool, page, 2, 64), BF16, i, cuda_device) for i in (1, 2))
    table = torch.zeros(seqs, 5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    starts = torch.tensor([0] + ql).cumsum(0).int()
    q = normal((int(starts[-1]), 4, 64), BF16, 3, cuda_device)
    for hint in (None, 3):
        out = ks.paged_attention(q, kp, vp, table.to(cuda_device), torch.tensor(kv, dtype=torch.int32, device=cuda_device),
                                 starts.to(cuda_device), max_q_len=hint)
        for b in range(0, seqs, 77):
            lo, hi = int(starts[b]), int(starts[b + 1])
            rows = slice(int(table[b, 0]) * page if need[b] else 0, None)
            k, v = kp.view(-1, 2, 64)[rows][:kv[b]], vp.view(-1, 2, 64)[rows][:kv[b]]
            check_rows(out[lo:hi], q[lo:hi], k, v, kv[b], True, 0.125, f"sequence {b}")


@pytest.mark.parametrize("lens", [STEP, PROMPT], ids=["step", "prompt"])
def test_paged_attention_is_reproducible_and_takes_a_workspace(cuda_device, lens):
    st = build(*lens, 8, 2, 128, BF16, 16, cuda_device, seed=5)
    most = max(lens[0])
    first = attend(st, max_q_len=most)
    need = ks.paged_attention_workspace(st["q"].shape[0], len(lens[0]), 8, 2, 128, 16, st["table"].shape[1], BF16,
                                        max_q_len=most, device=cuda_device)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=cuda_device)
    for _ in range(3):
        assert torch.equal(attend(st, workspace=ws, max_q_len=most), first)
    with pytest.raises(_abi.KsError):
        attend(st, workspace=ws[:need - 16], max_q_len=most)


def test_paged_attention_refusals(cuda_device):
    st = build([1, 2], [40, 30], 4, 2, 64, BF16, 16, cuda_device)
    for change, error in ((dict(kv=st["kv"].long()), TypeError), (dict(table=st["table"].long()), TypeError),
                          (dict(q=st["q"].float()), TypeError), (dict(q=st["q"].half()), TypeError),
                          (dict(q=st["q"][:, :3]), ValueError), (dict(q=st["q"][..., :32]), ValueError),
                          (dict(kv=st["kv"][:1]), ValueError), (dict(starts=st["starts"][:2]), ValueError),
                          (dict(kv=st["kv"].cpu()), ValueError), (dict(vp=st["vp"][:1]), ValueError),
                          (dict(table=st["table"][0]), ValueError)):
        with pytest.raises(error):
            attend({**st, **change})
    with pytest.raises(_abi.KsError):
        attend(st, out=st["q"])
    with pytest.raises(_abi.KsError):  # head rows that no 16-byte load reaches
        wide = torch.zeros(3, 4 * 64 + 4, dtype=BF16, device=cuda_device)
        attend({**st, "q": wide[:, 4:].view(3, 4, 64)})
    for bad in (dict(scale=math.nan), dict(scale=1e39), dict(scale=-math.inf), dict(max_q_len=-1), dict(max_q_len=2 ** 40)):
        with pytest.raises(ValueError):
            attend(st, **bad)
    with pytest.raises(_abi.KsError):  # the workspace over the output
        need = ks.paged_attention_workspace(3, 2, 4, 2, 64, 16, st["table"].shape[1], BF16, device=cuda_device)
        buf = torch.zeros(need + 4096, dtype=torch.uint8, device=cuda_device)
        attend(st, workspace=buf, out=buf[:3 * 4 * 64 * 2].view(BF16).view(3, 4, 64))
    for name in ("q", "kp", "vp"):  # and over what the call reads
        size = st[name].numel() * 2
        buf = torch.zeros(need + size, dtype=torch.uint8, device=cuda_device)
        inside = buf[need - 16:need - 16 + size].view(BF16).view(st[name].shape)
        with pytest.raises(_abi.KsError):
            attend({**st, name: inside}, workspace=buf[:need])
    with pytest.raises(RuntimeError):
        attend({**st, "q": st["q"].clone().requires_grad_()})


# ------------------------------------------------------------------------------------- together

def test_graph_replays_with_other_lengths(cuda_device):
    """One captured step, replayed with other contents of the lengths, the table and the queries;
    two graphs at once on two streams."""
    st = [build([1, 3, 1], [60, 300, 500], 8, 2, 128, BF16, 16, cuda_device, seed=20 * i) for i in (1, 2)]
    fresh = [build([2, 2, 1], [300, 60, 490], 8, 2, 128, BF16, 16, cuda_device, seed=20 * i) for i in (3, 4)]
    graphs, outs = [], []
    for s in st:
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            attend(s, max_q_len=3)
        torch.cuda.current_stream().wait_stream(warm)
        # room for the other lengths' pages
        s["kp"], s["vp"] = (torch.cat([p, torch.zeros(40, *p.shape[1:], dtype=BF16, device=cuda_device)]) for p in (s["kp"], s["vp"]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attend(s, max_q_len=3))
        graphs.append(g)
    for s, f in zip(st, fresh):
        for name in ("q", "table", "kv", "starts"):
            into = s[name][:, :f[name].shape[1]] if name == "table" else s[name]
            into.copy_(f[name])
        n = f["kp"].shape[0]
        s["kp"][:n], s["vp"][:n] = f["kp"], f["vp"]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for o, f in zip(outs, fresh):
        check_all(o, f)


def test_decoder_step_run(cuda_device):
    """A prompt in two chunks and three single tokens through norm, rotary positions into the cache
    and attention, for two sequences, against the whole sequence computed at once in 64 bits."""
    hidden, hq, hk, dim, page = 512, 8, 2, 64, 16
    g = torch.Generator().manual_seed(7)
    lens = [45, 70]
    x = [torch.randn(n, hidden, generator=g).to(BF16).to(cuda_device) for n in lens]
    w = (1 + 0.1 * torch.randn(hidden, generator=g)).to(BF16).to(cuda_device)
    proj = (torch.randn(hidden, (hq + 2 * hk) * dim, generator=g) / hidden ** 0.5).to(BF16).to(cuda_device)
    steps = ks.rotary_steps(dim, device=cuda_device)
    kp, vp = (torch.full((12, page, hk, dim), math.nan, dtype=BF16, device=cuda_device) for _ in range(2))
    table = torch.tensor([[4, 1, 9, 0, 0], [2, 3, 5, 7, 11]], dtype=torch.int32, device=cuda_device)
    done, outs, qs = [0, 0], [[], []], [[], []]
    for n in ([20, 41], [22, 26], [1, 1], [1, 1], [1, 1]):
        rows = torch.cat([x[b][done[b]:done[b] + n[b]] for b in range(2)])
        pos = torch.cat([torch.arange(done[b], done[b] + n[b]) for b in range(2)]).to(cuda_device)
        seq = torch.tensor([0] * n[0] + [1] * n[1], device=cuda_device)
        slots = table.long()[seq, pos // page] * page + pos % page
        qkv = ks.rms_norm(rows, w) @ proj
        q, k, v = (t.view(sum(n), -1, dim) for t in qkv.split([hq * dim, hk * dim, hk * dim], 1))
        q = ks.rotary_to_pages(q, k, v, pos, steps, kp, vp, slots)
        done = [done[b] + n[b] for b in range(2)]
        o = ks.paged_attention(q, kp, vp, table, torch.tensor(done, dtype=torch.int32, device=cuda_device),
                               torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=cuda_device), max_q_len=max(n))
        for b, part in enumerate(o.split(n)):
            outs[b].append(part)
        for b, part in enumerate(q.split(n)):
            qs[b].append(part)
    for b in range(2):
        n = lens[b]
        at = torch.arange(n, device=cuda_device)
        pg, pl = table.long()[b, at // page], at % page
        # the cache holds the projection's keys, rotated, and its values; the rows' attention is exact over it
        qkv = ks.rms_norm(x[b], w) @ proj
        _, k, v = (t.view(n, -1, dim) for t in qkv.split([hq * dim, hk * dim, hk * dim], 1))
        want, tol = rotated(k, at.cpu(), freqs(dim), False)
        # the projection of other row counts may add up in another order: one more rounding step
        close(kp[pg, pl], want, tol + 2 * torch.finfo(BF16).eps * (want.abs() + 1), "keys")
        check_rows(torch.cat(outs[b]), torch.cat(qs[b]), kp[pg, pl], vp[pg, pl], n, True, dim ** -0.5, f"sequence {b}")


def test_with_programmatic_dependent_launch(cuda_device):
    """A chain of steps with every launch scheduled early: each kernel waits for the one before."""
    st = build([1, 30, 2], [300, 200, 80], 8, 2, 128, BF16, 16, cuda_device, seed=9)
    pos = torch.arange(33, device=cuda_device)
    steps = ks.rotary_steps(128, device=cuda_device)

    def chain():
        x, got = st["q"], []
        for _ in range(6):
            x, _ = ks.rotary(x, None, pos, steps)
            x = attend({**st, "q": x}, max_q_len=30)
            got.append(x)
        return got
    want = chain()
    assert _abi.ks_set_launch_options(_abi.KS_LAUNCH_PDL) == _abi.KS_SUCCESS
    try:
        got = chain()
        torch.cuda.synchronize()
    finally:
        _abi.ks_set_launch_options(0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


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


def test_paged_attention_refuses_a_workspace_over_its_indices(cuda_device):
    st = build([1, 2], [40, 30], 2, 1, 64, BF16, 16, cuda_device, seed=14)
    need = ks.paged_attention_workspace(3, 2, 2, 1, 64, 16, st["table"].shape[1], BF16, device=cuda_device)
    for name in ("table", "kv", "starts"):
        size = st[name].numel() * 4
        for at in (0, need // 2 // 16 * 16, need - 16):
            buf = torch.zeros(need + size, dtype=torch.uint8, device=cuda_device)
            inside = buf[at:at + size].view(torch.int32).view(st[name].shape)
            inside.copy_(st[name])
            with pytest.raises(_abi.KsError):
                attend({**st, name: inside}, workspace=buf[:need])
        # behind the bytes that the call needs, in the same allocation, they are its own business
        buf = torch.zeros(need + size, dtype=torch.uint8, device=cuda_device)
        behind = buf[need:].view(torch.int32).view(st[name].shape)
        behind.copy_(st[name])
        check_all(attend({**st, name: behind}, workspace=buf), st, name=name)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq, hk, dim, n, keys", [
    (32, 1, 128, 40, 100), (32, 1, 64, 40, 1000), (8, 2, 128, 200, 1003), (4, 4, 64, 700, 730), (300, 1, 64, 9, 140),
])
def test_keys_behind_a_row_tile_may_hold_anything(cuda_device, dtype, hq, hk, dim, n, keys):
    """Later tokens' keys and values that are not finite reach no row tile before them, whichever kernel
    the hint picks."""
    st = build([n, 3], [keys, 50], hq, hk, dim, dtype, 16, cuda_device, seed=15)
    group = hq // hk
    for hint in (n, 1):
        # tokens of a row tile: 256 rows, or 16 where the hinted tokens' rows fit them
        tile = max(1, (16 if hint * group <= 16 else 256) // group)
        for m in {tile, (n - 1) // tile * tile}:
            if m >= n:
                continue
            bad = {**st, "kp": st["kp"].clone(), "vp": st["vp"].clone()}
            seen = keys - n + m  # keys that the first m tokens see
            for j in range(seen, keys):
                page = int(st["table"][0, j // 16])
                bad["kp"][page, j % 16], bad["vp"][page, j % 16] = (math.inf, math.nan) if j % 2 else (math.nan, -math.inf)
            out = attend(bad, max_q_len=hint)
            check_rows(out[:m], st["q"][:m], st["k"][0][:seen], st["v"][0][:seen], seen, True, dim ** -0.5,
                       f"hint {hint}, {m} of {n} tokens")
            check_rows(out[n:], st["q"][n:], st["k"][1], st["v"][1], 50, True, dim ** -0.5, "neighbour")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens, seqs, dim", [(1, 640, 64), (1, 320, 256), (20, 160, 64), (20, 160, 128)])
@pytest.mark.parametrize("at", [0, 5000, 15999])
@pytest.mark.parametrize("below", [10.0, 14.0, 16.0, 17.4, 20.0])
def test_many_small_probabilities_beside_a_large_one(cuda_device, dtype, tokens, seqs, dim, at, below):
    """One key draws most of the attention, the others' scores lie `below` under it: what they weigh
    together is kept. So many sequences (over the same pages) that a block has whole row tiles, all keys
    to one base. Tolerance as in check_rows, but for fp16 with probabilities that count 2^8 at the
    least for the largest: those below 2^-14 are off by 2^-25 at most, 2^-33 of the largest."""
    keys, heads, page = 16000, 8, 64
    kp = torch.zeros(keys // page, page, 1, dim, dtype=dtype, device=cuda_device)
    vp = torch.ones_like(kp)
    q = torch.zeros(seqs * tokens, heads, dim, dtype=dtype, device=cuda_device)
    q[..., 0] = 4.0
    kp[at // page, at % page, 0, 0] = below / 4
    vp[at // page, at % page] = 0.0
    table = torch.arange(keys // page, dtype=torch.int32, device=cuda_device).expand(seqs, -1)
    lens = torch.full((seqs,), keys, dtype=torch.int32, device=cuda_device)
    starts = torch.arange(0, (seqs + 1) * tokens, tokens, dtype=torch.int32, device=cuda_device)
    out = ks.paged_attention(q, kp, vp, table, lens, starts, scale=1.0, causal=False, max_q_len=tokens)
    score = 4.0 * float(kp[at // page, at % page, 0, 0])
    rest = (keys - 1) * math.exp(-score)
    want = rest / (1 + rest)
    u = torch.finfo(dtype).eps / 2
    tol = want * (u + 2 * ((dim + 8) * 2.0 ** -23 * score + 2.0 ** -21) + 4 * keys * 2.0 ** -23)
    if dtype == F16:
        tol += keys * 2.0 ** -33 / (1 + rest) + 2.0 ** -25
    tol += u * (want + tol)
    full = torch.full(out.shape, want, dtype=torch.float64, device=cuda_device)
    close(out, full, torch.full_like(full, tol), f"{below} below")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("negative", [False, True])
@pytest.mark.parametrize("powers", [5, 7, 7.9, 8.1, 9, 13.9, 14.1, 15, 15.9, 16.1, 17, 24, 60])
def test_scores_that_outgrow_the_first_keys(cuda_device, dtype, dim, negative, powers):
    """Scores rise by that many powers of two behind the first keys, and fall again: bases that have
    to be raised, just not, and probabilities at the ends of fp16."""
    n, keys = 20, 400
    st = build([n, 1], [keys, keys], 8, 2, dim, dtype, 16, cuda_device, seed=16, spoil=False)
    ramp = torch.cat([torch.zeros(130), torch.linspace(0, 1, 150), torch.linspace(1, 0.2, 120)]) * powers * math.log(2)
    st["q"][..., 0] = 4.0
    for b in range(2):
        k = st["k"][b]
        k[..., 0] = (ramp[:, None] / 4).to(cuda_device).to(dtype)
        k[..., 1:] *= 0.1
        if negative:
            k.neg_()
        for c in range(keys // 16):
            st["kp"][int(st["table"][b, c])] = k[16 * c:16 * c + 16]
    scale = -1.0 if negative else 1.0
    for hint in (n, 1):
        check_all(attend(st, scale=scale, max_q_len=hint), st, scale=scale, name=f"hint {hint}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [1, 23])
@pytest.mark.parametrize("order", ["parts_inside_heads", "heads_inside_parts", "head_major"])
def test_rotary_in_place_on_parts_that_alternate(cuda_device, dtype, tokens, order):
    """q, k and v interleaved in one projection, per head or per token: views that share no element."""
    heads, dim = 6, 64
    if order == "parts_inside_heads":
        both = normal((tokens, heads, 3, dim), dtype, 1, cuda_device)
        q, k, v = both.unbind(2)
    elif order == "heads_inside_parts":
        both = normal((tokens, 3, heads, dim), dtype, 1, cuda_device)
        q, k, v = both.unbind(1)
    else:
        both = normal((heads, tokens, 3, dim), dtype, 1, cuda_device)
        q, k, v = (t.transpose(0, 1) for t in both.unbind(2))
    pos = torch.arange(tokens) * 77 + 5
    steps = ks.rotary_steps(dim, device=cuda_device)
    (wq, tq), (wk, tk) = rotated(q, pos, freqs(dim), False), rotated(k, pos, freqs(dim), False)
    before = v.clone()
    ks.rotary(q, k, pos.to(cuda_device), steps, out=(q, k))
    close(q, wq, tq, "q")
    close(k, wk, tk, "k")
    assert torch.equal(v, before)


def write_and_read_pools(device, order, page_size, heads):
    """Pools of that memory order, written by rotary_to_pages and read by the attention over them."""
    pages, dim = 12, 64
    shape = {"page_parts": (pages, 2, page_size, heads, dim), "slot_parts": (pages, page_size, 2, heads, dim),
             "head_parts": (pages, page_size, heads, 2, dim), "dim_parts": (pages, page_size, heads, 2 * dim),
             "heads_outermost": (2, heads, pages, page_size, dim), "slots_outermost": (2, page_size, pages, heads, dim),
             "layers": (pages, 3, 2, heads, page_size, dim)}[order]
    both = normal(shape, F16, 1, device)
    kp, vp = {"page_parts": lambda: both.unbind(1), "slot_parts": lambda: both.unbind(2),
              "head_parts": lambda: both.unbind(3), "dim_parts": lambda: both.split(dim, 3),
              "heads_outermost": lambda: [t.permute(1, 2, 0, 3) for t in both],
              "slots_outermost": lambda: [t.transpose(0, 1) for t in both],
              "layers": lambda: [both[:, 1, i].transpose(1, 2) for i in range(2)]}[order]()
    assert kp.shape == vp.shape == (pages, page_size, heads, dim)
    before = both.clone()
    n = min(40, pages * page_size - 2)
    k, v, q = (normal((n, h, dim), F16, 2 + i, device) for i, h in enumerate((heads, heads, 2 * heads)))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(4)).int()[None].to(device)
    t = torch.arange(n, device=device)
    slots = table[0].long()[t // page_size] * page_size + t % page_size
    ks.rotary_to_pages(None, k, v, None, None, kp, vp, slots)
    assert torch.equal(kp[slots // page_size, slots % page_size], k)
    assert torch.equal(vp[slots // page_size, slots % page_size], v)
    i32 = dict(dtype=torch.int32, device=device)
    for hint in (1, n):
        out = ks.paged_attention(q, kp, vp, table, torch.tensor([n], **i32), torch.tensor([0, n], **i32), max_q_len=hint)
        check_rows(out, q, k, v, n, True, dim ** -0.5, f"{order} hint {hint}")
    kp[slots // page_size, slots % page_size] = 0
    vp[slots // page_size, slots % page_size] = 0
    after = both.clone()
    both.copy_(before)
    kp[slots // page_size, slots % page_size] = 0
    vp[slots // page_size, slots % page_size] = 0
    assert torch.equal(both, after), "nothing else was written"


@pytest.mark.parametrize("order", ["heads_outermost", "slots_outermost"])
@pytest.mark.parametrize("page_size, heads", [(16, 2), (1, 3), (5, 1)])
def test_pools_whose_pages_are_not_the_outermost_axis(cuda_device, order, page_size, heads):
    write_and_read_pools(cuda_device, order, page_size, heads)


@pytest.mark.parametrize("order", ["page_parts", "slot_parts", "head_parts", "dim_parts", "layers"])
@pytest.mark.parametrize("page_size, heads", [(16, 2), (1, 3), (5, 1)])
def test_pools_of_keys_and_values_that_alternate(cuda_device, order, page_size, heads):
    write_and_read_pools(cuda_device, order, page_size, heads)


def test_indices_between_an_outputs_rows(cuda_device):
    """Outputs that are columns of a wider buffer, with the call's indices in the columns beside: nothing
    is shared."""
    tokens, heads, dim = 4, 2, 64
    wide = torch.zeros(tokens, heads * dim + 64, dtype=BF16, device=cuda_device)
    out = wide[:, :heads * dim].view(tokens, heads, dim)
    beside = [wide[i, heads * dim:] for i in range(3)]  # 128 bytes each
    q = normal((tokens, heads, dim), BF16, 1, cuda_device)
    pos = beside[1].view(torch.int64)[:tokens]
    pos.copy_(torch.tensor([3, 9, 1000, 5]))
    steps = ks.rotary_steps(dim, device=cuda_device)
    ks.rotary(q, None, pos, steps, out=(out, None))
    close(out, *rotated(q, torch.tensor([3, 9, 1000, 5]), freqs(dim), False), "q")
    st = build([3, 1], [40, 30], heads, 1, dim, BF16, 16, cuda_device, seed=17)
    for name, where in zip(("table", "kv", "starts"), beside):
        inside = where.view(torch.int32)[:st[name].numel()].view(st[name].shape)
        inside.copy_(st[name])
        st[name] = inside
    check_all(attend(st, out=out), st)
