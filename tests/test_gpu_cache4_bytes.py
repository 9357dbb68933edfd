"""The 4-bit cache's bytes: what is written, compared byte for byte (a zero's sign too), and what is read back, compared
with the one rounding of u * code to its type.
"""
import math
import struct

import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from row_wise_rmsnorm_ks_gb300 import _abi
from test_gpu_cache4 import F8, MAGNITUDES, bits, pools, stored, unpacked
from test_gpu_decode_ops import close, freqs, no_faults, normal, rotated  # noqa: F401

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def same_bytes(pool, slots, x, factor, name):
    """The pool's slots hold x (64 bits): codes with bit 3 set where x < 0, none where the scale is 0."""
    codes, scales = stored(x, factor)
    codes = torch.where((scales == 0).repeat_interleave(16, -1), 0, codes)
    page_size = pool[0].shape[1]
    at = tuple(i.cpu() for i in (slots // page_size, slots % page_size))
    got = bits(pool[1])[at]
    assert torch.equal(got, scales), f"{name}: {int((got != scales).sum())} of {scales.numel()} scales differ"
    got = unpacked(pool[0][tuple(i.to(pool[0].device) for i in at)])
    assert torch.equal(got, codes), f"{name}: {int((got != codes).sum())} of {codes.numel()} codes differ"


def view(tokens, heads, dim, dtype, seed, device, aligned):
    x = normal((tokens * heads * dim + 1,), dtype, seed, device)
    return (x[:-1] if aligned else x[1:]).view(tokens, heads, dim)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens, aligned", [(1, True), (37, True), (37, False), (1101, True), (1101, False)])
def test_inverse_turns_queries_and_keys_alike(cuda_device, monkeypatch, dtype, interleaved, tokens, aligned):
    """KS_ROTARY_INVERSE, a flag of the C call: both sides turn the other way."""
    hq, hk, dim, rot, factor = 3, 2, 64, 32, 0.375
    call = _abi.ks_rotary_to_pages_4bit
    at = struct.calcsize("=10Q23qf")

    def inverse(args, stream):
        flags, = struct.unpack_from("=i", args, at)
        return call(args[:at] + struct.pack("=i", flags | _abi.KS_ROTARY_INVERSE) + args[at + 4:], stream)

    monkeypatch.setattr(_abi, "ks_rotary_to_pages_4bit", inverse)
    q, k, v = (view(tokens, h, dim, dtype, s, cuda_device, aligned) for h, s in ((hq, 1), (hk, 2), (hk, 3)))
    kp, vp = (pools(-(-tokens // 16), 16, hk, dim, cuda_device, seed=s) for s in (4, 5))
    slots = torch.arange(tokens, device=cuda_device)
    pos = torch.randint(-(1 << 20), 1 << 40, (tokens,), generator=torch.Generator().manual_seed(6))
    out = ks.rotary_to_pages_4bit(q, k, v, pos.to(cuda_device), ks.rotary_steps(rot, device=cuda_device), kp, vp, slots,
                                  interleaved=interleaved, k_scale=factor, scale=1.25)
    f = freqs(rot)
    close(out, *rotated(q, pos, f, interleaved, scale=1.25, inverse=True), "q")
    same_bytes(kp, slots, rotated(k, pos, f, interleaved, scale=1.25, inverse=True)[0], factor, "k")
    same_bytes(vp, slots, v, 1.0, "v")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("turn", [None, "halves", "neighbours"])
@pytest.mark.parametrize("tokens, aligned", [(40, True), (40, False), (1100, True), (1100, False)])
def test_signs_of_stored_zeros(cuda_device, dtype, turn, tokens, aligned):
    """Zeros of either sign, and values that become zero: a code has the sign of its value, and only a value below 0 has one.
    Half of the tokens are turned by nothing, which leaves the values next to 0 where they are."""
    hk, dim = 2, 64
    k, v = (view(tokens, hk, dim, dtype, s, cuda_device, aligned) for s in (1, 2))
    least = 2.0 ** -24 if dtype == F16 else 2.0 ** -40
    for x in (k, v):
        x[..., 0::16], x[..., 1::16], x[..., 2::16], x[..., 3::16] = 0.0, -0.0, least, -least
        x[..., 4::16], x[..., 5::16] = 0.0, 0.0
        x[..., 6::16], x[..., 7::16] = x[..., 6::16] * 2.0 ** -9, x[..., 7::16] * 2.0 ** -9
        x[3, 0, 16:32] = x[3, 0, 16:32] * 0.0                # a group of zeros of both signs
        x[5, 1, :16] = -(x[5, 1, :16].abs() * 2.0 ** -13)    # a group whose scale is 0
    kp, vp = (pools(-(-tokens // 16), 16, hk, dim, cuda_device, seed=s) for s in (4, 5))
    slots = torch.arange(tokens, device=cuda_device)
    pos = torch.randint(0, 1 << 18, (tokens,), generator=torch.Generator().manual_seed(6))
    pos[::2] = 0
    steps = ks.rotary_steps(dim, device=cuda_device) if turn else None
    ks.rotary_to_pages_4bit(None, k, v, pos.to(cuda_device) if turn else None, steps, kp, vp, slots, interleaved=turn == "neighbours")
    same_bytes(kp, slots, rotated(k, pos, freqs(dim), turn == "neighbours")[0] if turn else k, 1.0, "k")
    same_bytes(vp, slots, v, 1.0, "v")


@pytest.mark.parametrize("dtype, size, scale", [(F32, 1e30, 2.0 ** 60), (BF16, 1e30, -2.0 ** 60), (F16, 1000.0, 2.0 ** 126),
                                                (F32, 3e38, 2.0), (F32, 1.0, 2.0 ** 126)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [9, 1030])
def test_turned_values_beyond_32_bits(cuda_device, dtype, size, scale, interleaved, tokens):
    """Products of a turn past FP32's largest number, whose difference has a sign all the same. NaN stays NaN."""
    hk, dim, factor = 2, 32, 2.0 ** 60
    k = normal((tokens, hk, dim), F32, 1, cuda_device).clamp(-1, 1).mul(size).to(dtype)
    k[2, 0, 3] = math.nan
    v = normal((tokens, hk, dim), dtype, 2, cuda_device)
    kp, vp = (pools(-(-tokens // 16), 16, hk, dim, cuda_device, seed=s) for s in (4, 5))
    slots = torch.arange(tokens, device=cuda_device)
    pos = torch.randint(1, 1 << 18, (tokens,), generator=torch.Generator().manual_seed(6))
    ks.rotary_to_pages_4bit(None, k, v, pos.to(cuda_device), ks.rotary_steps(dim, device=cuda_device), kp, vp, slots,
                            interleaved=interleaved, scale=scale, k_scale=factor)
    same_bytes(kp, slots, rotated(k, pos, freqs(dim), interleaved, scale=scale)[0], factor, "k")


def once(x, dtype):
    """x (64 bits) rounded once to dtype, to the nearest, ties to even, in 64 bits."""
    digits, least, most = {F16: (11, -14, 65504.0), BF16: (8, -126, torch.finfo(BF16).max), F32: (24, -126, torch.finfo(F32).max)}[dtype]
    exponent = torch.frexp(x).exponent.sub(1).clamp(min=least).double()
    step = torch.exp2(exponent - (digits - 1))
    y = torch.round(x / step) * step
    return torch.where(y.abs() > most, torch.copysign(torch.tensor(math.inf, dtype=torch.float64), x), y)


def test_once_rounds_to_even():
    x = torch.tensor([1 + 2.0 ** -11, 1 + 3 * 2.0 ** -11, 65519.0, 65520.0, 2.0 ** -25, 3 * 2.0 ** -25, 0.0], dtype=torch.float64)
    assert once(x, F16).tolist() == [1.0, 1 + 2.0 ** -9, 65504.0, math.inf, 0.0, 2.0 ** -23, 0.0]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("aligned", [True, False])
def test_rows_are_rounded_once(cuda_device, dtype, aligned):
    """Every scale with every code, under factors of few and of 24 bits. u is the FP32 product of scale and factor."""
    scale = torch.arange(127, dtype=torch.uint8)
    codes = torch.arange(16, dtype=torch.uint8)
    row = (codes[0::2] | codes[1::2] << 4).to(cuda_device)
    pool = ks.empty_pages_4bit(1, 127, 1, 16, device=cuda_device)
    pool[0].copy_(row.expand(1, 127, 1, 8))
    pool[1].view(torch.uint8).copy_(scale.view(1, 127, 1, 1))
    value = MAGNITUDES[codes.long() & 7] * torch.where(codes > 7, -1.0, 1.0)
    slots = torch.arange(127, device=cuda_device)
    g = torch.Generator().manual_seed(1)
    factors = torch.exp2(torch.rand(300, generator=g) * 20 - 14).tolist()
    for factor in [0.64040798, 1.0, 0.375, 0.3, 251 / 4096, 2.0 ** -64, 2.0 ** 64, 1 + 2.0 ** -23, 1 + 2.0 ** -22, *factors]:
        unit = (scale.view(F8).float() * torch.tensor(factor, dtype=F32)).double()
        want = once(unit[:, None] * value, dtype)
        whole = [torch.zeros(127 * 16 + 1, dtype=dtype, device=cuda_device) for _ in range(2)]
        out = tuple((t[:-1] if aligned else t[1:]).view(127, 1, 16) for t in whole)
        for rows in ks.pages_4bit_to_rows(pool, pool, slots, k_scale=factor, v_scale=factor, dtype=dtype, out=out):
            assert torch.equal(rows[:, 0].double().cpu(), want), f"factor {factor}"


def test_pools_that_require_grad_are_refused(cuda_device):
    """As those of 16 bits: a pool's scales are a floating-point tensor, which may be a leaf."""
    k = normal((3, 2, 64), BF16, 1, cuda_device)
    kp, vp = (ks.empty_pages_4bit(4, 8, 2, 64, device=cuda_device) for _ in range(2))
    leaf = kp[0], kp[1].detach().requires_grad_()
    slots = torch.arange(3, device=cuda_device)
    i32 = dict(dtype=torch.int32, device=cuda_device)
    table, lens, starts = torch.zeros(1, 1, **i32), torch.full((1,), 3, **i32), torch.tensor([0, 3], **i32)
    calls = [lambda a, b: ks.rotary_to_pages_4bit(k, k, k, slots, ks.rotary_steps(64, device=cuda_device), a, b, slots),
             lambda a, b: ks.rotary_to_pages_4bit(None, k, k, None, None, a, b, slots),
             lambda a, b: ks.pages_4bit_to_rows(a, b, slots),
             lambda a, b: ks.paged_attention_4bit(k, a, b, table, lens, starts),
             lambda a, b: ks.paged_attention_4bit(k, a, b, table, lens, starts, out=torch.empty_like(k))]
    for call in calls:
        for pair in ((leaf, vp), (vp, leaf)):
            with pytest.raises(RuntimeError, match="inference"):
                call(*pair)
            with torch.no_grad():
                call(*pair)
