"""Paths of the 4-bit cache's operators that a call's sizes, strides and layouts pick, each against 64 bits."""
import re

import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from row_wise_rmsnorm_ks_gb300 import _abi
from test_gpu_cache4 import attend, build, check_all, pools
from test_gpu_cache4_bytes import same_bytes, view
from test_gpu_decode_ops import close, freqs, no_faults, normal, rotated  # noqa: F401

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.mark.parametrize("dim, page_size", [(64, 16), (96, 64), (128, 128), (80, 16), (256, 16)])
@pytest.mark.parametrize("lens", [([300], [400]), ([1, 1], [200, 77])], ids=["prompt", "step"])
def test_attention_over_heads_that_are_one(cuda_device, dim, page_size, lens):
    """Keys, or values, or both that all heads share: an expanded pool, whose heads are 0 bytes apart."""
    st = build(*lens, 6, 3, dim, BF16, page_size, cuda_device, seed=dim)
    kp, vp = (tuple(t[:, :, :1].expand(-1, -1, 3, -1) for t in st[p]) for p in ("kp", "vp"))
    k, v = ([t[:, :1].expand(-1, 3, -1) for t in st[x]] for x in ("k", "v"))
    for change in (dict(vp=vp, v=v), dict(kp=kp, k=k), dict(kp=kp, k=k, vp=vp, v=v)):
        shared = {**st, **change}
        check_all(attend(shared, max_q_len=max(lens[0])), shared)


def needed(st, rows):
    """The workspace that a call of up to `rows` new tokens a sequence asks for: which kernel it takes."""
    with pytest.raises(_abi.KsError) as e:
        attend(st, max_q_len=rows, workspace=torch.zeros(16, dtype=torch.uint8, device=st["q"].device))
    return int(re.search(r"(\d+) are needed", str(e.value)).group(1))


@pytest.mark.parametrize("dim, page_size, order, rows, cores", [
    (128, 16, "heads_outer", 24, False), (128, 16, "heads_outer", 40, True), (64, 16, "heads_outer", 40, False),  # rings
    (96, 16, "heads_outer", 24, True), (112, 16, "heads_outer", 24, False), (128, 24, "heads_outer", 24, True),
    (96, 24, "heads_outer", 24, False), (96, 16, "unaligned", 24, False), (128, 16, "unaligned", 24, False),
    (96, 24, "heads_outer", 40, True), (128, 16, "unaligned", 40, True), (64, 24, "heads_outer", 24, True),
    (64, 16, "unaligned", 24, False), (32, 128, "heads_outer", 24, True), (48, 5, "slots_outer", 24, False),
    (48, 5, "slots_outer", 40, True),
    (160, 16, "heads_outer", 40, False),
])
def test_drafts_on_tensor_cores_where_that_pays(cuda_device, dim, page_size, order, rows, cores):
    """17 .. 48 rows: 16-row tiles or the tensor cores' kernel, by how either's codes come."""
    st = build([24, 20], [500, 300], 2, 2, dim, BF16, page_size, cuda_device, order=order)
    tiles = needed(st, 16)
    assert (needed(st, rows) > tiles) == cores
    check_all(attend(st, max_q_len=rows), st)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens, hq, hk, dim, rot", [
    (1101, 6, 8, 128, 128),     # 512 groups a CTA, two for each thread; the last CTA has one token
    (1027, 0, 12, 256, 256),    # no queries; 1536 groups a CTA
    (1026, 2, 2, 512, 512),     # two tokens a CTA, whose sines fill the table
    (1025, 1, 3, 96, 40),       # part of a head, which ends within a group
    (1024, 3, 1, 1024, 1024),   # one token a CTA
    (2, 0, 130, 1024, 64),      # more groups than 64 CTAs have threads
])
def test_write_rounds(cuda_device, dtype, aligned, interleaved, tokens, hq, hk, dim, rot):
    """Sizes at which a thread of the writing kernels takes more than one group."""
    q = view(tokens, hq, dim, dtype, 1, cuda_device, aligned) if hq else None
    k, v = (view(tokens, hk, dim, dtype, s, cuda_device, aligned) for s in (2, 3))
    page_size = 24
    pages = -(-tokens // page_size) + 1
    kp, vp = (pools(pages, page_size, hk, dim, cuda_device, "slots_outer", s) for s in (4, 5))
    g = torch.Generator().manual_seed(6)
    slots = torch.randperm(pages * page_size, generator=g)[:tokens]
    pos = torch.randint(0, 1 << 30, (tokens,), generator=g)
    out = ks.rotary_to_pages_4bit(q, k, v, pos.to(cuda_device), ks.rotary_steps(rot, device=cuda_device), kp, vp,
                                  slots.to(cuda_device), interleaved=interleaved, k_scale=0.3)
    f = freqs(rot)
    if hq:
        close(out, *rotated(q, pos, f, interleaved), "q")
    same_bytes(kp, slots, rotated(k, pos, f, interleaved)[0], 0.3, "k")
    same_bytes(vp, slots, v, 1.0, "v")
