"""gated_add_rms_norm on the GPU against 64 bits.

Tolerances. e1 = (hidden / 512 + 64) 2^-24 bounds the relative error of an FP32 sum of squares of positive terms (chains of
at most hidden / 512 and a tree), half of it that of the norm's factor; both norms' factors, products and sums take at most
16 roundings more. So s is off by at most 2^-20 (|residual_scale r| + |branch|) + e1 |branch|, and the output by that times its
factor, plus the factor's own error: e1 and the root mean square of s's error relative to s's. Each result is rounded
once to its type, half a step relative to it (2^-25 for fp16 below its normal range).
"""
import math

import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from row_wise_rmsnorm_ks_gb300 import _abi
from test_gpu_decode_ops import close, no_faults, normal  # noqa: F401

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def reference(x, r, w, post, gate, residual_scale, block_scale, eps):
    hidden = x.shape[-1]
    e1 = (hidden / 512 + 64) * 2.0 ** -24
    x, r = x.double(), r.double()
    n = x
    if post is not None:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * post.double()
    branch = n * block_scale if gate is None else n * gate.double() * block_scale
    s = residual_scale * r + branch
    tol_s = 2.0 ** -20 * ((residual_scale * r).abs() + branch.abs()) + e1 * branch.abs()
    factor = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    y = s * factor * w.double()
    off = (tol_s * tol_s).mean(-1, keepdim=True).sqrt() * factor
    tol_y = y.abs() * (e1 + 2.0 ** -20 + 2 * off) + tol_s * factor * w.double().abs()
    return s, tol_s, y, tol_y


def check(x, r, x0, r0, w, post, gate, residual_scale, block_scale, eps, name):
    s, tol_s, y, tol_y = reference(x0, r0, w, post, gate, residual_scale, block_scale, eps)
    u, least = torch.finfo(x.dtype).eps / 2, 2.0 ** -25 if x.dtype == F16 else 0.0
    close(r, s, tol_s + u * (s.abs() + tol_s) + least, f"{name}: residual")
    close(x, y, tol_y + u * (y.abs() + tol_y) + least, f"{name}: x")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [None, "channel", "sequence", "token", "value", "row"])
@pytest.mark.parametrize("shape", [(1, 1, 8), (2, 3, 1), (3, 5, 1001), (4, 1, 1536), (2, 7, 4096), (1, 3, 14336), (3, 2, 40),
                                   (1, 2, 40000), (1, 2, 33001), (2, 100, 256)])
def test_matches_64_bits(cuda_device, dtype, post, gate, shape):
    x, r = normal(shape, dtype, 1, cuda_device, 3.0), normal(shape, dtype, 2, cuda_device, 2.0)
    w = (1 + 0.1 * normal(shape[-1:], F32, 3, cuda_device)).to(dtype)
    p = (0.5 + 0.1 * normal(shape[-1:], F32, 4, cuda_device)).to(dtype) if post else None
    sizes = {"channel": shape[-1:], "sequence": (shape[0], 1, shape[2]), "token": shape, "value": (1,), "row": (*shape[:2], 1)}
    g = normal(sizes[gate], dtype, 5, cuda_device, 0.5) if gate else None
    x0, r0 = x.clone(), r.clone()
    assert ks.gated_add_rms_norm(x, r, w, post_weight=p, gate=g, residual_scale=0.75, block_scale=1.5, eps=1e-5) is None
    check(x, r, x0, r0, w, p, g, 0.75, 1.5, 1e-5, str(shape))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows, hidden", [(400, 129), (400, 130), (400, 132), (50, 4095), (50, 4100), (200, 2001), (200, 2002), (50, 1),
                                          (160, 8196), (160, 16382), (20, 16383), (1, 16385), (160, 16390), (400, 1024)])
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
def test_rows_that_no_vector_fits(cuda_device, dtype, rows, hidden, offset):
    """Widths and addresses of every alignment, few rows and many; what lies beside the rows stays."""
    def rows_at(seed, factor):
        whole = torch.full((offset + rows * hidden + 8,), 7.0, dtype=dtype, device=cuda_device)
        part = whole[offset:offset + rows * hidden].view(rows, hidden)
        part.copy_(normal((rows, hidden), dtype, seed, cuda_device, factor))
        return whole, part
    (all_x, x), (all_r, r) = rows_at(1, 3.0), rows_at(2, 2.0)
    w = (1 + 0.1 * normal((hidden,), F32, 3, cuda_device)).to(dtype)
    p = (0.5 + 0.1 * normal((hidden,), F32, 4, cuda_device)).to(dtype)
    gate = normal((rows, hidden), dtype, 5, cuda_device)
    x0, r0 = x.clone(), r.clone()
    ks.gated_add_rms_norm(x, r, w, post_weight=p, gate=gate, residual_scale=0.75, block_scale=0.5)
    check(x, r, x0, r0, w, p, gate, 0.75, 0.5, 1e-6, f"{rows} of {hidden}")
    for whole in (all_x, all_r):
        assert bool((whole[:offset] == 7.0).all()) and bool((whole[offset + rows * hidden:] == 7.0).all())


@pytest.mark.parametrize("hidden", [4096, 4100, 1001])
def test_without_anything_is_the_fused_add(cuda_device, hidden):
    x, r = normal((37, hidden), BF16, 1, cuda_device), normal((37, hidden), BF16, 2, cuda_device)
    w = normal((hidden,), BF16, 3, cuda_device)
    x1, r1 = x.clone(), r.clone()
    ks.fused_add_rms_norm(x1, r1, w)
    ks.gated_add_rms_norm(x, r, w)
    assert torch.equal(r, r1)  # one FP32 sum, rounded once
    assert int((x.view(torch.int16).int() - x1.view(torch.int16).int()).abs().max()) <= 1


def test_unaligned_rows_and_guards(cuda_device):
    hidden, rows = 1024, 9
    for off in (0, 1, 4):
        bufs = [torch.full((rows * hidden + 64,), 9.0, dtype=F16, device=cuda_device) for _ in range(2)]
        x, r = (b[8 + off:8 + off + rows * hidden].view(rows, hidden) for b in bufs)
        x.copy_(normal((rows, hidden), F16, 1, cuda_device))
        r.copy_(normal((rows, hidden), F16, 2, cuda_device))
        w, x0, r0 = normal((hidden,), F16, 3, cuda_device), x.clone(), r.clone()
        g = normal((rows * hidden + 8,), F16, 4, cuda_device)[off:off + rows * hidden].view(rows, hidden)
        ks.gated_add_rms_norm(x, r, w, post_weight=w, gate=g)
        check(x, r, x0, r0, w, w, g, 1.0, 1.0, 1e-6, f"offset {off}")
        for b in bufs:
            assert bool((b[:8 + off] == 9.0).all()) and bool((b[8 + off + rows * hidden:] == 9.0).all())


def test_many_rows_and_non_finite_rows(cuda_device):
    rows, hidden = 5000, 512
    x, r = normal((rows, hidden), BF16, 1, cuda_device), normal((rows, hidden), BF16, 2, cuda_device)
    x[17, 3], r[4000, 5], x[123], r[123] = math.nan, math.inf, 0.0, 0.0
    x[200] = x[200] * 1e4
    w = normal((hidden,), BF16, 3, cuda_device)
    x0, r0 = x.clone(), r.clone()
    ks.gated_add_rms_norm(x, r, w, post_weight=w)
    good = torch.ones(rows, dtype=torch.bool, device=cuda_device)
    good[[17, 4000]] = False
    check(x[good], r[good], x0[good], r0[good], w, w, None, 1.0, 1.0, 1e-6, "rows")
    assert bool(x[17].isnan().all()) and not bool(x[123].any()) and not bool(r[123].any())


def test_graph_and_streams(cuda_device):
    x, r = normal((64, 2048), BF16, 1, cuda_device), normal((64, 2048), BF16, 2, cuda_device)
    w, g = normal((2048,), BF16, 3, cuda_device), normal((64, 1), BF16, 4, cuda_device)
    x0, r0 = x.clone(), r.clone()
    ks.gated_add_rms_norm(x, r, w, post_weight=w, gate=g)
    want = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ks.gated_add_rms_norm(x, r, w, post_weight=w, gate=g)
    for _ in range(2):
        x.copy_(x0)
        r.copy_(r0)
        graph.replay()
        assert torch.equal(x, want[0]) and torch.equal(r, want[1])
    side = torch.cuda.Stream()
    x.copy_(x0)
    r.copy_(r0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ks.gated_add_rms_norm(x, r, w, post_weight=w, gate=g)
    side.synchronize()
    assert torch.equal(x, want[0]) and torch.equal(r, want[1])


def test_refusals(cuda_device):
    x, r, w = torch.zeros(2, 3, 64, device=cuda_device), torch.zeros(2, 3, 64, device=cuda_device), torch.ones(64, device=cuda_device)
    for bad in (dict(gate=w.half()), dict(post_weight=w.half())):
        with pytest.raises(TypeError):
            ks.gated_add_rms_norm(x, r, w, **bad)
    for bad in (dict(gate=torch.ones(1, 3, 64, device=cuda_device)), dict(gate=torch.ones(3, 64, device=cuda_device)),
                dict(gate=torch.ones(32, device=cuda_device)), dict(gate=torch.ones(1, 2, 3, 64, device=cuda_device)),
                dict(post_weight=w[:32]), dict(eps=0.0), dict(residual_scale=math.inf), dict(block_scale=math.nan),
                dict(gate=torch.ones(64, 2, device=cuda_device)[:, 0])):
        with pytest.raises(ValueError):
            ks.gated_add_rms_norm(x, r, w, **bad)
    with pytest.raises(ValueError):
        ks.gated_add_rms_norm(x, r[:1], w)
    with pytest.raises(RuntimeError):
        ks.gated_add_rms_norm(x, r, w, gate=torch.ones(64, device=cuda_device, requires_grad=True))
    for bad in (lambda: ks.gated_add_rms_norm(x, x, w), lambda: ks.gated_add_rms_norm(x, r, x[0, 0]),
                lambda: ks.gated_add_rms_norm(x, r, w, gate=r), lambda: ks.gated_add_rms_norm(x, r, w, post_weight=r[1, 2])):
        with pytest.raises(_abi.KsError):
            bad()
    empty = torch.zeros(0, 64, device=cuda_device)
    ks.gated_add_rms_norm(empty, empty.clone(), w, gate=torch.ones(0, 1, device=cuda_device))
