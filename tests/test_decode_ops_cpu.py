"""The decode operators' refusals and host-side parts on CPU: every call below fails its checks
before any CUDA call (addresses are never read), and rotary_steps is plain arithmetic."""
import math
import os
import subprocess
import sys

import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from row_wise_rmsnorm_ks_gb300 import _abi
from row_wise_rmsnorm_ks_gb300 import build as ks_build

FAKE = 1 << 20
INVALID, DTYPE, OVERLAP = (_abi.KS_ERR_INVALID_ARGUMENT, _abi.KS_ERR_UNSUPPORTED_DTYPE,
                           _abi.KS_ERR_OVERLAP)


@pytest.fixture(scope="module", autouse=True)
def lib():
    ks_build.build()
    return _abi.load()


ROTARY = ["q_out", "q", "k_out", "k", "v", "positions", "steps", "k_pages", "v_pages", "slots",
          "tokens", "q_heads", "kv_heads", "head_dim", "rotary_dim", "pages", "page_size",
          "qo_t", "qo_h", "q_t", "q_h", "ko_t", "ko_h", "k_t", "k_h", "v_t", "v_h",
          "kp_p", "kp_s", "kp_h", "vp_p", "vp_s", "vp_h", "scale", "flags", "dtype", "reserved"]
ATTENTION = ["out", "q", "k_pages", "v_pages", "page_table", "kv_lens", "q_starts", "workspace",
             "workspace_bytes", "tokens", "seqs", "q_heads", "kv_heads", "head_dim", "pages",
             "page_size", "table_pages", "table_stride", "max_q_len", "o_t", "o_h", "q_t", "q_h",
             "kp_p", "kp_s", "kp_h", "vp_p", "vp_s", "vp_h", "scale", "flags", "dtype", "reserved"]


def rotary_args(**change):
    """4 tokens, 2 query and 1 key head of 16 values (fp32), and a cache of 4 pages of 8, all apart."""
    a = dict(q_out=FAKE, q=2 * FAKE, k_out=3 * FAKE, k=4 * FAKE, v=5 * FAKE, positions=6 * FAKE,
             steps=7 * FAKE, k_pages=8 * FAKE, v_pages=9 * FAKE, slots=10 * FAKE, tokens=4, q_heads=2,
             kv_heads=1, head_dim=16, rotary_dim=16, pages=4, page_size=8, qo_t=32, qo_h=16, q_t=32,
             q_h=16, ko_t=16, ko_h=16, k_t=16, k_h=16, v_t=16, v_h=16, kp_p=128, kp_s=16, kp_h=16,
             vp_p=128, vp_s=16, vp_h=16, scale=1.0, flags=0, dtype=_abi.KS_DTYPE_F32, reserved=0)
    a.update(change)
    return _abi.ROTARY_ARGS.pack(*(a[n] for n in ROTARY))


def attention_args(**change):
    """3 tokens of 2 sequences, 4 query and 2 key/value heads of 64 (bf16), 8 pages of 16."""
    a = dict(out=FAKE, q=2 * FAKE, k_pages=3 * FAKE, v_pages=4 * FAKE, page_table=5 * FAKE,
             kv_lens=6 * FAKE, q_starts=7 * FAKE, workspace=8 * FAKE, workspace_bytes=1 << 30, tokens=3,
             seqs=2, q_heads=4, kv_heads=2, head_dim=64, pages=8, page_size=16, table_pages=4,
             table_stride=4, max_q_len=2, o_t=256, o_h=64, q_t=256, q_h=64, kp_p=2048, kp_s=128,
             kp_h=64, vp_p=2048, vp_s=128, vp_h=64, scale=0.125, flags=1, dtype=_abi.KS_DTYPE_BF16,
             reserved=0)
    a.update(change)
    return _abi.ATTENTION_ARGS.pack(*(a[n] for n in ATTENTION))


BOTH = [
    (dict(dtype=9), DTYPE), (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=1026, rotary_dim=0), INVALID),
    (dict(rotary_dim=15), INVALID), (dict(rotary_dim=18), INVALID), (dict(rotary_dim=-2), INVALID),
    (dict(q_heads=-1), INVALID), (dict(q_heads=0, kv_heads=0), INVALID), (dict(flags=4), INVALID),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(k=0), INVALID), (dict(positions=0), INVALID),
    (dict(steps=0), INVALID), (dict(positions=6 * FAKE + 4), INVALID), (dict(q=2 * FAKE + 2), INVALID),
    (dict(q_t=-32), INVALID), (dict(q_t=1 << 61), INVALID),
    (dict(qo_h=8), OVERLAP), (dict(qo_t=16), OVERLAP), (dict(q_out=2 * FAKE + 64), OVERLAP),
    (dict(q_out=4 * FAKE), OVERLAP),
]


@pytest.mark.parametrize("change, status", BOTH + [
    (dict(k_out=0), INVALID), (dict(k_out=FAKE), OVERLAP), (dict(k_out=2 * FAKE), OVERLAP),
    # in place, but with other strides than the input's
    (dict(q_out=2 * FAKE, qo_t=48), OVERLAP),
])
def test_rotary_refuses(change, status):
    assert _abi.ks_rotary(rotary_args(**change), None) == status
    assert _abi.ks_last_error()


@pytest.mark.parametrize("change, status", BOTH + [
    (dict(v=0), INVALID), (dict(slots=0), INVALID), (dict(slots=10 * FAKE + 4), INVALID),
    (dict(k_pages=0), INVALID), (dict(v_pages=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(page_size=0), INVALID), (dict(pages=-1), INVALID), (dict(kp_p=64), INVALID),
    (dict(vp_s=8), INVALID), (dict(kp_h=-16), INVALID), (dict(k_pages=9 * FAKE + 512), OVERLAP),
    (dict(k_pages=4 * FAKE), OVERLAP), (dict(v_pages=5 * FAKE + 64), OVERLAP),
    (dict(q_out=8 * FAKE), OVERLAP),
    # key and value pages interleaved, but not far enough apart
    (dict(v_pages=8 * FAKE + 256, kp_p=256, vp_p=256), OVERLAP),
])
def test_rotary_to_pages_refuses(change, status):
    assert _abi.ks_rotary_to_pages(rotary_args(**change), None) == status
    assert _abi.ks_last_error()


@pytest.mark.parametrize("change, status", [
    (dict(dtype=_abi.KS_DTYPE_F32), DTYPE), (dict(dtype=7), DTYPE), (dict(tokens=-1), INVALID),
    (dict(seqs=-1), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=60), INVALID),
    (dict(head_dim=264), INVALID), (dict(q_heads=3), INVALID), (dict(kv_heads=0), INVALID),
    (dict(q_heads=0), INVALID), (dict(page_size=0), INVALID), (dict(pages=-1), INVALID),
    (dict(table_pages=-1), INVALID), (dict(table_stride=-4), INVALID), (dict(max_q_len=-1), INVALID),
    (dict(flags=2), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=3e38), INVALID), (dict(out=0), INVALID),
    (dict(q=0), INVALID),
    (dict(k_pages=0), INVALID), (dict(v_pages=0), INVALID), (dict(page_table=0), INVALID),
    (dict(kv_lens=0), INVALID), (dict(q_starts=0), INVALID), (dict(kv_lens=6 * FAKE + 2), INVALID),
    (dict(workspace=0), INVALID), (dict(workspace=8 * FAKE + 8), INVALID), (dict(q=2 * FAKE + 2), INVALID),
    (dict(q_t=260), INVALID), (dict(kp_s=-128), INVALID), (dict(vp_p=1 << 61), INVALID),
    (dict(o_h=56), OVERLAP), (dict(o_t=128), OVERLAP), (dict(out=2 * FAKE), OVERLAP),
    (dict(out=3 * FAKE), OVERLAP), (dict(out=4 * FAKE + 1024), OVERLAP),
])
def test_paged_attention_refuses(change, status):
    assert _abi.ks_paged_attention(attention_args(**change), None) == status
    assert _abi.ks_last_error()


def test_null_structs_are_refused():
    assert _abi.ks_rotary(None, None) == INVALID
    assert _abi.ks_rotary_to_pages(None, None) == INVALID
    assert _abi.ks_paged_attention(None, None) == INVALID
    assert _abi.ks_paged_attention_workspace(None)[0] == INVALID
    assert _abi.ks_paged_attention_workspace(attention_args(q_heads=3))[0] == INVALID


def test_empty_calls_launch_nothing():
    assert _abi.ks_rotary(rotary_args(tokens=0), None) == _abi.KS_SUCCESS
    assert _abi.ks_rotary_to_pages(rotary_args(tokens=0), None) == _abi.KS_SUCCESS
    assert _abi.ks_paged_attention(attention_args(tokens=0), None) == _abi.KS_SUCCESS
    assert _abi.ks_paged_attention(attention_args(seqs=0), None) == _abi.KS_SUCCESS
    assert _abi.ks_paged_attention_workspace(attention_args(tokens=0)) == (_abi.KS_SUCCESS, 0)


def test_argument_structs_have_the_headers_size():
    # pointers and 64-bit fields, then a float and three 32-bit fields
    assert _abi.ROTARY_ARGS.size == 8 * 33 + 16
    assert _abi.ATTENTION_ARGS.size == 8 * 29 + 16


def turns_to_angle(steps):
    return [(s % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for s in steps.tolist()]


def test_rotary_steps_are_the_frequencies():
    got = turns_to_angle(ks.rotary_steps(16, 10000.0))
    for j, f in enumerate(got):
        # one rounding of 53 bits in the power and quotient, half a step of 2^-64 turns
        assert f == pytest.approx(10000.0 ** (-2 * j / 16), rel=2 ** -50, abs=2 ** -60)


def test_rotary_steps_scalings():
    plain = turns_to_angle(ks.rotary_steps(64, 500000.0))
    linear = turns_to_angle(ks.rotary_steps(64, 500000.0, scaling="linear", factor=4))
    raised = turns_to_angle(ks.rotary_steps(64, 500000.0, scaling="base", factor=4))
    bands = turns_to_angle(ks.rotary_steps(64, 500000.0, scaling="bands", factor=4,
                                           original_length=8192, low=1.0, high=4.0))
    for j, f in enumerate(plain):
        assert linear[j] == pytest.approx(f / 4, rel=1e-12)
        turns = 8192 * f / (2 * math.pi)
        if turns >= 4:
            assert bands[j] == pytest.approx(f, rel=1e-12)
        elif turns <= 1:
            assert bands[j] == pytest.approx(f / 4, rel=1e-12)
        else:
            assert f / 4 < bands[j] < f
    assert raised[0] == pytest.approx(plain[0], rel=1e-12)
    assert raised[-1] == pytest.approx(plain[-1] / 4, rel=1e-9)


@pytest.mark.parametrize("args, kw", [
    ((0,), {}), ((7,), {}), ((8, 0.0), {}), ((8, math.inf), {}), ((8,), dict(factor=0.0)),
    ((8,), dict(scaling="other")), ((8,), dict(scaling="bands", factor=2.0)),
    ((8,), dict(scaling="bands", factor=2.0, original_length=100, low=4.0, high=1.0)),
    ((2,), dict(scaling="base", factor=2.0)),
])
def test_rotary_steps_refuses(args, kw):
    with pytest.raises(ValueError):
        ks.rotary_steps(*args, **kw)


def test_cpu_tensors_are_refused():
    q = torch.zeros(2, 4, 8)
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        ks.rotary(q, q, i, ks.rotary_steps(8))
    pool = torch.zeros(2, 4, 4, 8)
    with pytest.raises(ValueError):
        ks.rotary_to_pages(q, q, q, i, ks.rotary_steps(8), pool, pool.clone(), i)
    with pytest.raises(ValueError):
        ks.paged_attention(q.half(), pool.half(), pool.half(), i.view(1, 2).int(), i[:1].int(), i.int())
    with pytest.raises(TypeError):
        ks.rotary(q.double(), None, i, ks.rotary_steps(8))


@pytest.mark.parametrize("stride", [1 << 60, (1 << 63) - 1])
def test_paged_attention_refuses_tables_beyond_64_bits(stride):
    assert _abi.ks_paged_attention(attention_args(table_stride=stride), None) == INVALID


@pytest.mark.parametrize("change", [
    dict(out=5 * FAKE), dict(out=6 * FAKE), dict(out=7 * FAKE),
    dict(out=7 * FAKE - 1520),                               # q_starts lies in out's last row
    dict(out=5 * FAKE + 4096, page_table=5 * FAKE, table_stride=1024),  # the table's second row
])
def test_paged_attention_refuses_outputs_over_its_indices(change):
    """The kernels read lengths and tables while they write: other blocks would see other lengths."""
    assert _abi.ks_paged_attention(attention_args(**change), None) == OVERLAP


@pytest.mark.parametrize("change", [
    dict(q_out=6 * FAKE), dict(q_out=7 * FAKE - 448), dict(k_out=6 * FAKE - 248), dict(k_out=7 * FAKE),
])
def test_rotary_refuses_outputs_over_its_indices(change):
    assert _abi.ks_rotary(rotary_args(**change), None) == OVERLAP


@pytest.mark.parametrize("change", [
    dict(q_out=6 * FAKE), dict(q_out=7 * FAKE), dict(q_out=10 * FAKE), dict(k_pages=6 * FAKE),
    dict(k_pages=10 * FAKE - 2040), dict(v_pages=7 * FAKE), dict(v_pages=10 * FAKE),
    dict(v_pages=10 * FAKE, rotary_dim=0),
])
def test_rotary_to_pages_refuses_outputs_over_its_indices(change):
    assert _abi.ks_rotary_to_pages(rotary_args(**change), None) == OVERLAP


def test_strided_tensors_are_told_apart(tmp_path):
    """The host's overlap checks against counting bytes (strided_check.cpp)."""
    here = os.path.dirname(os.path.abspath(__file__))
    exe = tmp_path / "strided_check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", f"-I{ks_build.CSRC}",
                    os.path.join(here, "strided_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("change", [
    # [tokens, heads, 2, dim] projections whose parts cross by one element, from either side
    dict(q_out=2 * FAKE + 4 * 15, qo_t=64, qo_h=32, q_t=64, q_h=32), dict(q_out=2 * FAKE - 4 * 15, qo_t=64, qo_h=32, q_t=64, q_h=32),
    dict(k_out=2 * FAKE + 4 * 17, ko_t=64, ko_h=32, q_t=64, q_h=32),
])
def test_rotary_refuses_alternating_parts_that_cross(change):
    assert _abi.ks_rotary(rotary_args(**change), None) == OVERLAP


@pytest.mark.parametrize("change", [
    # [pages, page_size, 2, heads, head_dim]: one element too near, and a whole place apart
    dict(v_pages=8 * FAKE + 4 * 15, kp_p=256, vp_p=256, kp_s=32, vp_s=32),
    dict(v_pages=8 * FAKE + 4 * 32, kp_p=256, vp_p=256, kp_s=32, vp_s=32),
    # keys and values of a page of other strides, half a page apart
    dict(v_pages=8 * FAKE + 4 * 64, kp_p=256, vp_p=256, kp_s=16, vp_s=24),
])
def test_rotary_to_pages_refuses_alternating_pools_that_cross(change):
    assert _abi.ks_rotary_to_pages(rotary_args(**change), None) == OVERLAP


def test_imports_on_a_torch_without_cuda():
    """torch built without CUDA lacks the stream function that the calls use; importing needs no GPU."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import row_wise_rmsnorm_ks_gb300 as ks\n"
            "assert ks.rotary_steps(8).shape == (4,)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("change", [
    dict(tokens=(1 << 31) - 1), dict(tokens=(1 << 31) - 1023), dict(seqs=(1 << 30) + 1), dict(seqs=(1 << 31) - 2),
])
def test_paged_attention_refuses_sizes_its_indices_do_not_hold(change):
    """Tokens and sequences are numbered in 32 bits, a row tile's and a thread's share past the last."""
    args = attention_args(out=1 << 50, workspace=1 << 51, **change)
    assert _abi.ks_paged_attention(args, None) == INVALID
    assert _abi.ks_paged_attention_workspace(args)[0] == INVALID


@pytest.mark.parametrize("rotary_dim, base, factor, length, low, high", [
    (64, 500000.0, 4.0, 8192, 1.0, 4.0), (128, 10000.0, 32.0, 4096, 1.0, 32.0), (30, 1e6, 2.5, 1000, 0.5, 2.0),
])
def test_rotary_steps_between_the_bands(rotary_dim, base, factor, length, low, high):
    """The blend's weight is linear in the turns over the original length, 0 at `low` and 1 at `high`."""
    got = turns_to_angle(ks.rotary_steps(rotary_dim, base, scaling="bands", factor=factor, original_length=length,
                                         low=low, high=high))
    blended = 0
    for j, f in enumerate(got):
        plain = base ** (-2 * j / rotary_dim)
        turns = length * plain / (2 * math.pi)
        if low < turns < high:
            blended += 1
            # f = plain (1 - w) / factor + plain w
            w = (f / plain - 1 / factor) / (1 - 1 / factor)
            assert w == pytest.approx((turns - low) / (high - low), abs=1e-9)
        else:
            assert f == pytest.approx(plain if turns >= high else plain / factor, rel=1e-12)
    assert blended >= 2


@pytest.mark.parametrize("rotary_dim, base, factor", [(64, 500000.0, 4.0), (128, 10000.0, 8.0), (6, 100.0, 1.5)])
def test_rotary_steps_of_a_raised_base(rotary_dim, base, factor):
    """Every frequency: divided by factor^(j / (rotary_dim / 2 - 1)), from 1 for the fastest to factor."""
    got = turns_to_angle(ks.rotary_steps(rotary_dim, base, scaling="base", factor=factor))
    for j, f in enumerate(got):
        assert f == pytest.approx(base ** (-2 * j / rotary_dim) / factor ** (j / (rotary_dim / 2 - 1)), rel=1e-12)
