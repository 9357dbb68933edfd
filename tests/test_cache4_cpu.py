"""Refusals of the 4-bit cache's operators and of gated_add_rms_norm on CPU: every call below fails its checks before
any CUDA call (addresses are never read)."""
import math

import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from row_wise_rmsnorm_ks_gb300 import _abi
from row_wise_rmsnorm_ks_gb300 import build as ks_build
from test_decode_ops_cpu import ATTENTION, FAKE, ROTARY

INVALID, DTYPE, OVERLAP = (_abi.KS_ERR_INVALID_ARGUMENT, _abi.KS_ERR_UNSUPPORTED_DTYPE, _abi.KS_ERR_OVERLAP)
POOL = ["codes", "scales", "c_p", "c_s", "c_h", "s_p", "s_s", "s_h", "factor", "reserved"]


@pytest.fixture(scope="module", autouse=True)
def lib():
    ks_build.build()
    return _abi.load()


def pool(at, page_size, heads, dim, **change):
    """A pool head by head within a page; changes are named k_codes or v_s_p, say."""
    a = dict(codes=at, scales=at + FAKE // 2, c_p=heads * page_size * dim // 2, c_s=dim // 2, c_h=page_size * dim // 2,
             s_p=heads * page_size * dim // 16, s_s=dim // 16, s_h=page_size * dim // 16, factor=1.0, reserved=0)
    a.update(change)
    return [a[n] for n in POOL]


def split(change):
    return ({n: v for n, v in change.items() if n[:3] not in ("K__", "V__")},
            {n[3:]: v for n, v in change.items() if n.startswith("K__")},
            {n[3:]: v for n, v in change.items() if n.startswith("V__")})


def rotary_args(**change):
    """4 tokens, 2 query and 1 key head of 32 values (fp32), pools of 4 pages of 8, all apart."""
    own, k, v = split(change)
    a = dict(q_out=FAKE, q=2 * FAKE, k_out=0, k=4 * FAKE, v=5 * FAKE, positions=6 * FAKE, steps=7 * FAKE, k_pages=0,
             v_pages=0, slots=10 * FAKE, tokens=4, q_heads=2, kv_heads=1, head_dim=32, rotary_dim=32, pages=4, page_size=8,
             qo_t=64, qo_h=32, q_t=64, q_h=32, ko_t=0, ko_h=0, k_t=32, k_h=32, v_t=32, v_h=32,
             kp_p=0, kp_s=0, kp_h=0, vp_p=0, vp_s=0, vp_h=0, scale=1.0, flags=0, dtype=_abi.KS_DTYPE_F32, reserved=0)
    a.update(own)
    return _abi.ROTARY_4BIT_ARGS.pack(*(a[n] for n in ROTARY), *pool(8 * FAKE, 8, 1, 32, **k), *pool(9 * FAKE, 8, 1, 32, **v))


def attention_args(**change):
    """3 tokens of 2 sequences, 4 query and 2 key/value heads of 64 (bf16), 8 pages of 16."""
    own, k, v = split(change)
    a = dict(out=FAKE, q=2 * FAKE, k_pages=0, v_pages=0, page_table=5 * FAKE, kv_lens=6 * FAKE, q_starts=7 * FAKE,
             workspace=10 * FAKE, workspace_bytes=1 << 30, tokens=3, seqs=2, q_heads=4, kv_heads=2, head_dim=64, pages=8,
             page_size=16, table_pages=4, table_stride=4, max_q_len=2, o_t=256, o_h=64, q_t=256, q_h=64, kp_p=0, kp_s=0,
             kp_h=0, vp_p=0, vp_s=0, vp_h=0, scale=0.125, flags=1, dtype=_abi.KS_DTYPE_BF16, reserved=0)
    a.update(own)
    return _abi.ATTENTION_4BIT_ARGS.pack(*(a[n] for n in ATTENTION), *pool(3 * FAKE, 16, 2, 64, **k), *pool(4 * FAKE, 16, 2, 64, **v))


def rows_args(**change):
    """4 tokens, 2 heads of 32 (fp32), pools of 4 pages of 8."""
    own, k, v = split(change)
    a = dict(k_out=FAKE, v_out=2 * FAKE, slots=3 * FAKE)
    b = dict(tokens=4, kv_heads=2, head_dim=32, pages=4, page_size=8, k_t=64, k_h=32, v_t=64, v_h=32,
             dtype=_abi.KS_DTYPE_F32, reserved=0)
    for d in (a, b):
        d.update({n: x for n, x in own.items() if n in d})
    return _abi.ROWS_4BIT_ARGS.pack(*a.values(), *pool(8 * FAKE, 8, 2, 32, **k), *pool(9 * FAKE, 8, 2, 32, **v), *b.values())


def norm_args(**change):
    a = dict(x=FAKE, residual=2 * FAKE, weight=3 * FAKE, post_weight=4 * FAKE, gate=5 * FAKE, rows=6, hidden=64,
             rows_per_gate=2, gate_row_stride=64, gate_column_stride=1, eps=1e-6, residual_scale=1.0, block_scale=1.0,
             dtype=_abi.KS_DTYPE_F32)
    a.update(change)
    return _abi.GATED_NORM_ARGS.pack(*a.values())


POOLS = [(dict(K__codes=0), INVALID), (dict(V__scales=0), INVALID), (dict(K__codes=8 * FAKE + 4), INVALID),
         (dict(V__c_s=-16), INVALID), (dict(K__s_p=1 << 61), INVALID), (dict(K__factor=0.0), INVALID),
         (dict(V__factor=-1.0), INVALID), (dict(K__factor=math.nan), INVALID), (dict(V__factor=1e20), INVALID),
         (dict(K__factor=1e-20), INVALID)]


@pytest.mark.parametrize("change, status", POOLS + [
    (dict(dtype=9), DTYPE), (dict(tokens=-1), INVALID), (dict(head_dim=24, rotary_dim=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(rotary_dim=34), INVALID), (dict(rotary_dim=3), INVALID), (dict(kv_heads=0), INVALID), (dict(page_size=0), INVALID),
    (dict(pages=-1), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(q=0), INVALID), (dict(slots=0), INVALID),
    (dict(positions=0), INVALID), (dict(slots=10 * FAKE + 4), INVALID), (dict(scale=math.inf), INVALID), (dict(flags=4), INVALID),
    (dict(K__c_s=12), INVALID), (dict(K__c_p=64), OVERLAP), (dict(V__s_s=1), OVERLAP), (dict(K__codes=9 * FAKE), OVERLAP),
    (dict(K__scales=9 * FAKE + 8), OVERLAP), (dict(K__scales=8 * FAKE + 8), OVERLAP), (dict(V__codes=4 * FAKE), OVERLAP),
    (dict(K__scales=5 * FAKE + 64), OVERLAP), (dict(q_out=8 * FAKE), OVERLAP), (dict(V__codes=10 * FAKE), OVERLAP),
    (dict(K__scales=6 * FAKE + 8), OVERLAP), (dict(V__codes=7 * FAKE), OVERLAP), (dict(q_out=2 * FAKE + 64), OVERLAP),
])
def test_rotary_to_pages_4bit_refuses(change, status):
    assert _abi.ks_rotary_to_pages_4bit(rotary_args(**change), None) == status
    assert _abi.ks_last_error()


@pytest.mark.parametrize("change, status", [c for c in POOLS if "K__codes" not in c[0] or c[0]["K__codes"] == 0] + [
    (dict(K__codes=3 * FAKE + 4), INVALID),
    (dict(dtype=_abi.KS_DTYPE_F32), DTYPE), (dict(dtype=7), DTYPE), (dict(tokens=-1), INVALID), (dict(seqs=-1), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=72), INVALID), (dict(head_dim=272), INVALID), (dict(q_heads=3), INVALID),
    (dict(kv_heads=0), INVALID), (dict(page_size=0), INVALID), (dict(table_pages=-1), INVALID), (dict(max_q_len=-1), INVALID),
    (dict(flags=2), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=3e38), INVALID), (dict(scale=1e30, K__factor=1e10), INVALID),
    (dict(out=0), INVALID), (dict(q=0), INVALID), (dict(page_table=0), INVALID), (dict(kv_lens=0), INVALID), (dict(q_starts=0), INVALID),
    (dict(workspace=0), INVALID), (dict(workspace=10 * FAKE + 8), INVALID), (dict(q=2 * FAKE + 2), INVALID), (dict(q_t=260), INVALID),
    (dict(o_h=56), OVERLAP), (dict(out=2 * FAKE), OVERLAP), (dict(out=3 * FAKE), OVERLAP), (dict(out=4 * FAKE + FAKE // 2), OVERLAP),
    (dict(out=5 * FAKE), OVERLAP),
])
def test_paged_attention_4bit_refuses(change, status):
    assert _abi.ks_paged_attention_4bit(attention_args(**change), None) == status
    assert _abi.ks_last_error()


@pytest.mark.parametrize("change, status", POOLS + [
    (dict(dtype=5), DTYPE), (dict(tokens=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=40), INVALID),
    (dict(head_dim=1040), INVALID), (dict(page_size=0), INVALID), (dict(k_out=0), INVALID), (dict(slots=0), INVALID),
    (dict(k_out=FAKE + 2), INVALID), (dict(slots=3 * FAKE + 4), INVALID), (dict(k_t=-1), INVALID), (dict(v_h=1 << 60), INVALID),
    (dict(k_t=32), OVERLAP), (dict(v_out=FAKE + 128), OVERLAP), (dict(k_out=8 * FAKE), OVERLAP), (dict(v_out=3 * FAKE), OVERLAP),
])
def test_pages_4bit_to_rows_refuses(change, status):
    assert _abi.ks_pages_4bit_to_rows(rows_args(**change), None) == status
    assert _abi.ks_last_error()


@pytest.mark.parametrize("change, status", [
    (dict(dtype=3), DTYPE), (dict(rows=-1), INVALID), (dict(hidden=0), INVALID), (dict(eps=0.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(residual_scale=math.inf), INVALID), (dict(block_scale=math.nan), INVALID), (dict(x=0), INVALID), (dict(residual=0), INVALID),
    (dict(weight=0), INVALID), (dict(x=FAKE + 2), INVALID), (dict(gate=5 * FAKE + 1), INVALID), (dict(rows_per_gate=0), INVALID),
    (dict(gate_row_stride=-1), INVALID), (dict(gate_column_stride=2), INVALID), (dict(gate_row_stride=1 << 61), INVALID),
    (dict(rows=1 << 40, hidden=1 << 40), INVALID), (dict(residual=FAKE + 256), OVERLAP), (dict(weight=FAKE), OVERLAP),
    (dict(post_weight=2 * FAKE + 64), OVERLAP), (dict(gate=FAKE + 1024), OVERLAP), (dict(gate=2 * FAKE - 256), OVERLAP),
])
def test_gated_add_rms_norm_refuses(change, status):
    assert _abi.ks_gated_add_rms_norm(norm_args(**change), None) == status
    assert _abi.ks_last_error()


def test_null_and_empty():
    for f in (_abi.ks_rotary_to_pages_4bit, _abi.ks_pages_4bit_to_rows, _abi.ks_paged_attention_4bit, _abi.ks_gated_add_rms_norm):
        assert f(None, None) == INVALID
    assert _abi.ks_paged_attention_4bit_workspace(None)[0] == INVALID
    assert _abi.ks_rotary_to_pages_4bit(rotary_args(tokens=0), None) == _abi.KS_SUCCESS
    assert _abi.ks_pages_4bit_to_rows(rows_args(tokens=0), None) == _abi.KS_SUCCESS
    assert _abi.ks_paged_attention_4bit(attention_args(tokens=0), None) == _abi.KS_SUCCESS
    assert _abi.ks_gated_add_rms_norm(norm_args(rows=0), None) == _abi.KS_SUCCESS


def test_pools_are_made_head_by_head_and_cpu_tensors_are_refused():
    codes, scales = ks.empty_pages_4bit(3, 16, 2, 64)
    assert codes.shape == (3, 16, 2, 32) and scales.shape == (3, 16, 2, 4) and scales.dtype == torch.float8_e4m3fn
    assert codes.transpose(1, 2).is_contiguous() and scales.transpose(1, 2).is_contiguous()
    pair = codes, scales
    k, slots = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int64)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        ks.rotary_to_pages_4bit(None, k, k, None, None, pair, pair, slots)
    with pytest.raises(ValueError):
        ks.pages_4bit_to_rows(pair, pair, slots)
    with pytest.raises(ValueError):
        ks.paged_attention_4bit(k.half(), pair, pair, torch.zeros(1, 1, **i32), torch.zeros(1, **i32), torch.zeros(2, **i32))
    with pytest.raises(ValueError):
        ks.gated_add_rms_norm(k, k.clone(), torch.ones(64))
