"""A paged key/value cache held in 4 bits: written as positions are turned, read back, attended over.

    empty_pages_4bit(pages, page_size, kv_heads, head_dim, *, device) -> (codes, scales)
    rotary_to_pages_4bit(q, k, v, positions, steps, k_pages, v_pages, slots, *, k_scale, v_scale, ...) -> q_out
    pages_4bit_to_rows(k_pages, v_pages, slots, *, k_scale, v_scale, dtype, out) -> (k, v)
    paged_attention_4bit(q, k_pages, v_pages, page_table, kv_lens, q_starts, *, k_scale, v_scale, ...) -> out

A pool is a pair (codes, scales): uint8 [pages, page_size, kv_heads, head_dim / 2] and float8_e4m3fn
[pages, page_size, kv_heads, head_dim / 16], any stride order, 9/32 of the bytes of a 16-bit pool. Each
16 values of a head share a scale s; a value is held as a 4-bit float of the magnitudes 0, 0.5, 1, 1.5, 2,
3, 4, 6 times s times the pool's factor (k_scale, v_scale: one number per pool, the same in every call that
uses it). With the largest magnitude A of a group, s is A / (6 factor) rounded to e4m3 (2^-9 .. 448): a factor
of 1 serves values whose groups reach some hundredths to some thousands, another brings them there.
Factors, and the scale of rotated values, are FP32 numbers: what is held is defined by their FP32 values.

Tokens, checks, streams and errors are those of the 16-bit cache's operators.
"""
from __future__ import annotations

import torch

from . import _abi
from .decode import (_I32, _I64, _check_attention_rows, _first, _index, _inference, _rows, _turned, _turns)
from .ops import _BIG, _DTYPES, _grad, _launch

_U8, _F8 = torch.uint8, torch.float8_e4m3fn
_LEAST, _MOST = 2.0 ** -64, 2.0 ** 64


def empty_pages_4bit(pages: int, page_size: int, kv_heads: int, head_dim: int, *, device=None):
    """A pool of zeros, (codes, scales), laid out head by head within a page: the tokens of a page's head are
    contiguous, which reads a head's keys in the longest runs."""
    if head_dim < 16 or head_dim % 16:
        raise ValueError(f"head_dim must be a multiple of 16, got {head_dim}")
    codes = torch.zeros(pages, kv_heads, page_size, head_dim // 2, dtype=_U8, device=device)
    scales = torch.zeros(pages, kv_heads, page_size, head_dim // 16, dtype=_U8, device=device).view(_F8)
    return codes.transpose(1, 2), scales.transpose(1, 2)


def _pool(pool, name, device, kv_heads, dim):
    if not isinstance(pool, (tuple, list)) or len(pool) != 2:
        raise TypeError(f"{name} must be a pair (codes, scales); empty_pages_4bit makes one")
    for t, dtype, part, size in ((pool[0], _U8, "codes", dim // 2), (pool[1], _F8, "scales", dim // 16)):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(f"{name}'s {part} must be a tensor of {dtype}")
        if t.device != device:
            raise ValueError("tensors must be CUDA tensors on one device (there is no CPU path)")
        if t.dim() != 4 or t.shape[2] != kv_heads or t.shape[3] != size or t.shape[1] < 1:
            raise ValueError(f"{name}'s {part} must be [pages, page_size, {kv_heads}, {size}], got {tuple(t.shape)}")
        if t.stride(3) != 1 and size > 1:
            raise ValueError(f"{name}'s head rows must be contiguous")
    if pool[0].shape[:2] != pool[1].shape[:2]:
        raise ValueError(f"{name}'s codes and scales must have the same pages and page_size")


def _pools(k_pages, v_pages, k_scale, v_scale, device, kv_heads, dim):
    if dim < 16 or dim % 16:
        raise ValueError(f"head_dim must be a multiple of 16, got {dim}")
    _pool(k_pages, "k_pages", device, kv_heads, dim)
    _pool(v_pages, "v_pages", device, kv_heads, dim)
    if k_pages[0].shape != v_pages[0].shape:
        raise ValueError("k_pages and v_pages must have one shape")
    for v, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if not (isinstance(v, (int, float)) and _LEAST <= v <= _MOST):
            raise ValueError(f"{n} must be a number in 2^-64 .. 2^64")
    _inference(k_pages[1], v_pages[1])


def _fine(pool, shape, heads, dim, device):
    """A pool as the library's struct, but for the factor, if it is as it must be; all asked in one go."""
    codes, scales = pool
    c0, c1, c2, c3 = codes.stride()
    s0, s1, s2, s3 = scales.stride()
    return (codes.dtype is _U8 and scales.dtype is _F8 and codes.device == device and scales.device == device
            and codes.shape == (*shape, heads, dim // 2) and scales.shape == (*shape, heads, dim // 16)
            and c3 == s3 == 1 and not (scales.requires_grad and _grad())
            and (codes.data_ptr(), scales.data_ptr(), c0, c1, c2, s0, s1, s2))


def _packed(pool):
    """A pool as the library's struct, but for the factor."""
    codes, scales = pool
    return codes.data_ptr(), scales.data_ptr(), *codes.stride()[:3], *scales.stride()[:3]


def _check_to_pages(q, k, v, positions, steps, k_pages, v_pages, slots, k_scale, v_scale, scale, out):
    _first(k, "k")
    dev, dt = k.device, k.dtype
    _rows(k, "k", dt, dev)
    _rows(v, "v", dt, dev)
    tokens, hk, dim = k.shape
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    if hk == 0:
        raise ValueError("k and v must have heads")
    if q is not None:
        _rows(q, "q", dt, dev)
        if q.shape[0] != tokens or q.shape[2] != dim:
            raise ValueError("q must have k's tokens and head_dim")
    _pools(k_pages, v_pages, k_scale, v_scale, dev, hk, dim)
    _index(slots, "slots", _I64, dev, (tokens,))
    _inference(q, k, v, out)
    _turns(positions, steps, tokens, dim, dev, scale)
    if q is None:
        if out is not None:
            raise ValueError("out without q")
    elif out is not None:
        _rows(out, "out", dt, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")


def rotary_to_pages_4bit(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                         positions: torch.Tensor | None, steps: torch.Tensor | None, k_pages, v_pages,
                         slots: torch.Tensor, *, k_scale: float = 1.0, v_scale: float = 1.0,
                         interleaved: bool = False, scale: float = 1.0,
                         out: torch.Tensor | None = None) -> torch.Tensor | None:
    """rotary_to_pages() into 4-bit pools: token t's rotated key and its value are held in slot slots[t] (negative:
    nowhere), each rounded once, from the rotated value itself. Slots of one call must differ. steps None:
    nothing is rotated; q None: only the cache is written. Returns q_out (`out`, a new tensor, or None without q)."""
    try:
        dt, dev, code = k.dtype, k.device, _DTYPES[k.dtype]
        tokens, hk, dim = k.shape
        ks_, vs = k.stride(), v.stride()
        shape = k_pages[0].shape[:2]
        fine = (q is not None and out is None and k.is_cuda and hk > 0 and dim >= 16 and dim % 16 == 0
                and shape[1] > 0 and v.shape == k.shape and ks_[2] == vs[2] == 1 and q.dtype is dt and v.dtype is dt
                and q.device == dev and v.device == dev and len(k_pages) == 2 and len(v_pages) == 2
                and (kp := _fine(k_pages, shape, hk, dim, dev)) and (vp := _fine(v_pages, shape, hk, dim, dev))
                and slots.dtype is _I64 and slots.device == dev and slots.shape == (tokens,) and slots.is_contiguous()
                and -_BIG < scale < _BIG and k_scale.__class__ is v_scale.__class__ is float
                and _LEAST <= k_scale <= _MOST and _LEAST <= v_scale <= _MOST
                and _turned(positions, steps, tokens, dim, dev)
                and not (_grad() and (q.requires_grad or k.requires_grad or v.requires_grad)))
        if fine:
            qt, hq, qd = q.shape
            qs = q.stride()
            fine = qt == tokens and qd == dim and qs[2] == 1
    except (AttributeError, KeyError, ValueError, TypeError, IndexError):
        fine = False
    if not fine:
        _check_to_pages(q, k, v, positions, steps, k_pages, v_pages, slots, k_scale, v_scale, scale, out)
        shape, kp, vp = k_pages[0].shape[:2], _packed(k_pages), _packed(v_pages)
        hq, qs = (q.shape[1], q.stride()) if q is not None else (0, (0, 0))
    if q is not None and out is None:
        out = torch.empty((tokens, hq, dim), dtype=dt, device=dev)
    if tokens == 0:
        return out
    if q is None:
        q_p, o_p, qos = 0, 0, (0, 0)
    else:
        q_p, o_p, qos = q.data_ptr(), out.data_ptr(), out.stride()
    if steps is None:
        pos_p = steps_p = rot = 0
    else:
        pos_p, steps_p, rot = positions.data_ptr(), steps.data_ptr(), 2 * steps.shape[0]
    _launch(_abi.ks_rotary_to_pages_4bit, _abi.ROTARY_4BIT_ARGS.pack(
        o_p, q_p, 0, k.data_ptr(), v.data_ptr(), pos_p, steps_p, 0, 0, slots.data_ptr(), tokens, hq, hk, dim, rot,
        shape[0], shape[1], qos[0], qos[1], qs[0], qs[1], 0, 0, ks_[0], ks_[1], vs[0], vs[1],
        0, 0, 0, 0, 0, 0, scale, _abi.KS_ROTARY_INTERLEAVED if interleaved else 0, code, 0,
        *kp, k_scale, 0, *vp, v_scale, 0), dev)
    return out


def _check_to_rows(k_pages, v_pages, slots, k_scale, v_scale, dtype):
    if not isinstance(k_pages, (tuple, list)) or len(k_pages) != 2 or not isinstance(k_pages[0], torch.Tensor):
        raise TypeError("k_pages must be a pair (codes, scales); empty_pages_4bit makes one")
    codes = k_pages[0]
    if codes.device.type != "cuda":
        raise ValueError("tensors must be CUDA tensors on one device (there is no CPU path)")
    if codes.dim() != 4 or codes.shape[2] < 1:
        raise ValueError(f"k_pages' codes must be [pages, page_size, kv_heads, head_dim / 2], got {tuple(codes.shape)}")
    dev, hk, dim = codes.device, codes.shape[2], 2 * codes.shape[3]
    _pools(k_pages, v_pages, k_scale, v_scale, dev, hk, dim)
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; use float16, bfloat16 or float32")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise TypeError("slots must be a 1-D int64 tensor")
    tokens = slots.shape[0]
    _index(slots, "slots", _I64, dev, (tokens,))
    return codes, dev, hk, dim, tokens


def pages_4bit_to_rows(k_pages, v_pages, slots: torch.Tensor, *, k_scale: float = 1.0, v_scale: float = 1.0,
                       dtype: torch.dtype = torch.bfloat16, out: tuple | None = None) -> tuple:
    """What 4-bit pools hold in some slots: (k, v), each [tokens, kv_heads, head_dim] of `dtype`, rounded once (with
    a factor that is a power of two 16-bit types hold the values exactly, within their range). A negative slot gives
    zeros; slots may repeat. `out`: (k, v), tensors to write to that share nothing with each other, the pools or slots."""
    try:
        codes = k_pages[0]
        pages, page_size, hk, half = codes.shape
        dim, dev = 2 * half, codes.device
        tokens, = slots.shape
        fine = (codes.is_cuda and hk > 0 and page_size > 0 and half > 0 and half % 8 == 0 and len(k_pages) == 2
                and len(v_pages) == 2 and (kp := _fine(k_pages, (pages, page_size), hk, dim, dev))
                and (vp := _fine(v_pages, (pages, page_size), hk, dim, dev)) and dtype in _DTYPES and slots.dtype is _I64
                and slots.device == dev and slots.is_contiguous()
                and k_scale.__class__ is v_scale.__class__ is float and _LEAST <= k_scale <= _MOST
                and _LEAST <= v_scale <= _MOST)
    except (AttributeError, KeyError, ValueError, TypeError, IndexError):
        fine = False
    if not fine:
        codes, dev, hk, dim, tokens = _check_to_rows(k_pages, v_pages, slots, k_scale, v_scale, dtype)
        pages, page_size, kp, vp = *codes.shape[:2], _packed(k_pages), _packed(v_pages)
    if out is None:
        k = torch.empty((tokens, hk, dim), dtype=dtype, device=dev)
        v = torch.empty((tokens, hk, dim), dtype=dtype, device=dev)
        ks_ = vs = (hk * dim, dim)
    else:
        if not isinstance(out, (tuple, list)) or len(out) != 2:
            raise ValueError("out must be (k, v)")
        k, v = out
        for t, n in ((k, "k"), (v, "v")):
            _rows(t, n, dtype, dev)
            if t.shape != (tokens, hk, dim):
                raise ValueError(f"out's {n} must be [{tokens}, {hk}, {dim}], got {tuple(t.shape)}")
        _inference(k, v)
        ks_, vs = k.stride(), v.stride()
    if tokens == 0:
        return k, v
    _launch(_abi.ks_pages_4bit_to_rows, _abi.ROWS_4BIT_ARGS.pack(
        k.data_ptr(), v.data_ptr(), slots.data_ptr(), *kp, k_scale, 0, *vp, v_scale, 0,
        tokens, hk, dim, pages, page_size, ks_[0], ks_[1], vs[0], vs[1], _DTYPES[dtype], 0), dev)
    return k, v


def paged_attention_4bit_workspace(tokens: int, seqs: int, q_heads: int, kv_heads: int, head_dim: int,
                                   page_size: int, table_pages: int, dtype: torch.dtype, *,
                                   max_q_len: int | None = None, device=None) -> int:
    """Bytes of workspace that paged_attention_4bit() needs for these sizes on `device` (the current one). Fewer
    tokens, sequences or table pages with the rest unchanged never need more."""
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    args = _abi.ATTENTION_4BIT_ARGS.pack(
        *(0,) * 9, tokens, seqs, q_heads, kv_heads, head_dim, 0, page_size, table_pages, table_pages,
        max_q_len or 0, *(0,) * 10, 1.0, _abi.KS_ATTENTION_CAUSAL, _DTYPES[dtype], 0,
        *(0,) * 8, 1.0, 0, *(0,) * 8, 1.0, 0)
    with torch.cuda.device(device):
        st, need = _abi.ks_paged_attention_4bit_workspace(args)
    _abi.check(st)
    return need


def _check_attention(q, k_pages, v_pages, page_table, kv_lens, q_starts, k_scale, v_scale, scale, max_q_len, out, workspace):
    _first(q, "q")
    dev, dt = q.device, q.dtype
    if dt == torch.float32:
        raise TypeError("paged_attention_4bit takes float16 and bfloat16")
    _rows(q, "q", dt, dev)
    tokens, hq, dim = q.shape
    if not isinstance(k_pages, (tuple, list)) or len(k_pages) != 2 or getattr(k_pages[0], "ndim", 0) != 4:
        raise TypeError("k_pages must be a pair (codes, scales); empty_pages_4bit makes one")
    hk = k_pages[0].shape[2]
    _pools(k_pages, v_pages, k_scale, v_scale, dev, hk, dim)
    _check_attention_rows(q, hk, page_table, kv_lens, q_starts, scale, max_q_len, out, workspace)


# Workspace sizes by device and sizes: asking the library takes longer than looking them up.
_workspace_sizes: dict = {}


def _workspace_size(dev, *sizes):
    key = (dev.index, *sizes)
    need = _workspace_sizes.get(key)
    if need is None:
        if len(_workspace_sizes) >= 4096:
            _workspace_sizes.clear()
        need = _workspace_sizes[key] = paged_attention_4bit_workspace(*sizes[:-1], max_q_len=sizes[-1], device=dev)
    return need


def paged_attention_4bit(q: torch.Tensor, k_pages, v_pages, page_table: torch.Tensor, kv_lens: torch.Tensor,
                         q_starts: torch.Tensor, *, k_scale: float = 1.0, v_scale: float = 1.0,
                         scale: float | None = None, causal: bool = True, max_q_len: int | None = None,
                         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """paged_attention() over 4-bit pools: q, page_table, kv_lens, q_starts, scale, causal, max_q_len, out and
    workspace are as there (the workspace of at least paged_attention_4bit_workspace(...) bytes).

    Keys and values enter the products as codes times scales, without a rounding, and the factors in FP32 with the
    scores' scale and the output's. bfloat16 queries enter as float16 after a power of two has brought a row's largest
    magnitude to 1 .. 2 (values below 2^-14 of it lose at most 2^-25 of it), and probabilities as float16 for either
    type; scores, sums and outputs are FP32, one rounding at the end."""
    try:
        dt, dev, code = q.dtype, q.device, _DTYPES[q.dtype]
        tokens, hq, dim = q.shape
        pages, page_size, hk, _ = k_pages[0].shape
        seqs, width = page_table.shape
        qs = q.stride()
        table_stride, in_row = page_table.stride()
        fine = (out is None and workspace is None and code and q.is_cuda and hk > 0 and hq > 0 and hq % hk == 0
                and dim >= 16 and dim % 16 == 0 and page_size > 0 and qs[2] == in_row == 1
                and len(k_pages) == 2 and len(v_pages) == 2
                and (kp := _fine(k_pages, (pages, page_size), hk, dim, dev))
                and (vp := _fine(v_pages, (pages, page_size), hk, dim, dev)) and page_table.dtype is _I32
                and kv_lens.dtype is _I32 and q_starts.dtype is _I32 and page_table.device == dev
                and kv_lens.device == dev and q_starts.device == dev and kv_lens.shape == (seqs,)
                and q_starts.shape == (seqs + 1,) and kv_lens.is_contiguous() and q_starts.is_contiguous()
                and (scale is None or -_BIG < scale < _BIG) and k_scale.__class__ is v_scale.__class__ is float
                and _LEAST <= k_scale <= _MOST and _LEAST <= v_scale <= _MOST
                and (max_q_len is None or 0 <= max_q_len < 2 ** 31) and not (_grad() and q.requires_grad))
    except (AttributeError, KeyError, ValueError, TypeError, IndexError):
        fine = False
    if not fine or type(max_q_len) not in (int, type(None)):
        _check_attention(q, k_pages, v_pages, page_table, kv_lens, q_starts, k_scale, v_scale, scale, max_q_len, out,
                         workspace)
        kp, vp = _packed(k_pages), _packed(v_pages)
    if scale is None:
        scale = dim ** -0.5
    if out is None:
        out = torch.empty((tokens, hq, dim), dtype=dt, device=dev)
        os_ = (hq * dim, dim)
    else:
        os_ = out.stride()
    if tokens == 0 or seqs == 0:
        return out
    if workspace is None:
        ws_bytes = _workspace_size(dev, tokens, seqs, hq, hk, dim, page_size, width, dt, max_q_len)
        workspace = torch.empty(ws_bytes, dtype=_U8, device=dev)
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    _launch(_abi.ks_paged_attention_4bit, _abi.ATTENTION_4BIT_ARGS.pack(
        out.data_ptr(), q.data_ptr(), 0, 0, page_table.data_ptr(), kv_lens.data_ptr(), q_starts.data_ptr(),
        workspace.data_ptr(), ws_bytes, tokens, seqs, hq, hk, dim, pages, page_size, width, table_stride,
        max_q_len or 0, os_[0], os_[1], qs[0], qs[1], 0, 0, 0, 0, 0, 0, scale,
        _abi.KS_ATTENTION_CAUSAL if causal else 0, code, 0,
        *kp, k_scale, 0, *vp, v_scale, 0), dev)
    return out
