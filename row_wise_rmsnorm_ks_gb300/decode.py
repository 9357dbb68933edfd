"""The operators between the norms of a decoder block: rotary positions, the paged key/value cache
and attention over it.

    rotary_steps(rotary_dim, base=10000.0, *, scaling=None, ...) -> steps
    rotary(q, k, positions, steps, *, interleaved, inverse, scale, out) -> (q_out, k_out)
    rotary_to_pages(q, k, v, positions, steps, k_pages, v_pages, slots, *, ...) -> q_out
    paged_attention(q, k_pages, v_pages, page_table, kv_lens, q_starts, *, scale, causal,
                    max_q_len, out, workspace) -> out

Tokens of all sequences are packed: q is [tokens, q_heads, head_dim], k and v are [tokens, kv_heads,
head_dim]. The cache is two pools of pages, [pages, page_size, kv_heads, head_dim] (any stride order,
so [pages, kv_heads, page_size, head_dim] pools come as their transpose(1, 2)). Head rows are
contiguous; the other strides are free, so q, k and v may be views of one fused projection, and the two
pools views of one tensor.

Checks are those of the other operators: CUDA tensors of one dtype on one device, inference only;
what they find raises TypeError, ValueError or RuntimeError, and the library's own checks raise
KsError. Every launch goes to the tensors' device and the current torch stream.
"""
from __future__ import annotations

import math

import torch

from . import _abi
from .ops import _DTYPES


def rotary_steps(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None,
                 factor: float = 1.0, original_length: int | None = None, low: float = 1.0,
                 high: float = 32.0, device=None) -> torch.Tensor:
    """The frequencies f_j = base^(-2j / rotary_dim) as fractions of a turn in 64-bit fixed point:
    int64 [rotary_dim / 2], made once and kept. Scaled for contexts `factor` times as long:

        "linear"  f_j / factor (positions pressed together)
        "base"    base raised by factor^(rotary_dim / (rotary_dim - 2)): the slowest frequency is
                  divided by factor, the fastest kept
        "bands"   by the turns a pair makes over original_length: at most `low`, f_j / factor; at
                  least `high`, f_j; between, the linear blend of both

    A factor on the rotated values that some models add (0.1 ln(factor) + 1, say) is `scale` of
    rotary() and rotary_to_pages()."""
    if not isinstance(rotary_dim, int) or rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    for v, n in ((base, "base"), (factor, "factor")):
        if not (isinstance(v, (int, float)) and math.isfinite(v) and v > 0):
            raise ValueError(f"{n} must be finite and positive")
    if scaling not in (None, "linear", "base", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}; use None, 'linear', 'base' or 'bands'")
    if scaling == "base":
        if rotary_dim == 2:
            raise ValueError("scaling 'base' needs rotary_dim of at least 4")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    if scaling == "bands":
        if not original_length or original_length <= 0:
            raise ValueError("scaling 'bands' needs original_length")
        if not (math.isfinite(low) and math.isfinite(high) and 0 < low < high):
            raise ValueError("bands need 0 < low < high")
    steps = []
    for j in range(rotary_dim // 2):
        f = float(base) ** (-2 * j / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            turns = original_length * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = f * keep + f / factor * (1 - keep)
        step = round(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64
        steps.append(step - 2 ** 64 if step >= 2 ** 63 else step)
    return torch.tensor(steps, dtype=torch.int64, device=device)


# A decode step is a few microseconds of GPU time, so the calls keep their own time on the host small:
# each first asks everything in one expression, and goes through the checks one by one, which name what
# is wrong, only if that fails; the stream comes as its handle; the device is only changed where it is
# not the current one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # torch without CUDA has none, nor CUDA tensors
_current_device = torch.cuda.current_device
_grad = torch.is_grad_enabled
_I32, _I64 = torch.int32, torch.int64
_BIG = 2.0 ** 127  # what a scale may be: finite in 32 bits, times log2(e) too


def _launch(call, args: bytes, device: torch.device) -> None:
    index = device.index
    if _current_device() == index:
        status = call(args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = call(args, _raw_stream(index))
    if status:
        _abi.check(status)


def _rows(t, name, dtype, device):
    """A [tokens, heads, head_dim] tensor whose head rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} dtype {t.dtype} differs from {dtype}")
    if t.device != device:
        raise ValueError("tensors must be CUDA tensors on one device (there is no CPU path)")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}'s head rows must be contiguous")


def _pool(t, name, dtype, device, kv_heads, dim):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a tensor of {dtype}")
    if t.device != device:
        raise ValueError("tensors must be CUDA tensors on one device (there is no CPU path)")
    if t.dim() != 4 or t.shape[2] != kv_heads or t.shape[3] != dim or t.shape[1] < 1:
        raise ValueError(f"{name} must be [pages, page_size, {kv_heads}, {dim}], got {tuple(t.shape)}")
    if t.stride(3) != 1 and dim > 1:
        raise ValueError(f"{name}'s head rows must be contiguous")


def _index(t, name, dtype, device, shape):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a tensor of {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on the other tensors' device")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {shape}, got {tuple(t.shape)}")


def _inference(*tensors):
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError("these kernels are inference-only: inputs must not require grad")


def _first(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a float16, bfloat16 or float32 tensor")
    if t.device.type != "cuda":
        raise ValueError("tensors must be CUDA tensors on one device (there is no CPU path)")


def _turns(positions, steps, tokens, dim, device, scale):
    """Checks the positions and steps; returns their addresses and the rotated dimension."""
    if not (isinstance(scale, (int, float)) and -_BIG < scale < _BIG):
        raise ValueError("scale must be finite (below 2^127)")
    if steps is None:
        return 0, 0, 0
    _index(positions, "positions", torch.int64, device, (tokens,))
    if not isinstance(steps, torch.Tensor) or steps.dtype != torch.int64 or steps.dim() != 1:
        raise TypeError("steps must be a 1-D int64 tensor (rotary_steps makes it)")
    if steps.device != device or not steps.is_contiguous():
        raise ValueError("steps must be contiguous, on the other tensors' device")
    if 2 * steps.shape[0] > dim:
        raise ValueError(f"steps rotate {2 * steps.shape[0]} values of a head of {dim}")
    return positions.data_ptr(), steps.data_ptr(), 2 * steps.shape[0]


def _check_rotary(q, k, positions, steps, scale, out):
    _first(q, "q")
    dev, dt = q.device, q.dtype
    _rows(q, "q", dt, dev)
    tokens, hq, dim = q.shape
    if k is not None:
        _rows(k, "k", dt, dev)
        if k.shape[0] != tokens or k.shape[2] != dim:
            raise ValueError("k must have q's tokens and head_dim")
    _inference(q, k)
    _turns(positions, steps, tokens, dim, dev, scale)
    if out is not None:
        if not isinstance(out, (tuple, list)) or len(out) != 2 or (out[1] is None) != (k is None):
            raise ValueError("out must be (q_out, k_out), k_out None where k is")
        for t, s, n in ((out[0], q, "q_out"), (out[1], k, "k_out")):
            if s is not None:
                _rows(t, n, dt, dev)
                if t.shape != s.shape:
                    raise ValueError(f"{n} must have its input's shape")
        _inference(*out)


def _turned(positions, steps, tokens, dim, dev):
    """Whether positions and steps are as they must be, in one go."""
    return (positions.dtype is _I64 and steps.dtype is _I64 and positions.shape == (tokens,)
            and steps.dim() == 1 and 2 * steps.shape[0] <= dim and positions.device == dev
            and steps.device == dev and positions.is_contiguous() and steps.is_contiguous())


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, steps: torch.Tensor, *,
           interleaved: bool = False, inverse: bool = False, scale: float = 1.0,
           out: tuple | None = None) -> tuple:
    """Rotates the first 2 * len(steps) values of every head of q and k (None: q alone) by each
    token's position; the rest is copied. Pairs are (j, j + half), or neighbours with `interleaved`.
    `inverse` turns back, which is also the gradient's turn. `out`: (q_out, k_out), each a tensor of
    its input's shape that is the input itself (in place) or shares nothing with the inputs.
    Returns (q_out, k_out)."""
    try:
        dt, dev, code = q.dtype, q.device, _DTYPES[q.dtype]
        tokens, hq, dim = q.shape
        qs = q.stride()
        fine = (out is None and k is not None and q.is_cuda and qs[2] == 1 and k.dtype is dt
                and k.device == dev and -_BIG < scale < _BIG
                and _turned(positions, steps, tokens, dim, dev)
                and not (_grad() and (q.requires_grad or k.requires_grad)))
        if fine:
            kt, hk, kd = k.shape
            ks_ = k.stride()
            fine = kt == tokens and kd == dim and ks_[2] == 1
    except (AttributeError, KeyError, ValueError, TypeError):
        fine = False
    if not fine:
        _check_rotary(q, k, positions, steps, scale, out)
        hk, ks_ = (k.shape[1], k.stride()) if k is not None else (0, (0, 0))
    if out is None:
        qo = torch.empty((tokens, hq, dim), dtype=dt, device=dev)
        ko = None if k is None else torch.empty((tokens, hk, dim), dtype=dt, device=dev)
    else:
        qo, ko = out
    if dim == 0 or tokens == 0 or hq + hk == 0:
        return qo, ko
    if steps is None:
        pos_p = steps_p = rot = 0
    else:
        pos_p, steps_p, rot = positions.data_ptr(), steps.data_ptr(), 2 * steps.shape[0]
    qos = qo.stride()
    if hk:
        kos, k_p, ko_p = ko.stride(), k.data_ptr(), ko.data_ptr()
    else:
        kos, k_p, ko_p = (0, 0), 0, 0
    _launch(_abi.ks_rotary, _abi.ROTARY_ARGS.pack(
        qo.data_ptr(), q.data_ptr(), ko_p, k_p, 0, pos_p, steps_p, 0, 0, 0,
        tokens, hq, hk, dim, rot, 0, 1, qos[0], qos[1], qs[0], qs[1], kos[0], kos[1], ks_[0], ks_[1],
        0, 0, 0, 0, 0, 0, 0, 0, scale,
        (_abi.KS_ROTARY_INTERLEAVED if interleaved else 0) | (_abi.KS_ROTARY_INVERSE if inverse else 0),
        code, 0), dev)
    return qo, ko


def _check_to_pages(q, k, v, positions, steps, k_pages, v_pages, slots, scale, out):
    _first(k, "k")
    dev, dt = k.device, k.dtype
    _rows(k, "k", dt, dev)
    _rows(v, "v", dt, dev)
    tokens, hk, dim = k.shape
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    if hk == 0 or dim == 0:
        raise ValueError("k and v must have heads and a head_dim")
    if q is not None:
        _rows(q, "q", dt, dev)
        if q.shape[0] != tokens or q.shape[2] != dim:
            raise ValueError("q must have k's tokens and head_dim")
    _pool(k_pages, "k_pages", dt, dev, hk, dim)
    _pool(v_pages, "v_pages", dt, dev, hk, dim)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    _index(slots, "slots", torch.int64, dev, (tokens,))
    _inference(q, k, v, k_pages, v_pages, out)
    _turns(positions, steps, tokens, dim, dev, scale)
    if q is None:
        if out is not None:
            raise ValueError("out without q")
    elif out is not None:
        _rows(out, "out", dt, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")


def rotary_to_pages(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                    positions: torch.Tensor | None, steps: torch.Tensor | None,
                    k_pages: torch.Tensor, v_pages: torch.Tensor, slots: torch.Tensor, *,
                    interleaved: bool = False, scale: float = 1.0,
                    out: torch.Tensor | None = None) -> torch.Tensor | None:
    """rotary() with the keys and values landing in their cache: token t's rotated key and its value
    go to slot slots[t] (page slots[t] // page_size, place slots[t] % page_size); a negative slot
    writes neither. Slots of one call must differ (where two are one, a mixture of both tokens may be
    left there). steps None: nothing is rotated; q None: only the cache is written. Returns q_out (`out`,
    a new tensor, or None without q)."""
    try:
        dt, dev, code = k.dtype, k.device, _DTYPES[k.dtype]
        tokens, hk, dim = k.shape
        ks_, vs, kp, vp = k.stride(), v.stride(), k_pages.stride(), v_pages.stride()
        pages, page_size, pool_heads, pool_dim = shape = k_pages.shape
        fine = (q is not None and out is None and k.is_cuda and hk > 0 and dim > 0 and page_size > 0
                and v.shape == k.shape and pool_heads == hk and pool_dim == dim
                and v_pages.shape == shape and ks_[2] == vs[2] == kp[3] == vp[3] == 1
                and q.dtype is dt and v.dtype is dt and k_pages.dtype is dt and v_pages.dtype is dt
                and q.device == dev and v.device == dev and k_pages.device == dev
                and v_pages.device == dev and slots.dtype is _I64 and slots.device == dev
                and slots.shape == (tokens,) and slots.is_contiguous() and -_BIG < scale < _BIG
                and _turned(positions, steps, tokens, dim, dev)
                and not (_grad() and (q.requires_grad or k.requires_grad or v.requires_grad
                                      or k_pages.requires_grad or v_pages.requires_grad)))
        if fine:
            qt, hq, qd = q.shape
            qs = q.stride()
            fine = qt == tokens and qd == dim and qs[2] == 1
    except (AttributeError, KeyError, ValueError, TypeError):
        fine = False
    if not fine:
        _check_to_pages(q, k, v, positions, steps, k_pages, v_pages, slots, scale, out)
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
    _launch(_abi.ks_rotary_to_pages, _abi.ROTARY_ARGS.pack(
        o_p, q_p, 0, k.data_ptr(), v.data_ptr(), pos_p, steps_p, k_pages.data_ptr(),
        v_pages.data_ptr(), slots.data_ptr(), tokens, hq, hk, dim, rot, pages, page_size,
        qos[0], qos[1], qs[0], qs[1], 0, 0, ks_[0], ks_[1], vs[0], vs[1],
        kp[0], kp[1], kp[2], vp[0], vp[1], vp[2], scale,
        _abi.KS_ROTARY_INTERLEAVED if interleaved else 0, code, 0), dev)
    return out


def paged_attention_workspace(tokens: int, seqs: int, q_heads: int, kv_heads: int, head_dim: int,
                              page_size: int, table_pages: int, dtype: torch.dtype, *,
                              max_q_len: int | None = None, device=None) -> int:
    """Bytes of workspace that paged_attention() needs for these sizes on `device` (the current
    one): tokens rows of q, a page table of [seqs, table_pages]. Fewer tokens, sequences or table
    pages with the rest unchanged never need more."""
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    args = _abi.ATTENTION_ARGS.pack(
        *(0,) * 9, tokens, seqs, q_heads, kv_heads, head_dim, 0, page_size, table_pages, table_pages,
        max_q_len or 0, *(0,) * 10, 1.0, _abi.KS_ATTENTION_CAUSAL, _DTYPES[dtype], 0)
    with torch.cuda.device(device):
        st, need = _abi.ks_paged_attention_workspace(args)
    _abi.check(st)
    return need


def _check_attention(q, k_pages, v_pages, page_table, kv_lens, q_starts, scale, max_q_len, out,
                     workspace):
    _first(q, "q")
    dev, dt = q.device, q.dtype
    if dt == torch.float32:
        raise TypeError("paged_attention takes float16 and bfloat16")
    _rows(q, "q", dt, dev)
    tokens, hq, dim = q.shape
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be [pages, page_size, kv_heads, head_dim]")
    hk = k_pages.shape[2]
    _pool(k_pages, "k_pages", dt, dev, hk, dim)
    _pool(v_pages, "v_pages", dt, dev, hk, dim)
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    if hk == 0 or hq == 0 or hq % hk:
        raise ValueError(f"q's {hq} heads must be a multiple of the cache's {hk}")
    if not isinstance(page_table, torch.Tensor) or page_table.dtype != torch.int32:
        raise TypeError("page_table must be a tensor of torch.int32")
    if page_table.device != dev or page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be [seqs, pages], its rows contiguous, on q's device")
    seqs = page_table.shape[0]
    _index(kv_lens, "kv_lens", torch.int32, dev, (seqs,))
    _index(q_starts, "q_starts", torch.int32, dev, (seqs + 1,))
    _inference(q, k_pages, v_pages, out)
    if scale is not None and not (isinstance(scale, (int, float)) and -_BIG < scale < _BIG):
        raise ValueError("scale must be finite (below 2^127)")
    if max_q_len is not None and not (isinstance(max_q_len, int) and 0 <= max_q_len < 2 ** 31):
        raise ValueError("max_q_len must be an int in 0 .. 2^31 - 1")
    if out is not None:
        _rows(out, "out", dt, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is not None and (not isinstance(workspace, torch.Tensor) or workspace.device != dev
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor on q's device")


# Workspace sizes by device and sizes: asking the library takes longer than looking them up.
_workspace_sizes: dict = {}


def _workspace_size(dev, tokens, seqs, hq, hk, dim, page_size, table_pages, dtype, max_q_len):
    key = (dev.index, tokens, seqs, hq, hk, dim, page_size, table_pages, dtype, max_q_len)
    need = _workspace_sizes.get(key)
    if need is None:
        if len(_workspace_sizes) >= 4096:
            _workspace_sizes.clear()
        need = _workspace_sizes[key] = paged_attention_workspace(
            tokens, seqs, hq, hk, dim, page_size, table_pages, dtype, max_q_len=max_q_len, device=dev)
    return need


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    page_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor, *,
                    scale: float | None = None, causal: bool = True, max_q_len: int | None = None,
                    out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of new tokens over their sequences' pages (float16 or bfloat16).

    q [tokens, q_heads, head_dim] holds the new tokens of all sequences, sequence b's being
    q_starts[b] .. q_starts[b + 1] - 1; its keys and values, the new tokens' included, are the first
    kv_lens[b] places of the pages in page_table[b]. page_table [seqs, n], kv_lens [seqs] and
    q_starts [seqs + 1] are int32. Causal: the i-th of n new tokens sees kv_lens[b] - n + i + 1 keys;
    a row that sees none comes out 0. scale: 1 / sqrt(head_dim) unless given.

    Scores, sums and outputs are FP32; the probabilities are rounded to q's type for the product with the
    values (half a step relative to each; in float16 those below 2^-22 of a row's largest to multiples of
    2^-32 of it).

    max_q_len: the most new tokens of any sequence, where the caller knows it (1 for a decode step);
    it only picks the kernel, and without it all tokens are taken for one sequence's, which costs a step
    of many sequences a quarter of its time. `out`: a tensor of q's shape that shares nothing with what
    the call reads (rows outside every sequence are left as they were; in a new tensor they are undefined). `workspace`: a uint8
    CUDA tensor of at least paged_attention_workspace(...) bytes, for callers that keep one; calls
    that may run at once need their own. Without it one is taken from torch's allocator per call."""
    try:
        dt, dev, code = q.dtype, q.device, _DTYPES[q.dtype]
        tokens, hq, dim = q.shape
        pages, page_size, hk, pool_dim = shape = k_pages.shape
        seqs, width = page_table.shape
        qs, kp, vp = q.stride(), k_pages.stride(), v_pages.stride()
        table_stride, in_row = page_table.stride()
        fine = (out is None and workspace is None and code and q.is_cuda and hk > 0 and hq > 0
                and hq % hk == 0 and pool_dim == dim and page_size > 0 and v_pages.shape == shape
                and qs[2] == kp[3] == vp[3] == in_row == 1 and k_pages.dtype is dt
                and v_pages.dtype is dt and page_table.dtype is _I32 and kv_lens.dtype is _I32
                and q_starts.dtype is _I32 and k_pages.device == dev and v_pages.device == dev
                and page_table.device == dev and kv_lens.device == dev and q_starts.device == dev
                and kv_lens.shape == (seqs,) and q_starts.shape == (seqs + 1,)
                and kv_lens.is_contiguous() and q_starts.is_contiguous()
                and (scale is None or -_BIG < scale < _BIG)
                and (max_q_len is None or 0 <= max_q_len < 2 ** 31)
                and not (_grad() and (q.requires_grad or k_pages.requires_grad or v_pages.requires_grad)))
    except (AttributeError, KeyError, ValueError, TypeError):
        fine = False
    if not fine or type(max_q_len) not in (int, type(None)):
        _check_attention(q, k_pages, v_pages, page_table, kv_lens, q_starts, scale, max_q_len, out,
                         workspace)
    if scale is None:
        scale = dim ** -0.5 if dim else 1.0
    if out is None:
        out = torch.empty((tokens, hq, dim), dtype=dt, device=dev)
    if tokens == 0 or seqs == 0:
        return out
    if workspace is None:
        ws_bytes = _workspace_size(dev, tokens, seqs, hq, hk, dim, page_size, width, dt, max_q_len)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    os_ = out.stride()
    _launch(_abi.ks_paged_attention, _abi.ATTENTION_ARGS.pack(
        out.data_ptr(), q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
        kv_lens.data_ptr(), q_starts.data_ptr(), workspace.data_ptr(), ws_bytes, tokens, seqs, hq, hk,
        dim, pages, page_size, width, table_stride, max_q_len or 0, os_[0], os_[1], qs[0], qs[1],
        kp[0], kp[1], kp[2], vp[0], vp[1], vp[2], scale, _abi.KS_ATTENTION_CAUSAL if causal else 0,
        code, 0), dev)
    return out
