"""gated_add_rms_norm where its CTAs take several rows one after the other, every row against 64 bits. Tolerances are those of
test_gpu_gated_norm.
"""
import pytest
import torch

import row_wise_rmsnorm_ks_gb300 as ks
from test_gpu_decode_ops import no_faults, normal  # noqa: F401
from test_gpu_gated_norm import check

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


# Width, type, and the rows that an SM has at once: 2048 threads' worth of CTAs, at most 32, of one row or, a warp each, eight.
@pytest.mark.parametrize("hidden, dtype, at_once", [
    (256, BF16, 64), (512, F16, 64), (256, F32, 64),                # a warp a row, of 1 and 2 vectors a thread
    (1024, BF16, 32), (600, F32, 21),                               # 2 vectors
    (1288, BF16, 32), (4096, F16, 16), (8192, F32, 4),              # 4
    (16392, BF16, 6), (12288, F32, 5), (32768, F16, 4),             # 8, the next row fetched meanwhile
    (1001, BF16, 32), (1002, F16, 32), (1004, BF16, 32), (1001, F32, 32), (1002, F32, 32), (16383, BF16, 2),  # rows no vector fits
    (20480, F32, 3), (40000, BF16, 4), (65536, BF16, 2),            # read three times, by vectors
    (16385, BF16, 4), (16387, F32, 4), (16386, F16, 4),             # and value by value
])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["token", "row", None])
def test_several_rows_for_each_team(cuda_device, hidden, dtype, at_once, post, gate):
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    rows = 2 * sms * at_once + sms // 2 + 3  # some teams do a third one
    x, r = normal((rows, hidden), dtype, 1, cuda_device, 3.0), normal((rows, hidden), dtype, 2, cuda_device, 2.0)
    x *= torch.exp2(torch.arange(rows, device=cuda_device) % 7 - 3.0).to(dtype)[:, None]  # a row's norm is its own
    w = (1 + 0.1 * normal((hidden,), F32, 3, cuda_device)).to(dtype)
    p = (0.5 + 0.1 * normal((hidden,), F32, 4, cuda_device)).to(dtype) if post else None
    g = None if gate is None else normal((rows, hidden if gate == "token" else 1), dtype, 5, cuda_device, 0.5)
    x0, r0 = x.clone(), r.clone()
    ks.gated_add_rms_norm(x, r, w, post_weight=p, gate=g, residual_scale=0.75, block_scale=1.5)
    for at in range(0, rows, 512):  # some rows at a time: the reference is eight times their size
        s = slice(at, at + 512)
        check(x[s], r[s], x0[s], r0[s], w, p, None if g is None else g[s], 0.75, 1.5, 1e-6, f"rows from {at}")
