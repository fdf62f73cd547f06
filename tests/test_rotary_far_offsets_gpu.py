"""GPU test of the rotated append where the first new token's slot and its offset add up past 31 bits, against angles of 60
digits. Bounds as in test_rotary_gpu.py."""
from decimal import Decimal, getcontext

import pytest
import torch

from paged_reference import HALF, Problem
from test_paged_gpu import BF, F32, check, lla  # noqa: F401
from test_rotary_gpu import ERR

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
def test_positions_past_31_bits(lla, dtype):  # noqa: F811
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    freq = [1.0, 0.1, 10000.0 ** -0.25, 1e-4, 3.0, -0.7, 1e-9, 1e5]
    P = Problem([500, 90], [5, 3], 2, 1, 16, 16, 16, dtype, False, seed=3)
    offsets = [2 ** 31 - 1, 2 ** 31 - 400, 0, -2 ** 31, 7, 2 ** 31 - 87, 2 ** 31 - 88, 2 ** 31 - 89]
    pos = [495 + x for x in offsets[:5]] + [87 + x for x in offsets[5:]]
    spec = lla.RotarySpec(16, freq=freq)
    cache, q, _, starts = P.cuda(lla)
    g = torch.Generator().manual_seed(1)
    k = torch.randn(8, 1, 16, generator=g).to(dtype)
    got, _ = lla.lla_paged_append_rotary(k.cuda(), k.cuda(), cache, starts, spec, q,
                                         offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert lla.lla_stream_status() == 0
    angle = torch.tensor([[float((Decimal(p) * Decimal(f)) % two_pi) for f in freq] for p in pos], dtype=torch.float64)[:, None]
    slots = [(int(P.table[b, j // 16]), j % 16) for b, j in [(0, 495 + i) for i in range(5)] + [(1, 87 + i) for i in range(3)]]
    keys = torch.stack([cache.k_pages[pg, :, at] for pg, at in slots])
    for x, y in ((P.q, got), (k, keys)):
        a, b = x[..., :8].double(), x[..., 8:].double()
        want = torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)
        tol = ERR[dtype] * (a.abs() + b.abs()).repeat(1, 1, 2)
        check("y", y, want, tol + HALF[dtype] * (want.abs() + tol))
