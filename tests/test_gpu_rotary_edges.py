"""gptq_rotary at far positions, without slack for the reference's own angle: a row's angle is turns * position modulo 2^64
in units of 2^-64 turns, here in whole numbers of any length.

Tolerance, for u = 2^-11 (fp16) or 2^-8 (bf16): one rounding of the angle's turns to fp32 (pi 2^-25 rad), sine and cosine
within 2^-22, products and sum three roundings: u |ref| + 2^-20 (|a| + |b|) + 2^-25."""
import math

import pytest
import torch

import gptq_bit_weight_gemm_gb300 as g

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_bit_weight_gemm_gb300 import build as lib_build
    lib_build.build()
    assert torch.cuda.is_available()
    yield
    assert g.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (64, 10000.0), (6, 1.5)])
def test_angles_are_exact_at_every_position(dtype, interleaved, rot, theta):
    gen = torch.Generator().manual_seed(rot)
    turns, _ = g.rotary_table(rot, theta=theta)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (200,), generator=gen)
    pos[:8] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 131071, 10 ** 9 + 7])
    x = torch.randn((200, 3, (rot + 7) // 8 * 8), generator=gen).to(dtype)
    q, _ = g.rotary(x.to(DEV), x[:, :1].to(DEV), pos.int().to(DEV), turns, interleaved=interleaved)
    whole = [[t * p % 2 ** 64 for t in turns.tolist()] for p in pos.tolist()]
    angle = torch.tensor([[w / 2 ** 64 * 2 * math.pi for w in row] for row in whole], dtype=torch.float64)[:, None]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    d, got = x.double(), q.cpu().double()
    u = 2.0 ** (-11 if dtype == torch.float16 else -8)
    for to, ref in ((a, d[..., a] * angle.cos() - d[..., b] * angle.sin()), (b, d[..., a] * angle.sin() + d[..., b] * angle.cos())):
        tol = u * ref.abs() + 2.0 ** -20 * (d[..., a].abs() + d[..., b].abs()) + 2.0 ** -25
        assert bool(((got[..., to] - ref).abs() <= tol).all())
    assert torch.equal(got[..., rot:], d[..., rot:])
