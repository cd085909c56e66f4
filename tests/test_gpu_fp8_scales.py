"""The FP8 product where an activation's scale times a weight's is below 2^-126, on each of
its ways, against a 64-bit product on the GPU.

Bound (u = 2^-24; FP32 numbers below 2^-126 are multiples of 2^-149, BF16 ones of 2^-133):
the other products' 2^-8 of the value and 2^-23 (136 + blocks) sum |x w|, and
  2^-150 sum |qx qw|     the scales' product, off by half a step of 2^-149,
  2^-150 (blocks + 20)   a fused step a block, the joins of at most 16 warps and the rest,
  2^-134                 the store.
"""
import pytest
import torch

import fp8_paths
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu

# a shape for each way and each size of its groups
SHAPES = list({fp8_paths.instance(*s): s for s in reversed(fp8_paths.SHAPES)}.values())


def _product(x, w):
    k = x.cols
    sx = x.s.double().t().repeat_interleave(128, 1)[:, :k]
    sw = w.s.double().repeat_interleave(128, 0)[:w.rows].repeat_interleave(128, 1)[:, :k]
    qx, qw = x.q.double(), w.q.double()
    a, b = qx * sx, qw * sw
    return a @ b.t(), a.abs() @ b.abs().t(), qx.abs() @ qw.abs().t()


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products_of_scales_below_the_normal_range(m, n, k):
    """Rows of magnitudes 2^-112 to 2^-126, and one of zeros, against weights of 0.02."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x = torch.randn(m, k, device="cuda", generator=g)
    x = (x * torch.exp2(-112.0 - torch.arange(m, device="cuda") % 15)[:, None]).bfloat16()
    zero = m // 2
    if m > 1:
        x[zero] = 0.0
    xq = pk.pact_quant_fp8(x)
    w = pk.pact_pack_weight_fp8_fwd(0.02 * torch.randn(n, k, device="cuda", generator=g))
    assert float(xq.s.min()) * float(w.s.min()) < 2.0 ** -126
    y = pk.pact_linear_fp8_fwd(xq, w)
    pk.pact_check_status()
    want, mag, codes = _product(xq, w)
    blocks = -(-k // 128)
    tol = (2.0 ** -8 * want.abs() + 2.0 ** -23 * (136 + blocks) * mag
           + 2.0 ** -150 * (codes + blocks + 20) + 2.0 ** -134)
    over = (y.double() - want).abs() - tol * (1 + 2.0 ** -8)
    assert bool((over <= 0).all()), float(over.max())
    assert float(want.abs().max()) > 2.0 ** -118  # ordinary BF16 numbers among them
    if m > 1:
        assert not bool(y[zero].any())


def test_zero_blocks_against_the_smallest_weights():
    """Zero codes give zero whatever their scales' product rounds to."""
    x = pk.pact_quant_fp8(torch.zeros(40, 272, dtype=torch.bfloat16, device="cuda"))
    assert bool((x.s == 2.0 ** -126).all())
    for std in (1.0, 1e-4, 1e-30):
        w = pk.pact_pack_weight_fp8_fwd(std * torch.randn(144, 272, device="cuda"))
        y = pk.pact_linear_fp8_fwd(x, w)
        assert not bool(y.any())
