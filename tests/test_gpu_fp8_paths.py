"""The FP8 product on every one of its ways, with no addend, another tensor as addend (32-
and 16-byte aligned) and the output itself as addend, against a 64-bit product on the GPU.

Bound, as for the other products (u = 2^-24): 2^-8 of the value for the BF16 store, and
2^-23 (128 + blocks + 8) sum |x w| for the FP32 additions of a block in any order,
truncated or rounded, one fused step a block, the scales' product, the join and the addend.
"""
import pytest
import torch

import fp8_paths
import nvfp4_frozen_projection_gb300 as pk
from test_gpu_fp8 import Guarded

pytestmark = pytest.mark.gpu


def _inputs(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + 3 * n + 5 * k)
    x = pk.pact_quant_fp8(torch.randn(m, k, device="cuda", generator=g).bfloat16())
    w = pk.pact_pack_weight_fp8_fwd(0.02 * torch.randn(n, k, device="cuda", generator=g))
    return x, w, torch.randn(m, n, device="cuda", generator=g).bfloat16()


def _values(x, w):
    k = x.cols
    a = x.q.double() * x.s.double().t().repeat_interleave(128, 1)[:, :k]
    s = w.s.double().repeat_interleave(128, 0)[:w.rows].repeat_interleave(128, 1)[:, :k]
    return a, w.q.double() * s


@pytest.mark.parametrize("m,n,k", fp8_paths.SHAPES)
def test_product(m, n, k):
    x, w, add = _inputs(m, n, k)
    a, b = _values(x, w)
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    del a, b
    out = Guarded((m, n), torch.bfloat16)
    odd = torch.empty(m * n + 8, dtype=torch.bfloat16, device="cuda")[8:].view(m, n)
    assert odd.data_ptr() % 32 == 16
    for kind in ("none", "other", "itself", "odd"):
        res = {"none": None, "other": add, "itself": out.t, "odd": odd}[kind]
        if kind in ("itself", "odd"):
            res.copy_(add)
        y = pk.pact_linear_fp8_fwd(x, w, residual=res, y=out.t)
        pk.pact_check_status()
        out.check()
        exact = want if res is None else want + add.double()
        size = mag if res is None else mag + add.double().abs()
        tol = 2.0 ** -8 * exact.abs() + 2.0 ** -23 * (136 + -(-k // 128)) * size
        over = (y.double() - exact).abs() - tol * (1 + 2.0 ** -8)
        assert bool((over <= 0).all()), (kind, float(over.max()))
        if kind == "other":
            kept = y.clone()
        assert kind in ("none", "other") or torch.equal(y, kept), kind
    pk.pact_linear_fp8_fwd(x, w, residual=odd, y=odd)  # 16-byte aligned, in place
    pk.pact_check_status()
    assert torch.equal(odd, kept)


def test_shapes_take_their_ways_on_this_device():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for s in fp8_paths.SHAPES:
        assert pk.pact_test_fp8_plan(*s, sms=sms) == pk.pact_test_fp8_plan(*s), s
