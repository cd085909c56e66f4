"""How far the FP8 encode's definition, q = e4m3(RN(x RN(448 / t))), is from the nearest
code to 448 x / t: the two differ at ties alone, and there by one step."""
import numpy as np
import pytest
import torch

import fp8_ref as ref


@pytest.mark.parametrize("m,k,std", [(512, 2048, 1.0), (300, 1040, 1e-2), (64, 16384, 30.0)])
def test_codes_differ_at_ties_only(m, k, std):
    rng = np.random.default_rng(m)
    x = torch.from_numpy((rng.standard_normal((m, k)) * std).astype(np.float32)).bfloat16()
    x = x.float().numpy()
    q, s = ref.quant_fp32(x)
    t = np.maximum(ref.per_block(np.abs(x), lambda b: b.max(1)).astype(np.float64), ref.T_MIN)
    v = x.astype(np.float64) * 448.0 / ref.spread(t, k)
    near = ref.e4m3(v)
    differ = q != near
    # BF16 values and maxima have 8 bits: a quotient is a tie or at least 2^-13 off it, and
    # the two roundings of the definition move it by less than 2^-22
    mid = (q + near)[differ] / 2
    assert np.array_equal(mid, v[differ])
    assert np.all(np.abs(q - near)[differ] <= 2.0 ** -2 * np.abs(mid))
    assert differ.mean() < 1e-3  # 3 in 10,000 codes of normal data
    # either code is a nearest one: the value is off by half a step, no more
    step = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * ref.spread(s.T.astype(np.float64), k))
    assert np.all(np.abs(ref.dequant(q, s) - x) <= step * (1 + 2.0 ** -20))
