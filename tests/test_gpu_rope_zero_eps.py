"""The rotation's backward with norms and eps 0: what is not there (groups without heads, places
behind a group's last head) adds nothing to dgamma."""
import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("t,hq,hk,d", [(1, 1, 1, 16), (3, 5, 1, 48), (37, 9, 3, 128), (700, 11, 2, 80), (60, 17, 4, 256)])
def test_dgamma_without_eps(t, hq, hk, d, pairs):
    g = torch.Generator(device="cuda").manual_seed(t)

    def normal(h):
        return torch.randn(t, h, d, generator=g, device="cuda").bfloat16()

    q, k, dyq, dyk = normal(hq), normal(hk), normal(hq), normal(hk)
    gam = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    f = 10000.0 ** (-torch.arange(0, 16, 2, dtype=torch.float64, device="cuda") / 16)
    dq, dk, dgq, dgk = pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, pk.pact_rope_turns(f), q, k, gam, gam, 0.0, pairs,
                                                dgamma_q=True, dgamma_k=True)
    for got, dg, dy, x, heads, name in ((dq, dgq, dyq, q, hq, "q"), (dk, dgk, dyk, k, hk, "k")):
        want, wg, mag, magg = ref.rope_bwd(dy, pos, f, pairs, x, gam, 0.0)
        # as with eps: FP32 products and sums before one rounding; a thread adds the heads of at
        # most two tokens, then come 32 groups and the blocks
        ref.check(got, want, ref.U * (1 + ref.U) * want.abs() + 48 * ref.E * mag, "d" + name)
        ref.check(dg, wg, ref.E * (2 * heads + 64 + 2 * 24) * magg, "dgamma " + name)
