"""The sums for dgamma_q and dgamma_k over the blocks of the rotation's backward: the same
bits however often and beside whatever they are computed."""
import pytest
import torch

import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu


def signs(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1).bfloat16()


def make(t, h, d, seed):
    """x of plus and minus one, and a gradient of its sign and size 0 to 3."""
    x = signs((t, h, d), seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    return x, (x * torch.randint(0, 4, x.shape, generator=g, device="cuda")).bfloat16()


def test_the_same_sums_beside_other_work():
    """On two streams at once, with other kernels of the library on a third."""
    t, hq, hk, d = 4000, 16, 4, 64
    (q, dyq), (k, dyk) = make(t, hq, d, 1), make(t, hk, d, 3)
    gam = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    turns = pk.pact_rope_turns(10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d))

    def run():
        return pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, turns, q, k, gam, gam, dgamma_q=True, dgamma_k=True)

    first = run()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(50):
        for s in streams[:2]:
            with torch.cuda.stream(s):
                got.append(run())
        with torch.cuda.stream(streams[2]):
            pk.pact_qk_norm_rope(q, k, pos, turns, gam, gam)
    torch.cuda.synchronize()
    for again in got:
        assert all(torch.equal(a, b) for a, b in zip(again, first))
