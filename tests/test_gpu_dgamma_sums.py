"""The sums for dgamma_q and dgamma_k over the blocks of the rotation's backward: right at
every size, and the same bits however often and beside whatever they are computed."""
import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu

# tokens, query heads, key heads, D: from one block a side to more blocks than the sums' kernel
# has rows of threads, with few and many columns
SIZES = [(1, 1, 1, 16), (7, 8, 2, 64), (777, 8, 8, 96), (3000, 8, 2, 64), (2500, 32, 8, 128), (5000, 4, 4, 256),
         (20000, 32, 8, 64)]


def signs(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1).bfloat16()


def make(t, h, d, seed):
    """x of plus and minus one, and a gradient of its sign and size 0 to 3."""
    x = signs((t, h, d), seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    return x, (x * torch.randint(0, 4, x.shape, generator=g, device="cuda")).bfloat16()


@pytest.mark.parametrize("t,hq,hk,d", SIZES)
def test_the_sums_every_time(t, hq, hk, d):
    """With eps 0 and position 0 dgamma is the sum of dy x, none of whose terms is negative: a
    block's sum left out or counted twice would be far outside the bound, and a hundred calls
    give the same bits."""
    (q, dyq), (k, dyk) = make(t, hq, d, 1), make(t, hk, d, 3)
    gam = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(t, dtype=torch.int32, device="cuda")
    turns = pk.pact_rope_turns(torch.ones(8, dtype=torch.float64, device="cuda"))

    def run():
        return pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, turns, q, k, gam, gam, 0.0, dgamma_q=True, dgamma_k=True)[2:]

    got = [run() for _ in range(100)]
    for g, dy, x, heads in zip(got[0], (dyq, dyk), (q, k), (hq, hk)):
        want = (dy.double() * x.double()).sum((0, 1))
        # 1 / sqrt(1) within 2 units in the last place, the product, and FP32 sums: the heads of
        # at most two tokens a thread, 32 groups, 10 blocks a thread and 8 joins
        assert ((g.double() - want).abs() <= (2.0**-22 + ref.E * (2 * heads + 64)) * want).all()
    for again in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(again, got[0]))


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
