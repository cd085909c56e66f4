"""Norms of queries and keys with the rotary embedding, forward and backward, against the
plain 64-bit forms."""
import math

import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu
# FP32 up to the rounding: a row's sum of squares (13 additions), the square root and two
# divisions, two products, the sine (2 units) of an angle rounded to FP32, two more products
FP32 = 24 * ref.E


def make(t, hq, hk, d, norm, seed=0, far=100000):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

    pos = torch.randint(0, far, (t,), generator=g, device="cuda", dtype=torch.int32)
    gam = [(1.0 + normal(d, std=0.1).float()).bfloat16() for _ in range(2)] if norm else [None, None]
    return normal(t, hq, d), normal(t, hk, d, std=3.0), pos, gam, (normal(t, hq, d), normal(t, hk, d))


def freqs(rot):
    return 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


SHAPES = [(1, 32, 8, 64, 64), (1, 1, 1, 16, 16), (3, 5, 1, 80, 32), (17, 8, 8, 96, 96),
          (129, 4, 2, 112, 48), (300, 16, 4, 128, 128), (77, 3, 3, 256, 256), (40, 2, 1, 240, 16),
          (9000, 2, 1, 64, 64)]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("t,hq,hk,d,rot", SHAPES)
def test_forward(t, hq, hk, d, rot, pairs, norm):
    q, k, pos, (gq, gk), _ = make(t, hq, hk, d, norm)
    f = freqs(rot)
    oq, ok = pk.pact_qk_norm_rope(q, k, pos, pk.pact_rope_turns(f), gq, gk, eps=1e-5, interleaved=pairs)
    for got, x, gam, name in ((oq, q, gq, "q"), (ok, k, gk, "k")):
        want, mag = ref.rope(x, pos, f, pairs, gam, 1e-5)
        ref.check(got, want, ref.U * (1 + ref.U) * want.abs() + FP32 * mag, name)
        if rot < d and not norm:
            assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("t,hq,hk,d,rot", SHAPES)
def test_backward(t, hq, hk, d, rot, pairs, norm):
    q, k, pos, (gq, gk), (dyq, dyk) = make(t, hq, hk, d, norm)
    f = freqs(rot)
    x = (q, k) if norm else (None, None)
    dq, dk, dgq, dgk = pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, pk.pact_rope_turns(f), *x, gq, gk, 1e-5,
                                                pairs, dgamma_q=norm, dgamma_k=norm)
    for got, dg, dy, xx, gam, heads, name in ((dq, dgq, dyq, q, gq, hq, "q"), (dk, dgk, dyk, k, gk, hk, "k")):
        want, wg, mag, magg = ref.rope_bwd(dy, pos, f, pairs, xx, gam, 1e-5)
        # two sums over a head of D values more
        ref.check(got, want, ref.U * (1 + ref.U) * want.abs() + 2 * FP32 * mag, "d" + name)
        if norm:
            # a thread adds the heads of at most two tokens, then 32 groups, 19 blocks and 5 lanes
            ref.check(dg, wg, ref.E * (2 * heads + 64 + 2 * 24) * magg, "dgamma " + name)


@pytest.mark.parametrize("pos", [0, 1, -1, 123456789, 2**31 - 1, -2**31])
def test_far_positions(pos):
    """The angle of a far position is exact before its rounding: its fraction of a turn is
    computed here in whole numbers."""
    f = freqs(64)
    turns = pk.pact_rope_turns(f)
    for a, b in zip(f.tolist(), turns.tolist()):
        turn = a / (2 * math.pi)  # two roundings of 2^-53, which 2^-51 covers
        assert abs(b / 2.0**64 - turn) <= 2.0**-51 * turn + 2.0**-64
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[..., :32] = 1.0
    p = torch.tensor([pos], dtype=torch.int32, device="cuda")
    y, _ = pk.pact_qk_norm_rope(x, x, p, turns)
    for i, n in enumerate(turns.tolist()):
        frac = (pos * n) % 2**64 / 2.0**64
        c, s = math.cos(2 * math.pi * frac), math.sin(2 * math.pi * frac)
        assert abs(y[0, 0, i].item() - c) <= ref.U * abs(c) + 8 * ref.E
        assert abs(y[0, 0, 32 + i].item() - s) <= ref.U * abs(s) + 8 * ref.E


def test_negative_frequencies_turn_back():
    f = freqs(32)
    q, k, pos, _, _ = make(20, 2, 1, 32, False)
    a = pk.pact_qk_norm_rope(q, k, pos, pk.pact_rope_turns(-f))
    want, mag = ref.rope(q, -pos, f, False)
    ref.check(a[0], want, ref.U * (1 + ref.U) * want.abs() + FP32 * mag, "q")


@pytest.mark.parametrize("norm", [False, True])
def test_views_and_in_place(norm):
    """Heads that are columns of one fused matrix, turned in place: the same bits as apart,
    and the columns beside them stay."""
    t, hq, hk, d = 100, 4, 2, 96
    q, k, pos, (gq, gk), _ = make(t, hq, hk, d, norm)
    turns = pk.pact_rope_turns(freqs(d))
    want = pk.pact_qk_norm_rope(q, k, pos, turns, gq, gk)
    fused = torch.randn(t, (hq + 2 * hk) * d, device="cuda").bfloat16()
    v0 = fused[:, (hq + hk) * d:].clone()
    vq = fused[:, :hq * d].view(t, hq, d)
    vk = fused[:, hq * d:(hq + hk) * d].view(t, hk, d)
    vq.copy_(q)
    vk.copy_(k)
    pk.pact_qk_norm_rope(vq, vk, pos, turns, gq, gk, q_out=vq, k_out=vk)
    assert torch.equal(vq, want[0]) and torch.equal(vk, want[1])
    assert torch.equal(fused[:, (hq + hk) * d:], v0)


def test_backward_is_the_transpose():
    """<R x, dy> = <x, R^T dy> of the rotation alone."""
    q, k, pos, _, (dyq, dyk) = make(50, 3, 1, 128, False)
    turns = pk.pact_rope_turns(freqs(128))
    y, _ = pk.pact_qk_norm_rope(q, k, pos, turns)
    dx, *_ = pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, turns)
    a, b = (y.double() * dyq.double()).sum(), (q.double() * dx.double()).sum()
    size = (y.double().abs() * dyq.double().abs()).sum()
    assert abs(a - b) <= 2.1 * ref.U * size


def test_backward_repeats_itself_and_replays():
    q, k, pos, (gq, gk), (dyq, dyk) = make(3000, 8, 2, 64, True)
    turns = pk.pact_rope_turns(freqs(64))

    def run():
        return pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, turns, q, k, gq, gk, dgamma_q=True, dgamma_k=True)

    first = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            held = run()
    for t in held:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, held):
        assert torch.equal(a, b)


def test_past_32_bits():
    """The last tokens of tensors of more than 2^31 values: the same bits as from their own."""
    t, n = 140000, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    q, dy = (torch.randn(t, 128, 128, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, dk = q[:, :1].contiguous(), dy[:, :1].contiguous()
    gam = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    turns = pk.pact_rope_turns(freqs(128))
    a = pk.pact_qk_norm_rope(q, k, pos, turns, gam, gam)
    b = pk.pact_qk_norm_rope(q[-n:], k[-n:], pos[-n:], turns, gam, gam)
    assert torch.equal(a[0][-n:], b[0]) and torch.equal(a[1][-n:], b[1])
    a = pk.pact_qk_norm_rope_bwd(dy, dk, pos, turns, q, k, gam, gam)
    b = pk.pact_qk_norm_rope_bwd(dy[-n:], dk[-n:], pos[-n:], turns, q[-n:], k[-n:], gam, gam)
    assert torch.equal(a[0][-n:], b[0]) and torch.equal(a[1][-n:], b[1])


def test_zero_rows_and_a_zero_eps():
    """A head of zeros under eps > 0 stays zero; its gradient is finite."""
    q, k, pos, (gq, gk), (dyq, dyk) = make(4, 2, 1, 64, True)
    q.zero_()
    turns = pk.pact_rope_turns(freqs(64))
    y, _ = pk.pact_qk_norm_rope(q, k, pos, turns, gq, gk, eps=1e-6)
    assert int((y != 0).sum()) == 0
    dx, _, dg, _ = pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, turns, q, k, gq, gk, 1e-6, dgamma_q=True,
                                            dgamma_k=True)
    assert torch.isfinite(dx).all() and int((dg != 0).sum()) == 0


def test_refusals():
    q, k, pos, (gq, gk), _ = make(4, 2, 1, 64, True)
    turns = pk.pact_rope_turns(freqs(64))
    for bad in (lambda: pk.pact_qk_norm_rope(q.float(), k, pos, turns),
                lambda: pk.pact_qk_norm_rope(q[0], k, pos, turns),
                lambda: pk.pact_qk_norm_rope(q, k[..., :32], pos, turns),
                lambda: pk.pact_qk_norm_rope(q, k, pos.long(), turns),
                lambda: pk.pact_qk_norm_rope(q, k, pos[:3], turns),
                lambda: pk.pact_qk_norm_rope(q, k, pos, turns.int()),
                lambda: pk.pact_qk_norm_rope(q.transpose(0, 1), k, pos, turns),
                lambda: pk.pact_qk_norm_rope(q, k, pos, turns, gq.float(), gk.float()),
                lambda: pk.pact_qk_norm_rope(q, k, pos, turns, q_out=k),
                lambda: pk.pact_qk_norm_rope(q, k, pos, turns.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: pk.pact_qk_norm_rope(q, k[:3], pos, turns),
                lambda: pk.pact_qk_norm_rope(q, k, pos, turns, gq),
                lambda: pk.pact_qk_norm_rope(q, k, pos, torch.cat((turns, turns))),
                lambda: pk.pact_qk_norm_rope_bwd(q, k, pos, turns, None, None, gq, gk),
                lambda: pk.pact_qk_norm_rope_bwd(q, k, pos, turns, dgamma_q=True, dgamma_k=True),
                lambda: pk.pact_qk_norm_rope_bwd(q, k, pos, turns, q, k, gq, gk, dgamma_q=True)):
        with pytest.raises(pk.PactError):
            bad()
