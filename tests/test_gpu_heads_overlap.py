"""Outputs of the calls on heads and attention over their inputs: what is allowed gives the bits
of tensors that are apart, what is not is refused and leaves every tensor as it was."""
import pytest
import torch

import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu


def normal(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def offsets(lens):
    return torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")


# one tile and two, ragged ends beside the next sequence, keys in parts, rows that see nothing,
# groups that do not divide 128
CASES = [([37], [37], 4, 2, 64), ([300, 1, 255], [300, 1, 255], 5, 5, 96), ([130] * 40, [130] * 40, 2, 1, 64),
         ([1100] * 3, [1100] * 3, 48, 12, 128), ([1, 1, 3, 1], [4000, 77, 5000, 1], 6, 2, 96),
         ([2048], [2048], 1, 1, 128), ([100, 60], [40, 60], 2, 1, 64), ([129], [129], 3, 1, 48),
         ([1030] * 6, [1030] * 6, 32, 8, 64)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,hq,hk,d", CASES, ids=[f"{len(c[0])}x{max(c[1])}h{c[2]}d{c[4]}" for c in CASES])
def test_o_over_q(lq, lk, hq, hk, d, causal):
    q, k, v = normal((sum(lq), hq, d), 1), normal((sum(lk), hk, d), 2), normal((sum(lk), hk, d), 3)
    args = k, v, offsets(lq), offsets(lk), causal
    o, lse = pk.pact_attention_fwd(q, *args)
    for _ in range(5):
        x = q.clone()
        o2, lse2 = pk.pact_attention_fwd(x, *args, o=x)
        assert o2 is x and torch.equal(x, o) and torch.equal(lse, lse2)
    pk.pact_check_status()


def test_a_single_token_of_a_fused_matrix():
    """One row among the rows of the keys' matrix: apart from its columns, though between them."""
    t, hq, hk, d = 50, 4, 2, 64
    w = (hq + 2 * hk) * d
    qkv, grads = normal((t, w), 1), torch.zeros(t, w, device="cuda").bfloat16()

    def cut(m):
        q, k, v = m.split([hq * d, hk * d, hk * d], 1)
        return q[-1:].view(1, hq, d), k.unflatten(1, (hk, d)), v.unflatten(1, (hk, d))

    q, k, v = cut(qkv)
    args = offsets([1]), offsets([t])
    apart = [x.clone(memory_format=torch.contiguous_format) for x in (q, k, v)]
    do = normal((1, hq, d), 2)
    o, lse = pk.pact_attention_fwd(*apart, *args)
    want = pk.pact_attention_bwd(do, *apart, o, lse, *args)
    dq, dk, dv = cut(grads)
    o2, lse2 = pk.pact_attention_fwd(q, k, v, *args, o=q)
    assert torch.equal(o2, o) and torch.equal(lse, lse2)
    q.copy_(apart[0])
    pk.pact_attention_bwd(do, q, k, v, o, lse, *args, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(a, b) for a, b in zip(cut(grads), want))
    assert (grads[:-1, :hq * d] == 0).all()


def test_rotated_in_place_backward():
    """dq over dyq or q, and dk over dyk or k."""
    t, hq, hk, d = 70, 4, 4, 64
    q, k, dyq, dyk = (normal((t, h, d), i) for i, h in enumerate((hq, hk, hq, hk)))
    gam = normal((d,), 9)
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    turns = pk.pact_rope_turns(torch.linspace(0.1, 1.0, 32, dtype=torch.float64, device="cuda"))

    def run(dyq, dyk, q, k, **out):
        return pk.pact_qk_norm_rope_bwd(dyq, dyk, pos, turns, q, k, gam, gam, **out)

    want = run(dyq, dyk, q, k)[:2]
    for over_q in (0, 2):
        for over_k in (1, 3):
            x = [a.clone() for a in (dyq, dyk, q, k)]
            got = run(*x, dq=x[over_q], dk=x[over_k])[:2]
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    t, h, d = 200, 4, 64
    q, k, v, do = (normal((t, h, d), i) for i in range(4))
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    turns = pk.pact_rope_turns(torch.linspace(0.1, 1.0, 32, dtype=torch.float64, device="cuda"))
    c = offsets([t])
    o, lse = pk.pact_attention_fwd(q, k, v, c, c)
    big = normal((2 * t, h, d), 9)
    keep = [x.clone() for x in (q, k, v, do, o, lse, big)]
    for bad in (lambda: pk.pact_qk_norm_rope(q, k, pos, turns, q_out=k),
                lambda: pk.pact_qk_norm_rope(q, k, pos, turns, k_out=q),
                lambda: pk.pact_qk_norm_rope(q, k, pos, turns, q_out=v, k_out=v),
                lambda: pk.pact_qk_norm_rope_bwd(q, k, pos, turns, dq=k),
                lambda: pk.pact_qk_norm_rope_bwd(q, k, pos, turns, dk=q),
                lambda: pk.pact_qk_norm_rope_bwd(q, k, pos, turns, dq=big[:t], dk=big[t - 1:-1]),
                lambda: pk.pact_attention_fwd(q, k, v, c, c, o=k),
                lambda: pk.pact_attention_fwd(q, k, v, c, c, o=v),
                lambda: pk.pact_attention_fwd(big[:t], k, v, c, c, o=big[1:t + 1]),
                lambda: pk.pact_attention_fwd(q, k, v, c, c, lse=k.view(-1)[:2 * h * t].view(torch.float32).view(h, t)),
                lambda: pk.pact_attention_bwd(do, q, k, v, o, lse, c, c, dq=q),
                lambda: pk.pact_attention_bwd(do, q, k, v, o, lse, c, c, dk=k),
                lambda: pk.pact_attention_bwd(do, q, k, v, o, lse, c, c, dv=do),
                lambda: pk.pact_attention_bwd(do, q, k, v, o, lse, c, c, dk=big[:t], dv=big[:t]),
                lambda: pk.pact_attention_bwd(do, q, k, v, o, lse, c, c, dq=big[:t], dv=big[t - 1:-1])):
        with pytest.raises(pk.PactError):
            bad()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (q, k, v, do, o, lse, big)))
