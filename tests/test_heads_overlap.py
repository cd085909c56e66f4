"""Outputs of the calls on heads and attention that share memory with what another part of the
call reads or writes are refused, before the device is looked at.  Every call here is refused:
the addresses are never read."""
import pytest

import nvfp4_frozen_projection_gb300 as pk

P = 0x7000_0000_0000
INVALID = 1
ROWS, N, D = 8, 4, 64
STEP = 2**20  # between tensors that are apart


@pytest.fixture(scope="module")
def lib():
    from nvfp4_frozen_projection_gb300 import build
    build.build()
    return pk.load_library()


def heads(place, rows=ROWS, n=N, ld=None, off=0):
    """Tensor number `place`, `off` values in."""
    return pk._HeadsStruct(P + place * STEP + 2 * off, rows, n, n * D if ld is None else ld)


def refused(lib, rc):
    assert rc == INVALID
    return b"memory" in lib.pact_last_error() or b"in part" in lib.pact_last_error()


# where a tensor lies that shares memory with the one at place 0: itself, from its last row on,
# up to its first, and from the middle of a row on with rows further apart
SHARED = [dict(), dict(off=(ROWS - 1) * N * D + 64), dict(off=-(ROWS - 1) * N * D - 64), dict(ld=8 * D, off=2 * D)]


@pytest.mark.parametrize("at", SHARED)
@pytest.mark.parametrize("a,b", [("q_out", "k"), ("k_out", "q"), ("q_out", "k_out")])
def test_rotation(lib, a, b, at):
    t = {n: heads(i + 1) for i, n in enumerate(("q", "k", "q_out", "k_out"))}
    t[b], t[a] = heads(0), heads(0, **at)
    assert refused(lib, lib.pact_qk_norm_rope(t["q"], t["k"], D, 64, P, P, 0, None, None, 1e-5, t["q_out"], t["k_out"],
                                              None))


@pytest.mark.parametrize("at", SHARED)
@pytest.mark.parametrize("a,b", [("dq", "dyk"), ("dk", "dyq"), ("dq", "dk"), ("dq", "k"), ("dk", "q")])
def test_rotation_backward(lib, a, b, at):
    t = {n: heads(i + 1) for i, n in enumerate(("dyq", "dyk", "q", "k", "dq", "dk"))}
    t[b], t[a] = heads(0), heads(0, **at)
    assert refused(lib, lib.pact_qk_norm_rope_bwd(t["dyq"], t["dyk"], t["q"], t["k"], D, 64, P, P, 0, P, P, 1e-5,
                                                  t["dq"], t["dk"], None, None, None, 0, None))


@pytest.mark.parametrize("at", SHARED)
@pytest.mark.parametrize("b", ["q", "k", "v"])
def test_attention(lib, b, at):
    if b == "q" and not at:
        at = dict(off=64)  # o may be q itself, and no other
    t = {n: heads(i + 1) for i, n in enumerate("qkvo")}
    t[b], t["o"] = heads(0), heads(0, **at)
    assert refused(lib, lib.pact_attention_fwd(t["q"], t["k"], t["v"], D, P, P, 1, 1, 0.125, t["o"], P + 9 * STEP,
                                               None, 0, None))


@pytest.mark.parametrize("b", ["q", "k", "v", "o"])
def test_lse_over_a_tensor(lib, b):
    t = {n: heads(i + 1) for i, n in enumerate("qkvo")}
    for lse in (t[b].p, t[b].p + 2 * ROWS * N * D - 4, t[b].p - 4 * ROWS * N + 4):
        assert refused(lib, lib.pact_attention_fwd(t["q"], t["k"], t["v"], D, P, P, 1, 1, 0.125, t["o"], lse, None, 0,
                                                   None))


@pytest.mark.parametrize("at", SHARED)
@pytest.mark.parametrize("a,b", [(a, b) for a in ("dq", "dk", "dv") for b in ("q", "k", "v", "o", "do")] +
                         [("dq", "dk"), ("dk", "dv"), ("dv", "dq")])
def test_attention_backward(lib, a, b, at):
    names = ("do", "q", "k", "v", "o", "dq", "dk", "dv")
    t = {n: heads(i + 1) for i, n in enumerate(names)}
    t[b], t[a] = heads(0), heads(0, **at)
    assert refused(lib, lib.pact_attention_bwd(*[t[n] for n in names[:5]], P + 20 * STEP, D, P, P, 1, 1, 0.125,
                                               t["dq"], t["dk"], t["dv"], P + 30 * STEP, 1 << 30, None))


@pytest.mark.parametrize("a", ["dq", "dk", "dv"])
def test_attention_backward_lse(lib, a):
    names = ("do", "q", "k", "v", "o", "dq", "dk", "dv")
    t = {n: heads(i + 1) for i, n in enumerate(names)}
    assert refused(lib, lib.pact_attention_bwd(*[t[n] for n in names[:5]], t[a].p + 128, D, P, P, 1, 1, 0.125,
                                               t["dq"], t["dk"], t["dv"], P + 30 * STEP, 1 << 30, None))


def test_a_single_row_between_rows(lib):
    """A row in the gap of a wider matrix is apart from its columns until it reaches them."""
    wide = heads(0, ld=16 * D)
    for off in (3 * 16 * D + 12 * D + 8, 3 * 16 * D + 3 * D, 15 * D):
        one = heads(0, rows=1, off=off)
        rc = lib.pact_attention_bwd(heads(1, rows=1), heads(2, rows=1), heads(3), heads(4), heads(5, rows=1),
                                    P + 20 * STEP, D, P, P, 1, 1, 0.125, one, wide, heads(6), P + 30 * STEP, 1 << 30,
                                    None)
        assert refused(lib, rc)
