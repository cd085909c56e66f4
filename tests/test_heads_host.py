"""The calls on heads, attention and gradient lists without a GPU: bad arguments are refused
before the device is looked at; and the plain forms of the GPU tests against differences
and identities that they do not use."""
import ctypes

import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk

P = 0x7000_0000_0000  # an address that is aligned and never read: every call here is refused
INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from nvfp4_frozen_projection_gb300 import build
    build.build()
    return pk.load_library()


def heads(rows=8, n=4, d=64, p=P, ld=None):
    return pk._HeadsStruct(p, rows, n, n * d if ld is None else ld)


def test_turns_refusals(lib):
    f = lib.pact_rope_turns
    assert f(None, 4, P, None) == INVALID
    assert f(P, 4, None, None) == INVALID
    assert f(P, 0, P, None) == SHAPE
    assert f(P, 257, P, None) == SHAPE
    assert f(P + 4, 4, P, None) == ALIGN


def rope(lib, q=None, k=None, D=64, rot=64, pos=P, turns=P, gq=None, gk=None, eps=1e-5, qo=None, ko=None):
    return lib.pact_qk_norm_rope(heads() if q is None else q, heads(n=2, p=P + 2**20) if k is None else k, D, rot,
                                 pos, turns, 0, gq, gk, eps, heads(p=P + 2**22) if qo is None else qo,
                                 heads(n=2, p=P + 2**24) if ko is None else ko, None)


def test_rope_refusals(lib):
    for d in (0, 8, 24, 272):
        assert rope(lib, D=d) == SHAPE
    for rot in (0, 8, 24, 80, -16):
        assert rope(lib, rot=rot) == SHAPE
    assert rope(lib, q=heads(p=0)) == INVALID
    assert rope(lib, q=heads(p=P + 8)) == ALIGN
    assert rope(lib, q=heads(rows=0)) == SHAPE
    assert rope(lib, q=heads(rows=2**30 + 1)) == SHAPE
    assert rope(lib, q=heads(n=0)) == SHAPE
    assert rope(lib, q=heads(ld=248)) == SHAPE
    assert rope(lib, q=heads(ld=260)) == SHAPE
    assert rope(lib, q=heads(ld=2**30 + 8)) == SHAPE
    assert rope(lib, k=heads(rows=7, n=2)) == SHAPE
    assert rope(lib, qo=heads(n=2)) == SHAPE
    assert rope(lib, pos=None) == INVALID
    assert rope(lib, turns=None) == INVALID
    assert rope(lib, pos=P + 2) == ALIGN
    assert rope(lib, turns=P + 4) == ALIGN
    assert rope(lib, gq=P) == INVALID
    assert rope(lib, gq=P, gk=P + 2) == ALIGN
    for eps in (-1.0, float("nan"), float("inf")):
        assert rope(lib, eps=eps) == INVALID
    assert rope(lib, qo=heads(p=P + 16)) == INVALID           # overlaps q in part
    assert rope(lib, qo=heads(ld=512)) == INVALID             # q itself, other rows


def test_rope_backward_refusals(lib):
    def f(dgq=None, dgk=None, gq=P, gk=P, q=heads(p=P + 2**21), ws=P, size=1 << 30, dq=heads(p=P + 2**22)):
        return lib.pact_qk_norm_rope_bwd(heads(), heads(n=2, p=P + 2**20), q, heads(n=2, p=P + 2**23), 64, 64, P, P, 0,
                                         gq, gk, 1e-5, dq, heads(n=2, p=P + 2**24), dgq, dgk, ws, size, None)
    need = lib.pact_qk_norm_rope_bwd_workspace_size(8, 4, 2, 64)
    assert need > 0
    assert f(dgq=P) == INVALID
    assert f(q=None) == INVALID
    assert f(dgq=P, dgk=P, gq=None, gk=None) == INVALID
    assert f(dgq=P, dgk=P + 2) == ALIGN
    assert f(dgq=P, dgk=P, ws=None) == INVALID
    assert f(dgq=P, dgk=P, size=need - 1) == INVALID
    assert f(dgq=P, dgk=P, ws=P + 128) == INVALID
    assert f(dq=heads(p=P + 32)) == INVALID
    assert f(dq=heads(p=P + 2**21 + 32)) == INVALID
    for args in ((0, 4, 2, 64), (8, 0, 2, 64), (8, 4, 2, 24), (8, 4, 2, 272), (2**30 + 1, 4, 2, 64)):
        assert lib.pact_qk_norm_rope_bwd_workspace_size(*args) == 0


def attn(lib, q=None, k=None, v=None, D=64, cq=P, ck=P, n=2, scale=0.125, o=None, lse=P, ws=None,
         size=0):
    return lib.pact_attention_fwd(heads() if q is None else q, heads(n=2) if k is None else k,
                                  heads(n=2) if v is None else v, D, cq, ck, n, 1, scale,
                                  heads() if o is None else o, lse, ws, size, None)


def test_attention_refusals(lib):
    for d in (0, 8, 24, 144, -16):
        assert attn(lib, D=d) == SHAPE
    assert attn(lib, k=heads(n=3), v=heads(n=3)) == SHAPE
    assert attn(lib, v=heads(n=4)) == SHAPE
    assert attn(lib, v=heads(rows=9, n=2)) == SHAPE
    assert attn(lib, o=heads(rows=9)) == SHAPE
    assert attn(lib, q=heads(p=P + 2)) == ALIGN
    assert attn(lib, cq=None) == INVALID
    assert attn(lib, ck=P + 2) == ALIGN
    assert attn(lib, lse=None) == INVALID
    assert attn(lib, lse=P + 2) == ALIGN
    for n in (0, -1, 2**20 + 1):
        assert attn(lib, n=n) == SHAPE
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attn(lib, scale=s) == INVALID
    wide = heads(rows=2**30, n=65536, d=16)
    assert attn(lib, q=wide, k=wide, v=wide, o=wide, D=16) == SHAPE  # too many tiles


def test_attention_parts_refusals(lib):
    def size(tq=4, hq=8, tk=4096, hk=2, d=64, n=1):
        return lib.pact_attention_fwd_workspace_size(tq, hq, tk, hk, d, n)
    assert size() > 0 and size() % 4 == 0
    assert size(tk=2047) == size(tq=8192, hk=8) == size(n=3) == 0  # few keys, enough units
    for bad in (dict(tq=0), dict(hq=0), dict(tk=0), dict(hk=0), dict(hk=3), dict(d=24), dict(d=144), dict(n=0),
                dict(tq=2**30 + 1), dict(tk=2**30 + 1), dict(n=2**20 + 1), dict(hq=65552, hk=1), dict(tq=-4)):
        assert size(**bad) == 0

    def back(tq, hq, tk, hk, d=64, n=1):
        return lib.pact_attention_bwd_workspace_size(tq, hq, tk, hk, d, n)
    own = 2048 * 8 * 4
    assert back(2048, 8, 2048, 8) == own                       # every head has its keys
    assert back(2048, 8, 2048, 1) > own + 2 * 2 * 2048 * 64 * 4  # shared heads: dk and dv in parts
    assert back(64, 8, 4096, 8) > 64 * 8 * 64 * 2 * 4            # many keys: dq in parts
    for bad in ((0, 8, 8, 8), (8, 8, 8, 3), (8, 8, 0, 8), (8, 8, 8, 8, 24), (8, 8, 8, 8, 64, 0)):
        assert back(*bad) == 0

    def f(ws, n):
        k = heads(rows=4096, n=2, p=P + 2**21)
        return attn(lib, q=heads(rows=4, n=8), k=k, v=k, n=1, o=heads(rows=4, n=8, p=P + 2**20), ws=ws, size=n)
    assert f(P + 64, 1 << 30) == INVALID
    assert f(P, size() - 1) == INVALID


def test_attention_backward_refusals(lib):
    def f(do=heads(), o=heads(), dq=heads(), dk=heads(n=2), lse=P, ws=P, size=1 << 30):
        return lib.pact_attention_bwd(do, heads(), heads(n=2), heads(n=2), o, lse, 64, P, P, 1, 1, 0.125, dq, dk,
                                      heads(n=2), ws, size, None)
    need = lib.pact_attention_bwd_workspace_size(8, 4, 8, 2, 64, 1)
    assert need >= 8 * 4 * 4
    assert lib.pact_attention_bwd_workspace_size(0, 4, 8, 2, 64, 1) == 0
    assert f(do=heads(rows=9)) == SHAPE
    assert f(o=heads(p=0)) == INVALID
    assert f(dq=heads(n=2)) == SHAPE
    assert f(dk=heads(n=2, p=P + 8)) == ALIGN
    assert f(lse=None) == INVALID
    assert f(ws=None) == INVALID
    assert f(ws=P + 64) == INVALID
    assert f(size=need - 1) == INVALID


def test_grad_norm_refusals(lib):
    assert [lib.pact_grad_chunks(n) for n in (-1, 0, 1, 4096, 4097)] == [0, 0, 1, 1, 2]

    def f(data=P, numel=P, first=P, count=2, chunks=3, out=P, limit=1.0, norm=P, ws=P, size=1 << 20):
        t = pk._ListStruct(data, numel, first, count, chunks)
        return lib.pact_clip_grad_norm(ctypes.byref(t), out, limit, norm, ws, size, None)
    for name in ("data", "numel", "first", "out", "norm", "ws"):
        assert f(**{name: None}) == INVALID
    for name in ("data", "numel", "first", "out"):
        assert f(**{name: P + 4}) == ALIGN
    assert f(norm=P + 2) == ALIGN
    for n in (0, -1, 2**20 + 1):
        assert f(count=n) == SHAPE
    for n in (-1, 2**40 + 1):
        assert f(chunks=n) == SHAPE
    for limit in (-1.0, float("nan")):
        assert f(limit=limit) == INVALID
    assert f(size=lib.pact_grad_norm_workspace_size() - 1) == INVALID


# ---------------------------------------------------------------- the plain forms
def rnd(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_form(pairs):
    f = 10.0 ** (-torch.arange(8, dtype=torch.float64) / 8)
    x, pos = rnd(5, 3, 32), torch.tensor([0, 1, 7, 100, -3])
    y = ref.turn(x, pos, f, pairs)
    assert torch.equal(y[..., 16:], x[..., 16:]) and torch.equal(y[0], x[0])
    # a rotation keeps each pair's length, and two of them add up
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if pairs else (slice(0, 8), slice(8, 16))
    assert torch.allclose(y[..., a]**2 + y[..., b]**2, x[..., a]**2 + x[..., b]**2)
    assert torch.allclose(ref.turn(y, pos, f, pairs), ref.turn(x, 2 * pos, f, pairs))
    assert torch.allclose(ref.turn(y, pos, f, pairs, -1.0), x)


@pytest.mark.parametrize("norm", [False, True])
def test_rope_backward_form(norm):
    f = 10.0 ** (-torch.arange(8, dtype=torch.float64) / 8)
    x, dy, pos = rnd(5, 3, 32, seed=1), rnd(5, 3, 32, seed=2), torch.tensor([0, 1, 7, 100, -3])
    gam = rnd(32, seed=3) if norm else None
    dx, dg, _, _ = ref.rope_bwd(dy, pos, f, False, x, gam, 1e-2)

    def loss(x, gam):
        return float((ref.rope(x, pos, f, False, gam, 1e-2)[0] * dy).sum())
    h, e = 1e-5, rnd(5, 3, 32, seed=4)
    assert abs((loss(x + h * e, gam) - loss(x - h * e, gam)) / (2 * h) - float((dx * e).sum())) < 1e-6
    if norm:
        e = rnd(32, seed=5)
        assert abs((loss(x, gam + h * e) - loss(x, gam - h * e)) / (2 * h) - float((dg * e).sum())) < 1e-6


@pytest.mark.parametrize("causal", [False, True])
def test_attention_forms(causal):
    """The forward against a loop over single queries; the backward against differences,
    and two mistakes that differences must not forgive."""
    cq, ck = [0, 3, 3, 9, 11], [0, 5, 7, 11, 11]
    q, k, v, do = rnd(11, 4, 16, seed=1), rnd(11, 2, 16, seed=2), rnd(11, 2, 16, seed=3), rnd(11, 4, 16, seed=4)
    o, lse, *_ = ref.attention(q, k, v, cq, ck, causal, 0.25)
    for q0, q1, k0, k1 in ref.sequences(cq, ck):
        for i in range(q1 - q0):
            n = min(k1 - k0, i + 1 + (k1 - k0) - (q1 - q0)) if causal else k1 - k0
            for h in range(4):
                if n <= 0:
                    assert float(o[q0 + i, h].abs().sum()) == 0 and float(lse[h, q0 + i]) == -float("inf")
                    continue
                w = torch.stack([(q[q0 + i, h] * k[k0 + j, h // 2]).sum() * 0.25 for j in range(n)]).exp()
                assert torch.allclose(o[q0 + i, h], (w[:, None] * v[k0:k0 + n, h // 2]).sum(0) / w.sum())
                assert torch.allclose(lse[h, q0 + i], w.sum().log())
    (dq, dk, dv), _ = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, causal, 0.25)

    def loss(q, k, v):
        return float((ref.attention(q, k, v, cq, ck, causal, 0.25)[0] * do).sum())
    h = 1e-5
    for i, g in enumerate((dq, dk, dv)):
        e = rnd(*g.shape, seed=9 + i)
        up, down = [q, k, v], [q, k, v]
        up[i], down[i] = up[i] + h * e, down[i] - h * e
        diff = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(diff - float((g * e).sum())) < 1e-6
        if i < 2:
            assert abs(diff - float((g * e).sum()) / 0.25) > 1e-3   # the scale left out
    (dq0, *_), _ = ref.attention_bwd(do, q, k, v, torch.zeros_like(o), lse, cq, ck, causal, 0.25)
    assert float((dq0 - dq).abs().max()) > 1e-3                      # delta left out
