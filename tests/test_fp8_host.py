"""FP8 entry points without a GPU: the C calls check their arguments before they look
for a device, so bad ones are refused with the same codes here; and the plain forms of
the GPU tests against formats and identities they do not use."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_ref as ref
import nvfp4_frozen_projection_gb300 as pk

P = 0x7000_0000_0000  # an address that is aligned and never read: every call here is refused
INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from nvfp4_frozen_projection_gb300 import build
    build.build()
    return pk.load_library()


def f8(rows, cols, q=P, s=P):
    return ctypes.byref(pk._FP8Struct(q, s, rows, cols))


def test_quant_refusals(lib):
    f = lib.pact_quant_fp8
    assert f(None, 4, 64, 64, f8(4, 64), None) == INVALID
    assert f(P, 0, 64, 64, f8(0, 64), None) == SHAPE
    assert f(P, -1, 64, 64, f8(-1, 64), None) == SHAPE
    assert f(P, 2**30 + 1, 64, 64, f8(2**30 + 1, 64), None) == SHAPE
    for k in (0, 8, 24, 2**24 + 16, -16):
        assert f(P, 4, k, k, f8(4, k), None) == SHAPE
    assert f(P, 2**30, 2**24, 2**24, f8(2**30, 2**24), None) == SHAPE  # too many blocks
    assert f(P, 4, 64, 56, f8(4, 64), None) == SHAPE
    assert f(P, 4, 64, 68, f8(4, 64), None) == SHAPE
    assert f(P + 8, 4, 64, 64, f8(4, 64), None) == ALIGN
    assert f(P, 4, 64, 64, None, None) == INVALID
    assert f(P, 4, 64, 64, f8(4, 64, q=0), None) == INVALID
    assert f(P, 4, 64, 64, f8(4, 64, s=0), None) == INVALID
    assert f(P, 4, 64, 64, f8(5, 64), None) == SHAPE
    assert f(P, 4, 64, 64, f8(4, 64, q=P + 4), None) == ALIGN
    assert f(P, 4, 64, 64, f8(4, 64, s=P + 2), None) == ALIGN


@pytest.mark.parametrize("backward", [0, 1])
def test_pack_refusals(lib, backward):
    f = lib.pact_pack_weight_fp8_bwd if backward else lib.pact_pack_weight_fp8_fwd

    def out(n, k, **kw):
        return f8(k, n, **kw) if backward else f8(n, k, **kw)

    assert f(None, 32, 64, out(32, 64), None) == INVALID
    assert f(P, 24, 64, out(24, 64), None) == SHAPE
    assert f(P, 32, 72, out(32, 72), None) == SHAPE
    assert f(P, 2**24, 2**24, out(2**24, 2**24), None) == SHAPE
    assert f(P + 4, 32, 64, out(32, 64), None) == ALIGN
    assert f(P, 32, 64, out(64, 32), None) == SHAPE
    assert f(P, 32, 64, None, None) == INVALID


@pytest.mark.parametrize("name", ["pact_linear_fp8_fwd", "pact_linear_fp8_dgrad"])
def test_linear_refusals(lib, name):
    f = getattr(lib, name)
    assert f(None, f8(32, 64), None, P, None) == INVALID
    assert f(f8(4, 64), None, None, P, None) == INVALID
    assert f(f8(4, 64), f8(32, 64), None, None, None) == INVALID
    assert f(f8(0, 64), f8(32, 64), None, P, None) == SHAPE
    assert f(f8(2**30 + 1, 64), f8(32, 64), None, P, None) == SHAPE
    assert f(f8(4, 64), f8(32, 80), None, P, None) == SHAPE
    assert f(f8(4, 72), f8(32, 72), None, P, None) == SHAPE
    assert f(f8(4, 64), f8(24, 64), None, P, None) == SHAPE
    assert f(f8(2**30, 64), f8(2**17, 64), None, P, None) == SHAPE  # too many tiles
    assert f(f8(4, 64, q=0), f8(32, 64), None, P, None) == INVALID
    assert f(f8(4, 64), f8(32, 64, s=0), None, P, None) == INVALID
    assert f(f8(4, 64, q=P + 8), f8(32, 64), None, P, None) == ALIGN
    assert f(f8(4, 64), f8(32, 64), P + 2, P, None) == ALIGN
    assert f(f8(4, 64), f8(32, 64), None, P + 8, None) == ALIGN
    for add in (P + 16, P - 16, P + 2 * 4 * 32 - 16):  # in part the output's memory
        assert f(f8(4, 64), f8(32, 64), add, P, None) == INVALID


def test_norm_refusals(lib):
    f = lib.pact_add_rmsnorm_quant_fp8
    ok = dict(x=P, res=P, gamma=P, M=4, H=64, eps=1e-5, h=P, out=None, rstd=P)

    def call(**kw):
        a = {**ok, **kw}
        out = a["out"] or f8(a["M"], a["H"])
        return f(a["x"], a["res"], a["gamma"], a["M"], a["H"], a["eps"], a["h"], out, a["rstd"],
                 None)

    for k in ("x", "gamma", "rstd"):
        assert call(**{k: None}) == INVALID
    assert call(res=None) == INVALID and call(h=None) == INVALID
    for m in (0, -3, 2**30 + 1):
        assert call(M=m) == SHAPE
    for h in (0, 8, 40, 16400):
        assert call(H=h) == SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == INVALID
    for k in ("x", "res", "gamma", "h"):
        assert call(**{k: P + 8}) == ALIGN
    assert call(rstd=P + 2) == ALIGN
    assert call(out=f8(4, 80)) == SHAPE
    for k in ("x", "res", "h"):
        assert call(**{k: P + 2 * 4 * 64 - 16}) == INVALID


def test_norm_bwd_refusals(lib):
    f, size = lib.pact_add_rmsnorm_bwd, lib.pact_add_rmsnorm_bwd_workspace_size
    M = 10000
    ok = dict(h=P, gamma=P, rstd=P, dy=P, dres=P, M=M, H=64, dh=P, dg=P, ws=P, n=size(M, 64))

    def call(**kw):
        a = {**ok, **kw}
        return f(*(a[k] for k in ("h", "gamma", "rstd", "dy", "dres", "M", "H", "dh", "dg", "ws",
                                  "n")), None)

    for k in ("h", "gamma", "rstd", "dy", "dh", "ws"):
        assert call(**{k: None}) == INVALID
    for m in (0, 2**30 + 1):
        assert call(M=m) == SHAPE
    for h in (0, 24, 16400):
        assert call(H=h) == SHAPE
    for k in ("h", "gamma", "dy", "dres", "dh"):
        assert call(**{k: P + 8}) == ALIGN
    assert call(dg=P + 2) == ALIGN
    assert call(n=ok["n"] - 1) == INVALID and call(ws=P + 128) == INVALID
    for k in ("h", "dy", "dres"):
        assert call(**{k: P + 16}) == INVALID
    assert size(0, 64) == 0 and size(4, 40) == 0 and size(4, 16400) == 0
    assert size(M, 64) % 256 == 0 and size(M, 64) >= 64 * 4
    assert size(4, 64) == 0  # a small tensor needs none


def test_scale_counts(lib):
    assert lib.pact_fp8_scale_count(7, 144) == 14
    assert lib.pact_fp8_weight_scale_count(129, 144) == 4
    assert lib.pact_fp8_scale_count(0, 144) == 0
    assert pk.FP8.scale_shape(7, 144) == (2, 7) and pk.FP8Weight.scale_shape(129, 144) == (2, 2)


def test_bindings_refuse_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    g = torch.ones(64, dtype=torch.bfloat16)
    q = pk.FP8(x.to(torch.float8_e4m3fn), torch.ones(1, 4))
    for call in (lambda: pk.pact_quant_fp8(x), lambda: pk.pact_pack_weight_fp8_fwd(x.float()),
                 lambda: pk.pact_linear_fp8_fwd(q, q), lambda: pk.pact_linear_fp8_dgrad(x, q),
                 lambda: pk.pact_add_rmsnorm_quant_fp8(x, x, g),
                 lambda: pk.pact_add_rmsnorm_bwd(x, g, torch.ones(4), x)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- the plain forms
def test_e4m3_rounding_against_torch():
    """Every midpoint of neighbouring E4M3 values, and points beside it."""
    codes = torch.arange(0, 0x7F, dtype=torch.uint8)
    v = codes.view(torch.float8_e4m3fn).double().numpy()
    mid = (v[1:] + v[:-1]) / 2
    pts = np.concatenate([v, mid, mid * (1 + 2**-20), mid * (1 - 2**-20)])
    pts = np.concatenate([pts, -pts])
    want = torch.from_numpy(pts).float().to(torch.float8_e4m3fn).double().numpy()
    got = ref.e4m3(pts)
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))
    assert ref.e4m3(1e9) == 448.0 and ref.e4m3(-465.0) == -448.0


def test_quant_error_is_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((9, 400)).astype(np.float32)
    x[4] = 0
    q, s = ref.quant_fp32(x)
    d = ref.dequant(q, s)
    step = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * ref.spread(s.T.astype(np.float64), 400))
    assert np.all(np.abs(d - x) <= step * (1 + 2.0 ** -20))
    top = ref.per_block(np.abs(q), lambda b: b.max(1))
    assert np.all((top == 448) | (ref.per_block(np.abs(x), lambda b: b.max(1)) == 0))


def test_pack_is_one_weight_in_two_layouts():
    rng = np.random.default_rng(1)
    w = rng.standard_normal((144, 272)).astype(np.float32)
    q, s = ref.pack_fp32(w)
    qt, st = ref.pack_fp32(np.ascontiguousarray(w.T))
    assert np.array_equal(q.T, qt) and np.array_equal(s.T, st)
    assert np.array_equal(ref.dequant_weight(q, s).T, ref.dequant_weight(qt, st))


def _planted(h, gamma, rstd, dy, dres, mistake):
    n = h * rstd[:, None]
    dn = dy * (1 if mistake == "gamma left out" else gamma)
    c = (dn * n).sum(1, keepdims=True) / (h.shape[1] - (mistake == "mean over H - 1"))
    if mistake == "projection left out":
        c = 0 * c
    dh = rstd[:, None] ** (2 if mistake == "rstd squared" else 1) * (dn - n * c)
    return dh


@pytest.mark.parametrize("mistake", ["", "gamma left out", "mean over H - 1",
                                     "projection left out", "rstd squared"])
def test_norm_bwd_against_differences(mistake):
    rng = np.random.default_rng(2)
    h, dy = 2.0 * rng.standard_normal((3, 48)), rng.standard_normal((3, 48))
    gamma, eps = 1 + 0.3 * rng.standard_normal(48), 1e-5
    _, rstd = ref.norm(h, gamma, eps)
    dh, dgamma, _ = ref.norm_bwd(h, gamma, rstd, dy, None)
    if mistake:
        dh = _planted(h, gamma, rstd, dy, None, mistake)
    t, worst = 1e-6, 0.0
    for _ in range(3):
        E, e = rng.standard_normal(h.shape), rng.standard_normal(48)
        fd = ((ref.norm(h + t * E, gamma, eps)[0] - ref.norm(h - t * E, gamma, eps)[0]) * dy).sum()
        worst = max(worst, abs(fd / (2 * t) - (dh * E).sum()))
        fd = ((ref.norm(h, gamma + t * e, eps)[0] - ref.norm(h, gamma - t * e, eps)[0]) * dy).sum()
        assert abs(fd / (2 * t) - (dgamma * e).sum()) < 1e-6
    assert (worst < 1e-6) == (not mistake)
