"""The norm of many gradients and clipping, against 64-bit sums."""
import math

import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu


def tensors(sizes, seed=0, std=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n, generator=g, device="cuda") * std for n in sizes]


def exact(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


SIZES = [[1], [0, 5, 0], [4096], [4097, 4095, 3], [16, 2048 * 16, 16 * 8192] * 3, [700001, 1, 33],
         list(range(1, 300))]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("over", [0.5, 4.0])
def test_clip(sizes, over):
    ts = tensors(sizes)
    norm = exact(ts)
    limit = norm / over
    keep = [t.clone() for t in ts]
    outs = [torch.full_like(t, 7.0) for t in ts]
    grads = pk.GradList(ts)
    # 16 squares and their sum in FP32 (all terms positive), the rest in FP64, one rounding
    tol = 9 * ref.E + ref.E
    got = pk.pact_clip_grad_norm(grads, limit, out=pk.GradList(outs))
    assert abs(got.item() - norm) <= tol * norm
    assert abs(pk.pact_grad_norm(grads).item() - norm) <= tol * norm
    coef = min(1.0, limit / (norm + 1e-6))
    for t, k, o in zip(ts, keep, outs):
        assert torch.equal(t, k)
        want = k.double() * coef
        # the coefficient's own rounding, the norm's, limit's to FP32, and the product's
        ref.check(o, want, (tol + 4 * ref.E) * want.abs(), "out")
    pk.pact_clip_grad_norm(grads, limit)
    for t, o in zip(ts, outs):
        assert torch.equal(t, o)


def test_unaligned_views():
    """Tensors that begin at any value, and outputs that begin at another."""
    flat = tensors([50000])[0]
    at, views = 0, []
    for n in (1, 3, 4097, 4096, 10, 8195, 5):
        views.append(flat[at:at + n])
        at += n + 1  # the values between stay
    want = flat.clone()
    limit = exact(views) / 3
    pk.pact_clip_grad_norm(pk.GradList(views), limit)
    moved = torch.zeros_like(flat, dtype=torch.bool)
    at = 0
    for v in views:
        moved[at:at + v.numel()] = True
        at += v.numel() + 1
    assert torch.equal(flat[~moved], want[~moved])
    w = want[moved].double() / 3
    ref.check(flat[moved], w, 16 * ref.E * w.abs() + 1e-6 * w.abs() / limit, "clipped")


@pytest.mark.parametrize("size", [1e-40, 1e-30, 1e-15, 1.0, 1e20, 3e38])
def test_no_overflow_or_underflow(size):
    ts = [torch.full((1000,), size, device="cuda"), torch.zeros(5000, device="cuda"),
          torch.tensor([size / 2], device="cuda")]
    want = exact(ts)
    if want < 3.4e38:
        assert abs(pk.pact_grad_norm(pk.GradList(ts)).item() - want) <= 10 * ref.E * want + 2.0**-149
    else:
        assert pk.pact_grad_norm(pk.GradList(ts)).item() == math.inf
    # clipped all the same: the coefficient comes from the FP64 norm
    pk.pact_clip_grad_norm(pk.GradList(ts), want / 4)
    coef = min(1.0, want / 4 / (want + 1e-6))
    w = torch.tensor(size, dtype=torch.float32).double().item() * coef
    assert abs(ts[0][17].item() - w) <= 16 * ref.E * w + 2.0**-149


def test_nan_infinity_and_limits():
    def run(bad, limit):
        ts = tensors([100, 5000])
        ts[1][77] = bad
        norm = pk.pact_clip_grad_norm(pk.GradList(ts), limit).item()
        return norm, ts

    norm, ts = run(math.nan, 1.0)
    assert math.isnan(norm) and all(torch.isnan(t).all() for t in ts)
    norm, ts = run(math.inf, 1.0)
    assert norm == math.inf and int((ts[0] != 0).sum()) == 0 and math.isnan(ts[1][77].item())
    norm, ts = run(0.5, 0.0)
    assert norm > 0.5 and all(int((t != 0).sum()) == 0 for t in ts)
    norm, ts = run(0.5, math.inf)
    assert torch.equal(ts[0], tensors([100, 5000])[0])


def test_repeats_itself_and_replays():
    ts = tensors([100000, 77, 4096 * 40])
    grads = pk.GradList(ts)
    outs = [torch.zeros_like(t) for t in ts]
    olist = pk.GradList(outs)
    limit = exact(ts) / 2
    n1 = pk.pact_clip_grad_norm(grads, limit, out=olist)
    first = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            n2 = pk.pact_clip_grad_norm(grads, limit, out=olist)
    for o in outs:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(n1, n2) and all(torch.equal(a, b) for a, b in zip(first, outs))


def test_past_32_bits():
    """A tensor of more than 2^31 values; what its end holds counts and is clipped."""
    t = torch.zeros(2**31 + 5000, device="cuda")
    t[-3], t[7] = 3.0, 4.0
    grads = pk.GradList([t])
    assert pk.pact_clip_grad_norm(grads, 1.0).item() == 5.0
    assert abs(t[-3].item() - 0.6) < 1e-6 and abs(t[7].item() - 0.8) < 1e-6
    assert int((t != 0).sum()) == 2


def test_refusals():
    a, b = tensors([100, 100])
    for bad in (lambda: pk.GradList([]), lambda: pk.GradList([a.double()]), lambda: pk.GradList([a.cpu()]),
                lambda: pk.GradList([a, a]), lambda: pk.GradList([a, a[50:]]),
                lambda: pk.GradList([a.view(10, 10).t()[:, :5]]), lambda: pk.pact_grad_norm([a]),
                lambda: pk.pact_clip_grad_norm(pk.GradList([a]), 1.0, out=pk.GradList([b[:99]])),
                lambda: pk.pact_clip_grad_norm(pk.GradList([a]), 1.0, norm=b)):
        with pytest.raises(ValueError):
            bad()
    for limit in (-1.0, math.nan):
        with pytest.raises(pk.PactError):
            pk.pact_clip_grad_norm(pk.GradList([a]), limit)
