"""Attention over packed sequences, forward and backward, against the plain 64-bit forms."""
import math

import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu


def cu(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def dev(c):
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def make(lq, lk, hq, hk, d, seed=0):
    tq, tk = max(1, sum(lq)), max(1, sum(lk))
    return (normal((tq, hq, d), seed), normal((tk, hk, d), seed + 1), normal((tk, hk, d), seed + 2),
            normal((tq, hq, d), seed + 3, 0.1), cu(lq), cu(lk))


# lengths of queries and keys, query and key heads, D
CASES = [
    ([1], [1], 1, 1, 64),
    ([1], [1], 4, 1, 16),
    ([37], [37], 4, 2, 64),
    ([128], [128], 1, 1, 128),
    ([256], [256], 2, 2, 32),
    ([129], [129], 3, 1, 48),                          # groups that do not divide 128
    ([300, 1, 255], [300, 1, 255], 5, 5, 96),
    ([1, 1, 1], [1000, 5, 129], 8, 2, 128),            # single tokens over held keys
    ([3, 200], [700, 333], 6, 2, 80),
    ([100, 60], [40, 60], 2, 1, 64),                   # more queries than keys: rows that see nothing
    ([5, 0, 130, 7], [9, 4, 0, 7], 4, 2, 112),         # sequences without queries, without keys
    ([600], [600], 12, 1, 64),
    ([130] * 40, [130] * 40, 2, 1, 64),                # more sequences than lanes of a warp
    ([1000], [1000], 8, 2, 128),
]
IDS = [f"{len(a)}seq{max(a)}x{max(b)}h{h}-{g}d{d}" for a, b, h, g, d in CASES]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,hq,hk,d", CASES, ids=IDS)
def test_forward(lq, lk, hq, hk, d, causal):
    q, k, v, _, cq, ck = make(lq, lk, hq, hk, d)
    o, lse = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), causal)
    pk.pact_check_status()
    wo, wl, bo, bl = ref.attention(q, k, v, cq, ck, causal, d ** -0.5)
    ref.check(o, wo, bo, "o")
    ref.check(lse, wl, bl, "lse")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,hq,hk,d", CASES, ids=IDS)
def test_backward(lq, lk, hq, hk, d, causal):
    q, k, v, do, cq, ck = make(lq, lk, hq, hk, d, 10)
    o, lse = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), causal)
    got = pk.pact_attention_bwd(do, q, k, v, o, lse, dev(cq), dev(ck), causal)
    pk.pact_check_status()
    want, bounds = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, causal, d ** -0.5)
    for g, w, b, name in zip(got, want, bounds, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)


# several units for every SM: units of all lengths in one CTA, tiles 0 or 1 without keys, rows
# that see nothing, keys that end in either half of a tile
MANY = [
    ([700, 1, 1300, 257, 64], [700, 1, 1300, 257, 64], 32, 32, 128),
    ([900, 300], [1000, 333], 60, 20, 80),
    ([640, 129, 513], [640, 129, 513], 64, 16, 96),
    ([300, 500, 40, 0, 7], [200, 577, 0, 5, 1200], 48, 48, 112),
    ([1100] * 3, [1100] * 3, 48, 12, 128),
    ([1030] * 6, [1030] * 6, 32, 8, 64),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,hq,hk,d", MANY, ids=[f"h{c[2]}-{c[3]}d{c[4]}" for c in MANY])
def test_many_units(lq, lk, hq, hk, d, causal):
    q, k, v, _, cq, ck = make(lq, lk, hq, hk, d, 50)
    o, lse = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), causal)
    pk.pact_check_status()
    wo, wl, bo, bl = ref.attention(q, k, v, cq, ck, causal, d ** -0.5)
    ref.check(o, wo, bo, "o")
    ref.check(lse, wl, bl, "lse")


def test_many_units_keep_a_nan_in_its_sequence():
    lens = [700, 77, 900]
    q, k, v, _, cq, ck = make(lens, lens, 32, 32, 128)
    args = dev(cq), dev(ck)
    o, lse = pk.pact_attention_fwd(q, k, v, *args)
    for t in (q, k, v):
        t[700:777] = math.nan
    o2, lse2 = pk.pact_attention_fwd(q, k, v, *args)
    pk.pact_check_status()
    for a, b in ((o, o2), (lse.t(), lse2.t())):
        assert torch.equal(a[:700], b[:700]) and torch.equal(a[777:], b[777:])


def test_a_large_group():
    """Groups above 128 heads are cut at their largest divisor."""
    for hq, hk in ((130, 1), (160, 1), (254, 2)):
        q, k, v, do, cq, ck = make([9], [33], hq, hk, 32)
        o, lse = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck))
        wo, wl, bo, bl = ref.attention(q, k, v, cq, ck, True, 32 ** -0.5)
        ref.check(o, wo, bo, "o")
        ref.check(lse, wl, bl, "lse")
        got = pk.pact_attention_bwd(do, q, k, v, o, lse, dev(cq), dev(ck))
        want, bounds = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, True, 32 ** -0.5)
        for g, w, b, name in zip(got, want, bounds, ("dq", "dk", "dv")):
            ref.check(g, w, b, name)


@pytest.mark.parametrize("std,scale", [(8.0, 0.125), (1.0, 3.0), (0.0, 0.125), (30.0, 1e-3)])
def test_scores_of_all_sizes(std, scale):
    """Sharp rows whose maximum moves from tile to tile, and flat ones."""
    lens = [700, 90]
    q, k, v, do, cq, ck = make(lens, lens, 4, 2, 64, 5)
    q = (q.float() * std).bfloat16()
    k = (k * torch.linspace(0.05, 1.0, k.shape[0], device="cuda")[:, None, None].bfloat16())
    o, lse = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), False, scale)
    wo, wl, bo, bl = ref.attention(q, k, v, cq, ck, False, scale)
    ref.check(o, wo, bo, "o")
    ref.check(lse, wl, bl, "lse")
    got = pk.pact_attention_bwd(do, q, k, v, o, lse, dev(cq), dev(ck), False, scale)
    want, bounds = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, False, scale)
    for g, w, b, name in zip(got, want, bounds, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)


def test_descending_scores_never_rescale_and_ascending_always_do():
    """One column a tile dominates: the running maximum moves at every tile, or never."""
    for order in (1.0, -1.0):
        n, d = 640, 64
        q = torch.ones(n, 1, d, device="cuda").bfloat16()
        k = (torch.arange(n, device="cuda").float()[:, None, None] * order * 0.02).expand(n, 1, d)
        k = k.bfloat16().contiguous()
        v = normal((n, 1, d), 3)
        o, lse = pk.pact_attention_fwd(q, k, v, dev([0, n]), dev([0, n]), False, 1.0)
        wo, wl, bo, bl = ref.attention(q, k, v, [0, n], [0, n], False, 1.0)
        ref.check(o, wo, bo, "o")
        ref.check(lse, wl, bl, "lse")


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (3, 1, 96), (2, 2, 128)])
def test_rows_behind_the_sequences_stay(hq, hk, d):
    q, k, v, do, *_ = make([300], [420], hq, hk, d)
    cq, ck = [10, 100, 100, 250], [7, 200, 210, 390]
    full = [torch.full_like(t, 5.0) for t in (q, q, k, v)]
    o, dq, dk, dv = full
    lse = torch.full((hq, 300), 5.0, device="cuda")
    pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), o=o, lse=lse)
    pk.pact_attention_bwd(do, q, k, v, o, lse, dev(cq), dev(ck), dq=dq, dk=dk, dv=dv)
    wo, wl, bo, bl = ref.attention(q, k, v, cq, ck, True, d ** -0.5)
    ref.check(o, wo, bo, "o")
    ref.check(lse, wl, bl, "lse")
    want, bounds = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, True, d ** -0.5)
    for g, w, b, name in zip((dq, dk, dv), want, bounds, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
    for t in (o, dq):
        assert (t[:10] == 5).all() and (t[250:] == 5).all()
    assert (lse[:, :10] == 5).all() and (lse[:, 250:] == 5).all()
    for t in (dk, dv):
        assert (t[:7] == 5).all() and (t[390:] == 5).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("hq,hk,d", [(2, 1, 64), (3, 1, 128)])
def test_a_nan_stays_in_its_sequence(bad, hq, hk, d):
    """Every value of the sequences on both sides of one full of NaN is what it is without."""
    lens = [150, 77, 201]
    q, k, v, do, cq, ck = make(lens, lens, hq, hk, d)
    args = dev(cq), dev(ck)
    o, lse = pk.pact_attention_fwd(q, k, v, *args)
    g = pk.pact_attention_bwd(do, q, k, v, o, lse, *args)
    q2, k2, v2, do2 = (t.clone() for t in (q, k, v, do))
    for t in (q2, k2, v2, do2):
        t[150:227] = bad
    o2, lse2 = pk.pact_attention_fwd(q2, k2, v2, *args)
    g2 = pk.pact_attention_bwd(do2, q2, k2, v2, o2, lse2, *args)
    pk.pact_check_status()
    for a, b in zip((o, *g), (o2, *g2)):
        assert torch.equal(a[:150], b[:150]) and torch.equal(a[227:], b[227:])
    assert torch.equal(lse[:, :150], lse2[:, :150]) and torch.equal(lse[:, 227:], lse2[:, 227:])
    assert torch.isnan(o2[150:227]).any()


def test_views_of_one_fused_matrix():
    """q, k, v and their gradients as columns of one matrix each: the same bits as apart."""
    t, hq, hk, d = 333, 4, 2, 64
    q, k, v, do, cq, ck = make([t], [t], hq, hk, d)
    args = dev(cq), dev(ck)
    o, lse = pk.pact_attention_fwd(q, k, v, *args)
    g = pk.pact_attention_bwd(do, q, k, v, o, lse, *args)
    w = (hq + 2 * hk) * d
    fused, grads = torch.zeros(t, w + 8, device="cuda").bfloat16(), torch.zeros(t, w + 8, device="cuda").bfloat16()

    def cut(m):
        return (m[:, :hq * d].unflatten(1, (hq, d)), m[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                m[:, (hq + hk) * d:w].unflatten(1, (hk, d)))

    for a, b in zip(cut(fused), (q, k, v)):
        a.copy_(b)
    o2, lse2 = pk.pact_attention_fwd(*cut(fused), *args)
    pk.pact_attention_bwd(do, *cut(fused), o2, lse2, *args, dq=cut(grads)[0], dk=cut(grads)[1], dv=cut(grads)[2])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(g, cut(grads)):
        assert torch.equal(a, b)
    assert (grads[:, w:] == 0).all()


def test_wild_offsets_stay_inside():
    """Offsets out of range or falling are taken into the tensors; nothing leads outside."""
    q, k, v, do, *_ = make([200], [200], 2, 1, 64)
    pad = torch.full((64, 2, 64), 3.0, device="cuda").bfloat16()
    for c in ([-5, 300], [150, 20], [0, 2**31 - 1, -2**31, 200], [500, 600]):
        buf = torch.cat((pad, q, pad))
        o = buf[64:264]
        lse = torch.zeros(2, 200, device="cuda")
        pk.pact_attention_fwd(q, k, v, dev(c), dev(c), o=o, lse=lse)
        pk.pact_attention_bwd(do, q, k, v, o, lse, dev(c), dev(c))
        pk.pact_check_status()
        assert (buf[:64] == 3).all() and (buf[264:] == 3).all()


def test_repeats_itself_on_streams_and_in_graphs():
    lens = [400, 33, 517]
    q, k, v, do, cq, ck = make(lens, lens, 8, 2, 128)
    args = dev(cq), dev(ck)

    def run():
        o, lse = pk.pact_attention_fwd(q, k, v, *args)
        return (o, lse, *pk.pact_attention_bwd(do, q, k, v, o, lse, *args))

    first = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:  # two calls at once
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([run() for _ in range(3)])
    graphs = []
    for s in streams:
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                held = run()
        graphs.append((g, held))
    for g, held in graphs:
        for t in held:
            t.zero_()
    for s, (g, _) in zip(streams, graphs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for got in [r for o in outs for r in o] + [h for _, h in graphs]:
        for a, b in zip(first, got):
            assert torch.equal(a, b)


def test_past_32_bits():
    """A sequence whose rows lie more than 2^32 bytes, and 2^31 values, into every tensor:
    the same bits as from tensors of its own."""
    t, n, h, d = 140000, 300, 128, 128
    full = [torch.zeros(t, h, d, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    lse = torch.zeros(h, t, device="cuda")
    own = [normal((n, h, d), 70 + i) for i in range(4)]
    for a, b in zip(full, own):
        a[t - n:] = b
    q, k, v, do, o, dq, dk, dv = full
    c, c0 = dev([t - n, t]), dev([0, n])
    pk.pact_attention_fwd(q, k, v, c, c, o=o, lse=lse)
    pk.pact_attention_bwd(do, q, k, v, o, lse, c, c, dq=dq, dk=dk, dv=dv)
    pk.pact_check_status()
    wo, wl = pk.pact_attention_fwd(*own[:3], c0, c0)
    want = (wo, *pk.pact_attention_bwd(own[3], *own[:3], wo, wl, c0, c0))
    for a, b in zip(full[4:], want):
        assert torch.equal(a[t - n:], b) and not a[:t - n].any()
    assert torch.equal(lse[:, t - n:], wl) and not lse[:, :t - n].any()


def test_gradients_against_differences():
    """The kernels' gradients against differences of the 64-bit forward: a step along a
    random direction changes <o, do> by the gradient's product with it."""
    lens = [70, 200]
    q, k, v, do, cq, ck = make(lens, lens, 4, 2, 64, 21)
    args = dev(cq), dev(ck)
    o, lse = pk.pact_attention_fwd(q, k, v, *args)
    g = pk.pact_attention_bwd(do, q, k, v, o, lse, *args)
    _, bounds = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, True, 0.125)
    for i in range(3):
        ts = [t.double() for t in (q, k, v)]
        e = torch.randn(ts[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda",
                        dtype=torch.float64)
        h = 1e-4
        up, down = list(ts), list(ts)
        up[i], down[i] = ts[i] + h * e, ts[i] - h * e
        diff = sum(sg * (ref.attention(*x, cq, ck, True, 0.125)[0] * do.double()).sum() for sg, x in
                   ((1.0, up), (-1.0, down))) / (2 * h)
        got = (g[i].double() * e).sum()
        # each value of the gradient errs within its bound (o's own rounding in delta adds
        # U |do| |o| to dS, which a tenth of the bound's first term covers many times over)
        room = ref.T * (bounds[i] * e).pow(2).sum().sqrt() * 2
        assert abs(got - diff) <= room


def test_refusals():
    q, k, v, do, cq, ck = make([20], [20], 4, 2, 64)
    a, b = dev(cq), dev(ck)
    o, lse = pk.pact_attention_fwd(q, k, v, a, b)
    for bad in (lambda: pk.pact_attention_fwd(q.half(), k, v, a, b),
                lambda: pk.pact_attention_fwd(q, k, v[:10], a, b),
                lambda: pk.pact_attention_fwd(q, k, v, a.long(), b),
                lambda: pk.pact_attention_fwd(q, k, v, a, dev([0, 10, 20])),
                lambda: pk.pact_attention_fwd(q, k, v, a[:1], b[:1]),
                lambda: pk.pact_attention_fwd(q, k, v, a, b.cpu()),
                lambda: pk.pact_attention_fwd(q, k, v, a, b, o=o[:10]),
                lambda: pk.pact_attention_fwd(q, k, v, a, b, lse=lse.t()),
                lambda: pk.pact_attention_fwd(q.transpose(1, 2), k, v, a, b),
                lambda: pk.pact_attention_bwd(do, q, k, v, o, lse[:1], a, b),
                lambda: pk.pact_attention_bwd(do, q, k, v, o, lse, a, b, dk=q)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: pk.pact_attention_fwd(q[:, :3], k, v, a, b),
                lambda: pk.pact_attention_fwd(q, k, v, a, b, scale=0.0),
                lambda: pk.pact_attention_fwd(q, k, v, a, b, scale=math.nan),
                lambda: pk.pact_attention_fwd(q, k, v, a, b, scale=-1.0)):
        with pytest.raises(pk.PactError):
            bad()
    with pytest.raises(pk.PactError):
        pk.pact_attention_fwd(*(torch.zeros(4, 1, 144, device="cuda").bfloat16() for _ in range(3)), a, b)


# few tokens over many keys: the keys of a token are shared out over CTAs
PARTS = [
    ([1], [2100], 8, 1, 128),
    ([1], [70001], 4, 2, 16),
    ([2048], [2048], 1, 1, 128),
    ([2500], [2500], 2, 1, 64),
    ([1, 1, 3, 1], [4000, 77, 5000, 1], 6, 2, 96),     # parts without a key
    ([3, 0, 5], [9000, 500, 0], 4, 4, 112),
    ([2200], [2048], 1, 1, 48),                        # rows that see nothing
    ([9], [4096], 5, 1, 80),
    ([2, 2], [2300, 2300], 130, 1, 32),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,hq,hk,d", PARTS, ids=[f"{max(a)}x{max(b)}h{h}-{g}d{d}" for a, b, h, g, d in PARTS])
def test_parts_of_the_keys(lq, lk, hq, hk, d, causal):
    q, k, v, _, cq, ck = make(lq, lk, hq, hk, d, 40)
    assert pk.load_library().pact_attention_fwd_workspace_size(q.shape[0], hq, k.shape[0], hk, d, len(lq)) > 0
    o, lse = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), causal)
    pk.pact_check_status()
    wo, wl, bo, bl = ref.attention(q, k, v, cq, ck, causal, d ** -0.5)
    ref.check(o, wo, bo, "o")
    ref.check(lse, wl, bl, "lse")
    o2, lse2 = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_one_part_without_a_workspace():
    q, k, v, _, cq, ck = make([40], [5000], 4, 2, 64, 45)
    a, b = dev(cq), dev(ck)
    o, lse = torch.empty_like(q), torch.empty(4, 40, device="cuda")
    fields = [pk._HeadsStruct(t.data_ptr(), *t.shape[:2], t.stride(0)) for t in (q, k, v, o)]
    lib = pk.load_library()
    rc = lib.pact_attention_fwd(*fields[:3], 64, a.data_ptr(), b.data_ptr(), 1, 1, 0.125, fields[3], lse.data_ptr(),
                                None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    pk.pact_check_status()
    wo, wl, bo, bl = ref.attention(q, k, v, cq, ck, True, 0.125)
    ref.check(o, wo, bo, "o")
    ref.check(lse, wl, bl, "lse")


def test_parts_leave_other_rows():
    q, k, v, _, _, _ = make([20], [6000], 4, 2, 64, 50)
    o = torch.full_like(q, 7.0)
    lse = torch.full((4, 20), 7.0, device="cuda")
    args = dev([2, 3, 9]), dev([100, 3000, 5990])
    pk.pact_attention_fwd(q, k, v, *args, o=o, lse=lse)
    pk.pact_check_status()
    wo, wl, bo, bl = ref.attention(q, k, v, [2, 3, 9], [100, 3000, 5990], True, 0.125)
    ref.check(o, wo, bo, "o")
    ref.check(lse, wl, bl, "lse")
    for rows in (slice(0, 2), slice(9, 20)):
        assert (o[rows] == 7.0).all() and (lse[:, rows] == 7.0).all()


def test_parts_keep_a_nan_to_its_head_and_sequence():
    lq, lk = [1, 4], [5000, 4700]
    q, k, v, _, cq, ck = make(lq, lk, 4, 2, 64, 60)
    args = dev(cq), dev(ck)
    o, lse = pk.pact_attention_fwd(q, k, v, *args)
    v2, k2 = v.clone(), k.clone()
    v2[4321, 1] = math.nan      # sequence 0, its second key head
    k2[9000, 0, 3] = math.nan   # sequence 1, its first
    o2, lse2 = pk.pact_attention_fwd(q, k2, v2, *args)
    assert torch.isnan(o2[0, 2:]).all() and torch.isnan(o2[1:, :2]).all() and torch.isnan(lse2[:2, 1:]).all()
    assert torch.equal(o2[0, :2], o[0, :2]) and torch.equal(o2[1:, 2:], o[1:, 2:])
    assert torch.equal(lse2[:2, 0], lse[:2, 0]) and torch.equal(lse2[2:], lse[2:])


def test_parts_in_graphs_on_two_streams():
    cases = [make([1], [4000 + 700 * i], 8, 2, 128, 70 + 10 * i) for i in range(2)]
    want, got, graphs, streams = [], [], [], [torch.cuda.Stream() for _ in cases]
    for (q, k, v, _, cq, ck), st in zip(cases, streams):
        a, b = dev(cq), dev(ck)
        want.append(pk.pact_attention_fwd(q, k, v, a, b))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = pk.pact_attention_fwd(q, k, v, a, b)
            for _ in range(5):
                out = pk.pact_attention_fwd(q, k, v, a, b, o=out[0], lse=out[1])
        got.append(out)
        graphs.append((g, a, b))
    for _ in range(3):
        for (g, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    pk.pact_check_status()
    for (o, lse), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


# few tiles: the work of dk and dv (shared heads), or of dq (many keys), is shared out
BWD_PARTS = [
    ([1024], [1024], 16, 2, 64),
    ([700], [700], 8, 1, 128),
    ([900, 1, 0, 1100], [900, 70, 5, 1100], 24, 1, 96),
    ([520, 600], [400, 600], 130, 1, 32),
    ([200], [2304], 4, 4, 128),
    ([3, 0, 70], [9000, 500, 40], 4, 2, 48),
    ([1], [5000], 8, 1, 80),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,hq,hk,d", BWD_PARTS,
                         ids=[f"{max(a)}x{max(b)}h{h}-{g}d{d}" for a, b, h, g, d in BWD_PARTS])
def test_backward_in_parts(lq, lk, hq, hk, d, causal):
    q, k, v, do, cq, ck = make(lq, lk, hq, hk, d, 80)
    size = pk.load_library().pact_attention_bwd_workspace_size(q.shape[0], hq, k.shape[0], hk, d, len(lq))
    assert size > 2 * 4 * q.shape[0] * hq + 256
    o, lse = pk.pact_attention_fwd(q, k, v, dev(cq), dev(ck), causal)
    got = pk.pact_attention_bwd(do, q, k, v, o, lse, dev(cq), dev(ck), causal)
    pk.pact_check_status()
    want, bounds = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, causal, d ** -0.5)
    for g, w, b, name in zip(got, want, bounds, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
    again = pk.pact_attention_bwd(do, q, k, v, o, lse, dev(cq), dev(ck), causal)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("tq,tk,cq,ck,hq,hk", [(1300, 1200, [7, 500, 1200], [0, 493, 1190], 16, 1),
                                               (100, 9000, [7, 20, 90], [3, 4000, 8990], 4, 4)])
def test_backward_in_parts_leaves_other_rows(tq, tk, cq, ck, hq, hk):
    q, k, v, do, _, _ = make([tq], [tk], hq, hk, 64, 90)
    args = dev(cq), dev(ck)
    o, lse = pk.pact_attention_fwd(q, k, v, *args)
    outs = [torch.full_like(x, 7.0) for x in (q, k, v)]
    pk.pact_attention_bwd(do, q, k, v, o, lse, *args, dq=outs[0], dk=outs[1], dv=outs[2])
    pk.pact_check_status()
    want, bounds = ref.attention_bwd(do, q, k, v, o, lse, cq, ck, True, 0.125)
    for g, w, b, c, name in zip(outs, want, bounds, (cq, ck, ck), ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
        assert (g[:c[0]] == 7.0).all() and (g[c[-1]:] == 7.0).all()
