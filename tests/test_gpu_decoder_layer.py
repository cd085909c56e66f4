"""A whole decoder layer: every stage of the attention between the projections against the
plain 64-bit forms fed with the GPU's own upstream tensors, the adapters' gradients clipped
together, and a step captured in a graph."""
import numpy as np
import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk
from nvfp4_frozen_projection_gb300 import workloads as wl
from nvfp4_frozen_projection_gb300.stack import DecoderLayer

from stage_checks import check_quant

pytestmark = pytest.mark.gpu
LENS = [100, 1, 219]
CU = [0, 100, 101, 320]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().cuda()


@pytest.fixture(scope="module", params=[False, True], ids=["plain", "norms"])
def layer(request):
    d = wl.layer3b(m=320, hidden=512, kv=128, inter=1024)
    f = 500000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    gammas = [(1.0 + 0.1 * torch.randn(64, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    st = DecoderLayer.from_workload(d, "cuda", 8, 2, f, *(gammas if request.param else (None, None)))
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in LENS]).cuda()
    x, dy = dev(d["x"]), dev(d["dy"])

    def step():
        st.forward(x, cu, pos)
        st.backward(dy, cu, pos)
        return st.adapter_grads(dy)

    step()
    torch.cuda.synchronize()
    pk.pact_check_status()
    return st, f.cuda(), pos, step


def test_stages(layer):
    st, f, pos, _ = layer
    eps = st.eps
    for x, y, gam in ((st.qh, st.qr, st.gamma_q), (st.kh, st.kr, st.gamma_k)):
        want, mag = ref.rope(x, pos, f, False, gam, eps)
        ref.check(y, want, ref.U * (1 + ref.U) * want.abs() + 24 * ref.E * mag, "rotated")
    wo, wl_, bo, bl = ref.attention(st.qr, st.kr, st.vh, CU, CU, True, 0.125)
    ref.check(st.attn, wo, bo, "attention")
    ref.check(st.lse, wl_, bl, "lse")
    check_quant("attnq", st.attnq, st.attn.view(st.m, -1))
    do = st.dattn.view_as(st.attn)
    rot = pk.pact_attention_bwd(do, st.qr, st.kr, st.vh, st.attn, st.lse, *[torch.tensor(
        CU, dtype=torch.int32, device="cuda")] * 2)
    want, bounds = ref.attention_bwd(do, st.qr, st.kr, st.vh, st.attn, st.lse, CU, CU, True, 0.125)
    for g, w, b, name in zip(rot, want, bounds, ("dq", "dk", "dv")):
        ref.check(g, w, b, name)
    assert torch.equal(rot[2], st.dv.view_as(st.vh))
    for dyr, x, got, gam, dg, heads in ((rot[0], st.qh, st.dq, st.gamma_q, st.dgamma_q, 8),
                                        (rot[1], st.kh, st.dk, st.gamma_k, st.dgamma_k, 2)):
        want, wg, mag, magg = ref.rope_bwd(dyr, pos, f, False, x, gam, eps)
        ref.check(got.view_as(x), want, ref.U * (1 + ref.U) * want.abs() + 48 * ref.E * mag, "turned back")
        if gam is not None:
            ref.check(dg, wg, ref.E * (2 * heads + 64 + 2 * 24) * magg, "dgamma")


def test_clipping_all_gradients_together(layer):
    st, _, _, step = layer
    step()
    ts = st.grad_list.tensors
    keep = [t.double().clone() for t in ts]
    norm = float(sum(t.square().sum() for t in keep)) ** 0.5
    # all parameters' gradients: of the fused gate|up B the diagonal blocks
    parts = [t.double() for pair in st.grads.values() for t in pair]
    if st.gamma_q is not None:
        parts += [st.dgamma_q.double(), st.dgamma_k.double()]
    dB = st.grads["gate_up"][1]
    r, w = dB.shape
    off = dB[:r // 2, w // 2:].double().square().sum() + dB[r // 2:, :w // 2].double().square().sum()
    whole = float(sum(t.square().sum() for t in parts) - off) ** 0.5
    assert abs(whole - norm) <= 1e-12 * norm
    got = st.clip_grads(norm / 5)
    assert abs(got.item() - norm) <= 10 * ref.E * norm
    for t, k in zip(ts, keep):
        w = k * ((norm / 5) / (norm + 1e-6))
        ref.check(t, w, 14 * ref.E * w.abs(), "clipped")


def test_a_captured_step(layer):
    st, _, _, step = layer

    def run():
        step()
        return st.clip_grads(0.5)

    norm = run().clone()
    first = [t.clone() for t in (st.out, st.dx, *st.grad_list.tensors)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            held = run()
    for t in (st.out, st.dx, *st.grad_list.tensors):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    pk.pact_check_status()
    assert torch.equal(norm, held)
    for a, b in zip(first, (st.out, st.dx, *st.grad_list.tensors)):
        assert torch.equal(a, b)
