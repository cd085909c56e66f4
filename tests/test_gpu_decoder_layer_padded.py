"""A decoder layer over a padded batch: rows that belong to no sequence add nothing to any
gradient, and nothing of an earlier batch, or of what the buffers held, comes through."""
import math

import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk
from nvfp4_frozen_projection_gb300 import workloads as wl
from nvfp4_frozen_projection_gb300.stack import DecoderLayer

from stage_checks import check_quant
from test_gpu_decoder_layer import dev

pytestmark = pytest.mark.gpu
M = 320
FULL, PART = [0, 100, 101, 320], [7, 90, 90, 250]   # rows in front, behind, and a sequence without any


@pytest.fixture(scope="module", params=[(False, True), (True, True), (True, False)], ids=["plain", "norms", "one stream"])
def layer(request):
    norms, concurrent = request.param
    d = wl.layer3b(m=M, hidden=512, kv=128, inter=1024)
    f = 500000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    gammas = [(1.0 + 0.1 * torch.randn(64, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    st = DecoderLayer.from_workload(d, "cuda", 8, 2, f, *(gammas if norms else (None, None)))
    st.concurrent = concurrent
    pos = torch.arange(M, dtype=torch.int32, device="cuda") % 97
    x, dy = dev(d["x"]), dev(d["dy"])
    dy[:PART[0]] = 0
    dy[PART[-1]:] = 0

    def step(cu):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st.forward(x, cu, pos)
        st.backward(dy, cu, pos)
        st.adapter_grads(dy)
        torch.cuda.synchronize()
        pk.pact_check_status()
        return [t.clone() for t in (st.out, st.dx, st.attn, st.dq, st.dk, st.dv, *st.grad_list.tensors)]

    return st, f.cuda(), pos, step


def pads(t):
    return torch.cat((t[:PART[0]], t[PART[-1]:]))


@pytest.mark.parametrize("before", [0.0, 1e4, math.nan])
def test_nothing_comes_through(layer, before):
    st, _, _, step = layer
    want = step(PART)
    for t in (st.attn, st.dq, st.dk, st.dv, st.lse, st.qr, st.kr):
        t.fill_(before)
    for a, b in zip(step(PART), want):
        assert torch.equal(a, b)
    step(FULL)
    for a, b in zip(step(PART), want):
        assert torch.equal(a, b)


def test_rows_of_no_sequence(layer):
    st, f, pos, step = layer
    step(FULL)
    step(PART)
    for t in (st.attn, st.dq, st.dk, st.dv, st.dattn):
        assert int((pads(t) != 0).sum()) == 0
    assert torch.isfinite(st.out).all() and torch.isfinite(st.dx).all()
    wo, wl_, bo, bl = ref.attention(st.qr, st.kr, st.vh, PART, PART, True, 0.125)
    ref.check(st.attn, wo, bo, "attention")
    check_quant("attnq", st.attnq, st.attn.view(M, -1))
    if st.gamma_q is None:
        return
    # dgamma over the rows of the sequences alone
    do = st.dattn.view_as(st.attn)
    cu = torch.tensor(PART, dtype=torch.int32, device="cuda")
    out = [torch.zeros_like(t) for t in (st.qr, st.kr, st.vh)]
    pk.pact_attention_bwd(do, st.qr, st.kr, st.vh, st.attn, st.lse, cu, cu, dq=out[0], dk=out[1], dv=out[2])
    rows = slice(PART[0], PART[-1])
    for dyr, x, gam, dg, heads in ((out[0], st.qh, st.gamma_q, st.dgamma_q, 8), (out[1], st.kh, st.gamma_k, st.dgamma_k, 2)):
        _, wg, _, magg = ref.rope_bwd(dyr[rows], pos[rows], f, False, x[rows], gam, st.eps)
        ref.check(dg, wg, ref.E * (2 * heads + 64 + 2 * 24) * magg, "dgamma")
