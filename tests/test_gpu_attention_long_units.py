"""Attention over so many keys that one tile of queries goes through them for seconds: roles
that have nothing to do meanwhile wait for it and do not give up."""
import math

import pytest
import torch

import heads_ref as ref
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu
D = 16
SEQS, SHORT = 700, 16          # one token each; the keys of all sequences but the first
KEYS = 2**30
LONG = KEYS - (SEQS - 1) * SHORT


@pytest.fixture(scope="module")
def keys():
    """Zeros but for the first and the last key of the long sequence."""
    k, v = (torch.zeros(KEYS, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[0, 0, 0] = k[LONG - 1, 0, 1] = 32.0
    v[0, 0, 0], v[LONG - 1, 0, 1] = 2.0, -2.0
    v[LONG:] = 1.0
    yield k, v
    del k, v
    torch.cuda.empty_cache()


def queries(n):
    """Scores of 128 at both keys, 0 (a weight of 2^-185, which vanishes) at the others."""
    q = torch.zeros(n, 1, D, dtype=torch.bfloat16, device="cuda")
    q[:, 0, :2] = 4.0
    return q


def test_one_tile_of_two(keys):
    """Without a workspace a token's keys are one unit, and the CTA's second tile has none."""
    k, v = keys
    q = queries(1)
    o, lse = torch.empty_like(q), torch.empty(1, 1, device="cuda")
    cq = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, LONG], dtype=torch.int32, device="cuda")
    fields = [pk._HeadsStruct(t.data_ptr(), t.shape[0], 1, D) for t in (q, k, v, o)]
    rc = pk.load_library().pact_attention_fwd(*fields[:3], D, cq.data_ptr(), ck.data_ptr(), 1, 1, 1.0, fields[3],
                                              lse.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    pk.pact_check_status()
    # weights of one half each: every number is a whole one
    assert o[0, 0].tolist() == [1.0, -1.0] + [0.0] * 14
    assert abs(lse.item() - (128 + math.log(2))) <= 4 * ref.E * 129


def test_statistics_ahead_of_a_unit(keys):
    """Several tiles for every SM, the first of which is the long one."""
    k, v = keys
    q = queries(SEQS)
    cq = torch.arange(SEQS + 1, dtype=torch.int32, device="cuda")
    ck = torch.tensor([0] + [LONG + SHORT * i for i in range(SEQS)], dtype=torch.int32, device="cuda")
    do = torch.zeros_like(q)
    do[:, 0, :2] = 1.0
    o = torch.ones_like(q)     # of the short sequences, whose scores are all 0
    o[0] = 0.0
    o[0, 0, 0], o[0, 0, 1] = 1.0, -1.0
    lse = torch.full((1, SEQS), math.log(SHORT), device="cuda")
    lse[0, 0] = 128 + math.log(2)
    dq, dk, dv = pk.pact_attention_bwd(do, q, k, v, o, lse, cq, ck, True, 1.0)
    pk.pact_check_status()
    # P is a half at both keys, dP 2 and -2, delta 0: dS 1 and -1 (its error, that of an exponent
    # of 185 in FP32, is far below BF16's)
    assert dq[0, 0].tolist() == [32.0, -32.0] + [0.0] * 14
    assert dk[0, 0].tolist() == [4.0, 4.0] + [0.0] * 14 and dk[LONG - 1, 0].tolist() == [-4.0, -4.0] + [0.0] * 14
    assert dv[0, 0].tolist() == dv[LONG - 1, 0].tolist() == [0.5, 0.5] + [0.0] * 14
    # the short ones: P = 1/16 (BF16's rounding of exp(-lse) at most), dP = delta = 2
    assert ((dv[LONG:, 0, :2].float() - 1 / 16).abs() <= ref.U * (2 + ref.U) / 16).all()
    assert int((dv[LONG:, 0, 2:] != 0).sum()) == 0 and int((dq[1:] != 0).sum()) == 0
    for t in (dk, dv):  # 32 GB each: piece by piece
        assert not any(piece.any() for piece in t[1:LONG - 1].split(2**24))
