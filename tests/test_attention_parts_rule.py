"""When attention's forward takes a workspace: the binding asks the library from a number of
keys on, below which the library's answer is always zero."""
import pytest
import torch

import nvfp4_frozen_projection_gb300 as pk


@pytest.fixture(scope="module")
def lib():
    from nvfp4_frozen_projection_gb300 import build
    build.build()
    return pk.load_library()


def test_where_the_binding_begins_to_ask(lib):
    size = lib.pact_attention_fwd_workspace_size
    asked = 0
    for n in (1, 2, 3, 7, 33, 1000):
        for hq, hk in ((1, 1), (8, 1), (8, 8), (6, 2), (130, 1)):
            for tq in (1, 2, 5, 100, 1000, 3000):
                for below in (1, 100, 2000):
                    assert size(tq, hq, pk._PARTS_KEYS * n - below, hk, 64, n) == 0
                asked += size(tq, hq, pk._PARTS_KEYS * n, hk, 64, n) > 0
    assert asked > 0  # nor is it a number that no call reaches


@pytest.mark.gpu
@pytest.mark.parametrize("tk,launches", [(pk._PARTS_KEYS - 1, 1), (pk._PARTS_KEYS, 2), (30000, 2)])
def test_the_join_is_launched(tk, launches):
    q, k, v = (torch.randn(t, h, 64, device="cuda").bfloat16() for t, h in ((1, 8), (tk, 2), (tk, 2)))
    a, b = (torch.tensor([0, t], dtype=torch.int32, device="cuda") for t in (1, tk))
    pk.pact_attention_fwd(q, k, v, a, b)
    before = pk.pact_launch_count()
    pk.pact_attention_fwd(q, k, v, a, b)
    assert pk.pact_launch_count() - before == launches
    pk.pact_check_status()
