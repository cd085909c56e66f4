"""What no result of the FP8 kernels shows, read from their source: the scope of waits in a
pair, and the debug build's checks."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nvfp4_frozen_projection_gb300", "csrc")


def _code(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))


def _calls(src, name):
    """The first argument and the template arguments of each call of `name`."""
    return [(m.group(2).strip(), m.group(1)) for m in
            re.finditer(r"\b%s(<\w+>)?\(([^,()]*)" % name, src)]


@pytest.mark.parametrize("barrier", ["full0", "empty0", "accf0", "acce0"])
def test_waits_on_barriers_of_a_pair_have_cluster_scope(barrier):
    """In a pair the other CTA's copies, commits and releases arrive on these barriers, so
    every wait on them is wait_x, wait_x_for, wait_tmem or mbar_test_two<PAIR>: cluster scope
    there, CTA scope in a kernel without a pair.  Those of accumulators are relaxed, and a
    tcgen05 fence follows each."""
    src = _code("fp8_gemm.cu")
    src = src[src.index("k_fp8_gemm("):]
    tmem = barrier in ("accf0", "acce0")
    waits = [c for c, _ in (_calls(src, "wait_tmem") if tmem else
                            _calls(src, "wait_x") + _calls(src, "wait_x_for"))]
    tests = _calls(src, "mbar_test_two")
    assert any(c.startswith(barrier) for c in waits)
    assert not [c for c, _ in _calls(src, "mbar_wait") if c.startswith(barrier)]
    assert tests and all(t == "<PAIR>" for _, t in tests)
    assert re.search(r"return PAIR \? mbar_wait_cluster\(bar, par, ns, flag\)", src)
    assert re.search(r"return PAIR \? mbar_wait_cluster<true>\(bar, par, kFp8WaitNs", src)
    # the fence: before the next MMA, and before the next TMEM load
    for wait, use in (("!wait_tmem(acce0", "mma_f8<PAIR>("), ("if (!(ok = wait_block()))", "tmem_ld16(")):
        after = src[src.index(wait):]
        assert "tc_fence_after();" in after[:after.index(use)]


def test_cluster_waits_acquire_at_cluster_scope():
    src = _code("tcgen05.cuh")
    for name in ("mbar_try_wait_cluster", "mbar_test_two"):
        body = src[src.index(" %s(" % name):]
        body = body[:body.index("\n}")]
        for order in ("acquire", "relaxed"):
            wait = r"mbarrier\.(?:try|test)_wait\.parity\.%s\.cluster" % order
            assert len(re.findall(wait, body)) == 1


@pytest.mark.parametrize("name", ["fp8_quant.cu", "fp8_norm.cu", "fp8_gemm.cu"])
def test_stores_to_global_memory_are_checked_in_the_debug_build(name):
    """Each store at an address computed by hand is under PACT_IN, in its own statement or
    the lines just before it."""
    lines = [ln for ln in _code(name).split("\n") if ln.strip()]
    store = re.compile(r"(\*reinterpret_cast<\w+\*>\((q|h_out|dh|p|p\.out|out) \+.*|"
                       r"\b(s|rstd_out|dgamma|out)\[.*\]) =[^=]?")
    found = [i for i, ln in enumerate(lines) if store.search(ln)]
    assert found
    for i in found:
        assert any("PACT_IN(" in ln for ln in lines[max(0, i - 7):i + 1]), lines[i]
