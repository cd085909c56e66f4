"""How the FP8 product chooses among its kernels, without a GPU."""
import pytest

import fp8_paths
import nvfp4_frozen_projection_gb300 as pk


@pytest.fixture(scope="module", autouse=True)
def lib():
    from nvfp4_frozen_projection_gb300 import build
    build.build()
    return pk.load_library()


def test_the_gpu_tests_take_every_way():
    got = {fp8_paths.instance(*s) for s in fp8_paths.SHAPES}
    assert got == fp8_paths.ALL, (sorted(fp8_paths.ALL - got), sorted(got - fp8_paths.ALL))


def test_plan_refusals():
    for rows, n, k in ((0, 64, 64), (4, 24, 64), (4, 64, 8), (2**30 + 1, 64, 64), (2**30, 2**17, 64)):
        with pytest.raises(pk.PactError) as e:
            pk.pact_test_fp8_plan(rows, n, k)
        assert e.value.code == 2
    with pytest.raises(pk.PactError) as e:
        pk.pact_test_fp8_plan(4, 64, 64, sms=1)
    assert e.value.code == 1


@pytest.mark.parametrize("rows,n,k", [(1, 16, 16), (1, 2**24, 16), (1, 16, 2**24), (2**30, 16, 16),
                                      (1024, 2**24, 2**24), (2**30, 16256, 2**24)])
def test_plan_of_the_largest_sizes(rows, n, k):
    """A grid of every way stays within its limits."""
    way, share, whole = pk.pact_test_fp8_plan(rows, n, k)
    if way == "few":
        assert rows <= 1024 and share in (4, 8, 16)
    tiles = -(-rows // 256) * -(-n // 256)
    assert way != "pairs" or 0 <= whole < tiles
    assert way != "shared" or 2 <= share <= 4
