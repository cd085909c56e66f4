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


# Products of few tokens whose ways differ by 4 % or more on a GB300, weights out of HBM (us):
# the way that is faster, and both times.
MEASURED = [
    (1, 8192, 8192, "few", 13.9, 17.3), (1, 8192, 16384, "few", 24.8, 27.6),
    (1, 16384, 16384, "few", 46.4, 48.8), (1, 28672, 8192, "few", 37.9, 45.0),
    (1, 14336, 14336, "tiles", 37.6, 39.3), (1, 14336, 4096, "few", 12.9, 14.2),
    (1, 32000, 4096, "few", 24.2, 25.9), (1, 5120, 13824, "few", 17.2, 18.7),
    (1, 10240, 5120, "few", 13.6, 14.7), (1, 131072, 512, "tiles", 16.4, 20.2),
    (8, 28672, 8192, "few", 39.5, 44.8), (8, 8192, 16384, "few", 25.8, 27.9),
    (8, 12288, 12288, "tiles", 30.9, 37.1), (8, 14336, 14336, "tiles", 37.8, 43.1),
    (8, 10240, 8192, "tiles", 20.6, 22.8), (8, 10240, 5120, "tiles", 14.7, 15.5),
    (8, 5120, 13824, "shared", 18.7, 20.0), (8, 8192, 8192, "few", 14.0, 17.4),
]


@pytest.mark.parametrize("rows,n,k,way,us,other", MEASURED)
def test_the_faster_way_is_taken_for_few_tokens(rows, n, k, way, us, other):
    assert us < other and pk.pact_test_fp8_plan(rows, n, k)[0] == way
