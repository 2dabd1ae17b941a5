"""The sizes that the GPU tests run in the name of a form of the 4-bit product do take that form."""
import pytest

from linear_forms import NAMES, PAIR, ROWS, SINGLE, SIZES, WIDE


@pytest.fixture(scope="module")
def lib():
    import torch  # noqa: F401  (loads the CUDA runtime the library links against)
    from dynamic_column_sparse_b200 import build, chipmunk
    build.build()
    return chipmunk.load_library()


@pytest.mark.parametrize("form", SIZES, ids=NAMES.get)
def test_sizes_take_the_form_they_stand_for(lib, form):
    for T, N, K in SIZES[form]:
        assert lib.chipmunk_selftest_linear_fp4_form(T, N, K, 0) == form, (T, N, K)
        # quantised x changes nothing but that no form quantises it
        quantised = lib.chipmunk_selftest_linear_fp4_form(T, N, K, 1)
        assert quantised == form if form != ROWS else quantised in (SINGLE, PAIR, WIDE)


def test_unsupported_sizes_have_no_form(lib):
    f = lib.chipmunk_selftest_linear_fp4_form
    assert f(1, 8, 32, 0) == ROWS and f(9, 8, 32, 0) == SINGLE
    for T, N, K in [(0, 8, 32), (1, 0, 32), (1, 12, 32), (1, 8, 48), (1, 8, 0), (1, (1 << 20) + 8, 32), (1, 8, 1 << 17),
                    (1 << 30, 1 << 20, 32), ((1 << 30) + 1, 8, 32)]:
        assert f(T, N, K, 0) == -1 and f(T, N, K, 1) == -1, (T, N, K)
