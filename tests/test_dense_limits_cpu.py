"""What the products' and norms' calls refuse and how they end, as far as that goes without a GPU."""
import pytest

from _util import ensure_built


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import sherman_morrison_inverse_gb300 as vla
    return vla.load_library()


def test_the_wait_limit_needs_a_handle(lib):
    assert lib.vla_wait_limit(None, 100) == 1
    assert b"handle" in lib.vla_last_error(None)
