"""Refusals of the serving operators at their limits, found before any CUDA
call (CPU only)."""
import pytest

from late_interaction_retrieval_gb300 import binding
from late_interaction_retrieval_gb300 import build as lik_build

N = None


@pytest.fixture(scope="module")
def lib():
    return binding.load(lik_build.build())


def attention(lib, **changed):
    a = dict(dtype=2, rows=3, q_heads=4, heads=2, dim=32, q=(128, 32), pages=4, page_size=16, cols=4, stride=4,
             requests=2, added=2, scale=0.2, out=(128, 32))
    a.update(changed)
    return lib.lik_cache_attention(N, a["dtype"], a["rows"], a["q_heads"], a["dim"], *a["q"], N, N, N, N, a["pages"],
                                   a["heads"], a["page_size"], N, a["cols"], a["stride"], N, N, a["requests"],
                                   a["added"], a["scale"], N, *a["out"], N, N, 0, N)


@pytest.mark.parametrize("out", [(0, 32), (128, 0), (0, 0), (127, 32), (96, 32), (128, 31), (31, 96), (32, 95), (16, 128)])
def test_outputs_whose_rows_overlap(lib, out):
    """Strides under which two (row, head) share an element: whichever was written last would stay."""
    assert attention(lib, out=out) == 1
    assert b"overlap" in lib.lik_last_error_message()


@pytest.mark.parametrize("changed", [dict(out=(128, 32)), dict(out=(129, 32)), dict(out=(32, 96)), dict(out=(40, 200)),
                                     dict(out=(512, 64)), dict(rows=1, out=(0, 32)), dict(rows=1, out=(7, 33)),
                                     dict(q_heads=2, heads=2, out=(64, 32)), dict(q_heads=1, heads=1, out=(32, 0)),
                                     dict(rows=0, out=(0, 0)), dict(q=(0, 0))])
def test_layouts_that_do_not_overlap(lib, changed):
    """Rows or heads first, gaps, a single row or head, and inputs that repeat: no refusal of the layout."""
    attention(lib, **changed)
    assert b"overlap" not in lib.lik_last_error_message()


@pytest.mark.parametrize("cols,page,status", [(2 ** 27 - 1, 16, 2), (2 ** 23 - 1, 256, 2), (2 ** 27 - 255, 16, 2)])
def test_tables_whose_positions_pass_31_bits(lib, cols, page, status):
    """Positions are counted in 32 bits, a tile or a few ahead of the last."""
    assert attention(lib, cols=cols, stride=cols, page_size=page) == status
    assert lib.lik_last_error_message()
    size = binding.ctypes.c_size_t(7)
    assert lib.lik_cache_attention_workspace_bytes(3, 4, 2, 32, 2, page, cols, 2, binding.ctypes.byref(size)) == status
