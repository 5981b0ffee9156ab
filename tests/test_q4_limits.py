"""Limits of the paged 4-bit cache's operators that the host checks (no GPU:
every case is refused before a launch)."""
import ctypes

import pytest

import mtp_speculative_decoding_step_gb300 as m

FAKE = 0x100000  # never dereferenced
BAD = 9


@pytest.fixture(scope="module")
def L():
    from mtp_speculative_decoding_step_gb300 import _build
    _build.build()
    return m.lib()


PLAN = dict(stream=None, rows=4, page=16, max_pages=8, n_pages=32, max_tokens=10, cover=FAKE, keep=2 * FAKE, new=3 * FAKE,
            table=4 * FAKE, free=5 * FAKE, cover_out=6 * FAKE, start=7 * FAKE, slot=8 * FAKE, pos=9 * FAKE, status=None)
WRITTEN = dict(table=4 * 8, free=32, cover_out=4, start=5, slot=10, pos=10)  # int32 elements


@pytest.mark.parametrize("length", ["cover", "keep", "new"])
@pytest.mark.parametrize("out", list(WRITTEN))
def test_plan_refuses_outputs_over_its_lengths(L, length, out):
    """Blocks still read the lengths while others write: keep := keep + new in place would give a page to two rows."""
    for at in (PLAN[length], PLAN[length] + 4 * (PLAN["rows"] - 1), PLAN[length] - 4 * (WRITTEN[out] - 1)):
        assert L.kv_page_plan(*{**PLAN, out: at}.values()) == BAD


@pytest.mark.parametrize("name,val", [
    ("rows", 0), ("rows", 4097), ("page", 0), ("page", 24), ("max_pages", 0), ("n_pages", 0), ("max_tokens", -1),
    *((name, None) for name in ("cover", "keep", "new", "table", "free", "cover_out", "start", "slot", "pos")),
    ("max_pages", 1 << 29), ("n_pages", 1 << 27), ("max_pages", 1 << 27)])
def test_plan_refuses_each_bad_argument_among_apart_arrays(L, name, val):
    assert L.kv_page_plan(*{**PLAN, name: val}.values()) == BAD
