"""Scale arrays of the paged append: the units of a page's keys and values write them at the
same time, so they must not overlap (no GPU; the check comes before any launch)."""

import pytest

from tests.test_paged_args import FAKE, append, attend, lib  # noqa: F401 (lib is a fixture)

BYTES = 4 * 2 * 4  # [4 pages, 2 heads] fp32


@pytest.mark.parametrize("off", [0, 4, BYTES - 4, -4, 4 - BYTES])
def test_append_refuses_overlapping_scales(lib, off):  # noqa: F811
    assert append(lib, k_scales=FAKE, v_scales=FAKE + off) == -1
    assert b"k_scales and v_scales overlap" in lib.sba_last_error()


@pytest.mark.parametrize("off", [BYTES, -BYTES])
def test_neighbouring_scales_pass_that_check(lib, off):  # noqa: F811
    # refused for its head count, which is looked at before the scales, and never launched
    assert append(lib, k_scales=FAKE, v_scales=FAKE + off, Hq=1 << 17, qs=1 << 24, qos=1 << 24) == -2
    assert b"65535" in lib.sba_last_error()


def test_reading_calls_may_share_scales(lib):  # noqa: F811
    assert attend(lib, k_scales=FAKE, v_scales=FAKE, ws=None) == -1
    assert b"workspace" in lib.sba_last_error()
