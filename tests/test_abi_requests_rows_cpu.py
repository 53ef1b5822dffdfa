"""Pitches of a single row in the per-request entry points, no GPU needed: a
lone row has no next one, so in place means the same address whatever the two
pitches say.  (With the device overridden to another one, ARCH is what comes
after all argument checks.)"""
import ctypes

import pytest

from test_abi_requests_cpu import BASE, FAKE, G, L, OUT, Y, adapters, apply, lib, logits, rules  # noqa: F401

ARCH, OVERLAP = -5, -7


@pytest.fixture
def other_device(lib):  # noqa: F811
    lib.moe_q4_test_override_device(1, 9, 0)
    yield
    lib.moe_q4_test_override_device(0, 0, 0)


def test_a_lone_row_in_place_at_any_pitches(lib, other_device):  # noqa: F811
    for ldb, ldy in ((1000, 1000), (1000, 1001), (4000, 1000), (1 << 32, 1000)):
        assert apply(lib, adapters(), T=1, base=Y, ldb=ldb, y=Y, ldy=ldy) == ARCH
        assert logits(lib, rules(n_masks=3), T=1, l=L, ld=ldb, out=L, ldo=ldy) == ARCH


@pytest.mark.parametrize("T", [1, 2])
def test_what_is_not_in_place_still_may_not_overlap(lib, other_device, T):  # noqa: F811
    assert apply(lib, adapters(), T=T, base=Y, y=Y + 4) == OVERLAP
    assert apply(lib, adapters(), T=T, base=Y + 4 * 999, y=Y) == OVERLAP
    assert logits(lib, rules(), T=T, l=L, out=L + 4) == OVERLAP
    if T == 2:
        assert apply(lib, adapters(), T=T, base=Y, ldb=1001, y=Y) == OVERLAP
        assert logits(lib, rules(), T=T, l=L, ld=1001, out=L) == OVERLAP
