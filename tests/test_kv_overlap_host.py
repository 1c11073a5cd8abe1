"""Outputs of the rotated key/value cache's calls whose rows share elements are refused: which value they would hold
depends on the order of the blocks (CPU only; nothing that is accepted here reaches a launch)."""
import itertools

import pytest

from hadamard_incoherence_transforms_b200 import _lib
from tests.test_kv_host import FAKE, attend, kv


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def shares(tokens, heads, d, ts, hs):
    seen = set()
    for t, h in itertools.product(range(tokens), range(heads)):
        row = set(range(t * ts + h * hs, t * ts + h * hs + d))
        if seen & row:
            return True
        seen |= row
    return False


STRIDES = [0, 8, 64, 120, 128, 136, 192, 256, 384, 512, 640, 768, 1024, 1152]


@pytest.mark.parametrize("tokens,heads", [(1, 2), (1, 4), (2, 2), (3, 4), (5, 2), (2, 8), (7, 6)])
def test_every_layout(lib, tokens, heads):
    """Layouts without shared elements come as far as the missing workspace, the others no further than the check."""
    both = set()
    for ts, hs in itertools.product(STRIDES, STRIDES):
        status = attend(lib, kv(), tokens=tokens, heads=heads, ts=ts, hs=hs, ws=None, nws=0)
        want = _lib.HIT_EINVAL if shares(tokens, heads, 128, ts, hs) else _lib.HIT_EWORKSPACE
        assert status == want, (ts, hs)
        both.add(want)
        if want == _lib.HIT_EINVAL:
            assert b"overlap" in lib.hit_last_error()
    assert len(both) == 2


def test_one_row_may_have_any_stride(lib):
    c = kv(kv_heads=1)
    assert attend(lib, c, tokens=1, heads=1, ts=0, hs=0, ws=None, nws=0) == _lib.HIT_EWORKSPACE


def test_read(lib):
    def read(ts, hs, vts, vhs):
        return lib.rht_kv_read(kv(), FAKE, FAKE, 4, ts, hs, vts, vhs, 1, None)

    assert read(0, 128, 256, 128) == _lib.HIT_EINVAL and b"of k" in lib.hit_last_error()
    assert read(256, 128, 256, 0) == _lib.HIT_EINVAL and b"of v" in lib.hit_last_error()
    assert read(256, 128, 128, 256) == _lib.HIT_EINVAL


def test_inputs_may_be_broadcast(lib):
    """Keys, values and queries are only read: one head for all is taken as far as the next check."""
    assert lib.rht_kv_append(kv(), FAKE, FAKE + 8, 4, 0, 0, 256, 128, 1, None) == _lib.HIT_EALIGN  # of v
