"""The flag that asks for zeros in rows of no sequence: where it is taken and where not (CPU only)."""
import re

import pytest

from hadamard_incoherence_transforms_b200 import _lib, api
from tests.test_kv_host import FAKE, append, attend, kv


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_the_binding_has_the_headers_value():
    text = open(_lib.__file__.replace("hadamard_incoherence_transforms_b200/_lib.py", "include/hit.h")).read()
    assert int(re.search(r"#define HIT_KV_ZERO (\w+)", text).group(1), 0) == api._KV_ZERO


def test_the_flag_goes_with_output_types_only(lib):
    z = api._KV_ZERO
    for dt in (0, 1):
        assert attend(lib, kv(), tokens=0, do=dt | z) == _lib.HIT_OK
        assert lib.rht_kv_read(kv(), FAKE, FAKE, 0, 256, 128, 256, 128, dt | z, None) == _lib.HIT_OK
        assert lib.rht_kv_read(kv(seqs=0), None, None, 4, 256, 128, 256, 128, dt | z, None) == _lib.HIT_OK
        assert attend(lib, kv(), tokens=0, dq=dt | z) == _lib.HIT_EUNSUPPORTED
        assert append(lib, kv(), dtype=dt | z) == _lib.HIT_EUNSUPPORTED
    for bad in (2 | z, 5 | z, 2 * z, 1 | 2 * z, -1):
        assert attend(lib, kv(), tokens=0, do=bad) == _lib.HIT_EUNSUPPORTED
        assert lib.rht_kv_read(kv(), FAKE, FAKE, 0, 256, 128, 256, 128, bad, None) == _lib.HIT_EUNSUPPORTED


def test_a_call_without_sequences_still_checks_its_output(lib):
    z = api._KV_ZERO
    c = kv(seqs=0, cu=0, lens=0)
    assert attend(lib, c, out=None, do=1 | z) == _lib.HIT_EINVAL
    assert attend(lib, c, out=FAKE + 2, do=1 | z) == _lib.HIT_EALIGN
    assert lib.rht_kv_read(c, FAKE + 4, FAKE, 4, 256, 128, 256, 128, 1 | z, None) == _lib.HIT_EALIGN
