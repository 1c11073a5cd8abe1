"""The rotated key/value cache's entry points refuse bad arguments on the host, before any CUDA call (CPU only)."""
import ctypes

import pytest
import torch

import hadamard_incoherence_transforms_b200 as hit
from hadamard_incoherence_transforms_b200 import _lib, api

FAKE = 0x10000  # never dereferenced: checks fail first


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


FIELDS = ["k_codes", "k_scales", "v_codes", "v_scales", "page_table", "lens", "cu", "k_signs", "v_signs", "inv_freq",
          "positions", "rope_axis", "pages", "page_size", "ld_table", "ld_positions", "kv_heads", "head_dim", "bits", "seqs",
          "max_pages", "n_freq", "rope_axes", "interleaved"]


def kv(**change):
    v = dict.fromkeys(FIELDS[:9], FAKE) | dict.fromkeys(FIELDS[9:12], 0)
    v |= {"pages": 8, "page_size": 16, "ld_table": 4, "ld_positions": 0, "kv_heads": 2, "head_dim": 128, "bits": 4,
          "seqs": 2, "max_pages": 4, "n_freq": 0, "rope_axes": 1, "interleaved": 0}
    v |= change
    return api._KV.pack(*(v[f] for f in FIELDS))


def append(lib, c, k=FAKE, v=FAKE, tokens=4, ts=256, hs=128, dtype=1):
    return lib.rht_kv_append(c, k, v, tokens, ts, hs, ts, hs, dtype, None)


def attend(lib, c, q=FAKE, out=FAKE, tokens=4, heads=8, ts=1024, hs=128, dq=1, do=1, scale=0.1, causal=1, window=0,
           max_new=1, ws=FAKE, nws=1 << 40):
    return lib.rht_kv_attention(c, q, out, tokens, heads, ts, hs, ts, hs, dq, do, ctypes.c_float(scale), causal, window,
                                max_new, ws, nws, None)


def test_struct_matches_the_header():
    assert api._KV.size == 12 * 8 + 4 * 8 + 8 * 4
    text = open(_lib.__file__.replace("hadamard_incoherence_transforms_b200/_lib.py", "include/hit.h")).read()
    body = text[text.index("typedef struct hit_kv {"):text.index("} hit_kv;")]
    names = [line.split()[-1].strip("*;") for line in body.splitlines()[1:] if line.strip()]
    assert names == FIELDS


BAD = [
    ({"head_dim": 96}, _lib.HIT_EUNSUPPORTED),
    ({"head_dim": 32}, _lib.HIT_EUNSUPPORTED),
    ({"bits": 3}, _lib.HIT_EUNSUPPORTED),
    ({"bits": 16}, _lib.HIT_EUNSUPPORTED),
    ({"kv_heads": 0}, _lib.HIT_EINVAL),
    ({"page_size": 24}, _lib.HIT_EUNSUPPORTED),
    ({"page_size": 0}, _lib.HIT_EUNSUPPORTED),
    ({"page_size": 1 << 17}, _lib.HIT_EUNSUPPORTED),
    ({"pages": -1}, _lib.HIT_EINVAL),
    ({"pages": 1 << 31}, _lib.HIT_EINVAL),
    ({"seqs": -1}, _lib.HIT_EINVAL),
    ({"max_pages": -1}, _lib.HIT_EINVAL),
    ({"ld_table": 3}, _lib.HIT_EINVAL),
    ({"cu": 0}, _lib.HIT_EINVAL),
    ({"lens": 0}, _lib.HIT_EINVAL),
    ({"page_table": 0}, _lib.HIT_EINVAL),
    ({"v_scales": 0}, _lib.HIT_EINVAL),
    ({"k_codes": FAKE + 8}, _lib.HIT_EALIGN),
    ({"k_scales": FAKE + 4}, _lib.HIT_EALIGN),
    ({"lens": FAKE + 2}, _lib.HIT_EALIGN),
]
BAD_ROPE = [
    ({"inv_freq": FAKE, "n_freq": 65}, _lib.HIT_EINVAL),
    ({"inv_freq": FAKE, "n_freq": -8}, _lib.HIT_EINVAL),
    ({"inv_freq": FAKE, "n_freq": 20}, _lib.HIT_EUNSUPPORTED),
    ({"inv_freq": FAKE, "n_freq": 18, "interleaved": 1}, _lib.HIT_EUNSUPPORTED),
    ({"inv_freq": FAKE, "n_freq": 64, "positions": FAKE, "ld_positions": 3}, _lib.HIT_EINVAL),
    ({"inv_freq": FAKE, "n_freq": 64, "positions": FAKE, "ld_positions": 4, "rope_axes": 3}, _lib.HIT_EINVAL),
    ({"inv_freq": FAKE, "n_freq": 64, "positions": FAKE, "ld_positions": 4, "rope_axes": 0}, _lib.HIT_EINVAL),
    ({"inv_freq": FAKE + 1, "n_freq": 64}, _lib.HIT_EALIGN),
]


@pytest.mark.parametrize("change,status", BAD)
def test_bad_caches(lib, change, status):
    c = kv(**change)
    assert append(lib, c) == status
    assert attend(lib, c) == status
    assert lib.rht_kv_read(c, FAKE, FAKE, 4, 256, 128, 256, 128, 1, None) == status
    assert lib.hit_last_error()


@pytest.mark.parametrize("change,status", BAD_ROPE)
def test_bad_rotary_arguments(lib, change, status):
    assert append(lib, kv(**change)) == status
    assert attend(lib, kv(**change)) == status


def test_bad_operands(lib):
    c = kv()
    assert append(lib, None) == _lib.HIT_EINVAL
    assert append(lib, c, dtype=2) == _lib.HIT_EUNSUPPORTED
    assert append(lib, c, k=None) == _lib.HIT_EINVAL
    assert append(lib, c, v=FAKE + 8) == _lib.HIT_EALIGN
    assert append(lib, c, ts=260) == _lib.HIT_EALIGN
    assert append(lib, c, hs=-128) == _lib.HIT_EINVAL
    assert append(lib, c, tokens=-1) == _lib.HIT_EINVAL
    assert append(lib, c, tokens=1 << 31) == _lib.HIT_EINVAL
    assert lib.rht_kv_read(c, FAKE + 4, FAKE, 4, 256, 128, 256, 128, 0, None) == _lib.HIT_EALIGN
    assert lib.rht_kv_read(c, FAKE, FAKE, 4, 254, 128, 256, 128, 0, None) == _lib.HIT_EALIGN
    assert lib.rht_kv_read(c, FAKE, FAKE, 4, 256, 128, 256, 128, 5, None) == _lib.HIT_EUNSUPPORTED
    assert attend(lib, c, heads=7) == _lib.HIT_EINVAL
    assert attend(lib, c, heads=0) == _lib.HIT_EINVAL
    assert attend(lib, c, dq=3) == _lib.HIT_EUNSUPPORTED
    assert attend(lib, c, scale=float("nan")) == _lib.HIT_EINVAL
    assert attend(lib, c, scale=float("inf")) == _lib.HIT_EINVAL
    assert attend(lib, c, window=-1) == _lib.HIT_EINVAL
    assert attend(lib, c, causal=0, window=5) == _lib.HIT_EINVAL
    assert attend(lib, c, max_new=0) == _lib.HIT_EINVAL
    assert attend(lib, c, q=None) == _lib.HIT_EINVAL
    assert attend(lib, c, out=FAKE + 2) == _lib.HIT_EALIGN
    assert attend(lib, c, tokens=(1 << 31) - 1) == _lib.HIT_EUNSUPPORTED


def test_nothing_to_do_succeeds_without_a_device(lib):
    assert append(lib, kv(), tokens=0) == _lib.HIT_OK
    assert append(lib, kv(seqs=0)) == _lib.HIT_OK
    assert append(lib, kv(pages=0)) == _lib.HIT_OK
    assert attend(lib, kv(), tokens=0) == _lib.HIT_OK
    assert attend(lib, kv(seqs=0, cu=0, lens=0)) == _lib.HIT_OK
    assert lib.rht_kv_read(kv(), None, None, 4, 256, 128, 256, 128, 1, None) == _lib.HIT_OK
    assert lib.rht_kv_read(kv(), FAKE, FAKE, 0, 256, 128, 256, 128, 1, None) == _lib.HIT_OK


def tensors(d=64, bits=4, hk=2, page=16, seqs=2):
    codes = torch.zeros(4, hk, page, d * bits // 8, dtype=torch.uint8)
    return [codes, torch.zeros(4, hk, page), codes.clone(), torch.zeros(4, hk, page),
            torch.zeros(seqs, 3, dtype=torch.int32), torch.zeros(seqs, dtype=torch.int32),
            torch.zeros(seqs + 1, dtype=torch.int32)]


def test_binding_refuses_tensors_that_do_not_fit():
    q = torch.zeros(4, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        hit.rht_kv_attention(q, *tensors())
    with pytest.raises(ValueError, match="CUDA"):
        hit.rht_kv_append(q[:, :2], q[:, :2], *tensors())
    with pytest.raises(ValueError, match="CUDA"):
        hit.rht_kv_read(*tensors(), rows=4, head_dim=64)
    dev = -1  # what tensors on the CPU answer

    def pack(change=None, at=None, **kw):
        t = tensors()
        if at is not None:
            t[at] = change(t[at])
        return api._kv(64, dev, 4, *t, kw.pop("k_signs", None), kw.pop("v_signs", None), **kw)

    assert len(pack()) == api._KV.size
    for at, change in [(0, lambda x: x.int()), (0, lambda x: x[0]), (1, lambda x: x.double()), (1, lambda x: x[:2]),
                       (2, lambda x: x[:3]), (3, lambda x: x[..., :5]), (4, lambda x: x.long()), (4, lambda x: x[0]),
                       (4, lambda x: x[:, ::2]), (5, lambda x: x.long()), (5, lambda x: x[:1]), (6, lambda x: x[:2]),
                       (0, lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)),
                       (0, lambda x: x[..., :31])]:
        with pytest.raises(ValueError):
            pack(change, at)
    f, p = torch.ones(32), torch.zeros(3, 4, dtype=torch.int32)
    ax = torch.zeros(32, dtype=torch.int8)
    assert pack(inv_freq=f, positions=p, rope_axis=ax)
    for kw in [{"inv_freq": f.double()}, {"inv_freq": f, "positions": p}, {"positions": p[0]}, {"rope_axis": ax},
               {"inv_freq": f, "rope_axis": ax}, {"inv_freq": f, "positions": p[:, :3], "rope_axis": ax},
               {"inv_freq": f, "positions": p.long(), "rope_axis": ax}, {"inv_freq": f, "positions": p, "rope_axis": ax[:9]},
               {"k_signs": torch.ones(63, dtype=torch.int8)}, {"v_signs": torch.ones(64)}]:
        with pytest.raises(ValueError):
            pack(**kw)


def test_cache_shapes():
    assert hit.kv_cache_shapes(10, 16, 8, 128, 4) == ((10, 8, 16, 64), (10, 8, 16))
    assert hit.kv_cache_shapes(10, 16, 8, 128, 8) == ((10, 8, 16, 128), (10, 8, 16))


def test_workspace_sizes_and_refusals(lib):
    """Small calls need the parts of two tiles for each block; prompts the queries and larger tiles too."""
    size = lib.rht_kv_workspace_bytes
    assert 0 < size(4, 8, 2, 128, 1) == size(1 << 20, 8, 2, 128, 1)
    assert size(4096, 8, 2, 128, 4096) >= 4096 * 8 * (128 * 2 + 4)
    assert size(4096, 8, 2, 256, 4096) >= 4096 * 8 * (256 * 2 + 4)
    assert size(10, 8, 2, 64, 1 << 40) == size(10, 8, 2, 64, 10)  # no more new tokens than tokens
    for bad in ((0, 8, 2, 128, 1), (4, 7, 2, 128, 1), (4, 8, 0, 128, 1), (4, 8, 2, 96, 1), (4, 8, 2, 128, 0)):
        assert size(*bad) == 0
    for tokens, max_new in ((4, 1), (4096, 4096)):
        need = size(tokens, 8, 2, 128, max_new)
        for kw in ({"ws": None}, {"nws": need - 1}, {"nws": 0}):
            assert attend(lib, kv(), tokens=tokens, max_new=max_new, **kw) == _lib.HIT_EWORKSPACE
        assert attend(lib, kv(), tokens=tokens, max_new=max_new, ws=FAKE + 4, nws=need) == _lib.HIT_EALIGN
