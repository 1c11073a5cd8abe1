"""Arguments of the rotated key/value cache's calls at the ends of their ranges."""
import pytest
import torch

import hadamard_incoherence_transforms_b200 as hit
from tests._kv import Cache, heads
from tests.test_gpu_kv import cu_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 63, 2 ** 64 + 5, 2 ** 31, 2 ** 32 + 1])
@pytest.mark.parametrize("d,g,new", [(64, 2, [9, 3]), (128, 1, [200, 90]), (256, 2, [70, 40])])
def test_windows_longer_than_any_sequence(window, d, g, new):
    """See everything, also where part of a sequence's tokens lies before its start."""
    c = Cache(111, [max(1, new[0] // 3), 150], 1, d, 4, 16).fill()
    q, _ = heads(c.r, sum(new), g, d, torch.bfloat16)
    args = (q, *c.on(), torch.from_numpy(cu_of(new)).cuda())
    want = hit.rht_kv_attention(*args, **c.signs())
    got = hit.rht_kv_attention(*args, **c.signs(), window=window)
    assert torch.equal(got, want) and (want[:new[0] - new[0] // 3] == 0).all() and (want[-1] != 0).any()


@pytest.mark.parametrize("max_new", [2 ** 31, 2 ** 63 - 1, 2 ** 63, 2 ** 64])
def test_bounds_of_new_tokens_above_all(max_new):
    c = Cache(113, [90, 150], 1, 64, 4, 16).fill()
    q, _ = heads(c.r, 43, 2, 64, torch.bfloat16)
    args = (q, *c.on(), torch.from_numpy(cu_of([3, 40])).cuda())
    assert torch.equal(hit.rht_kv_attention(*args, **c.signs(), max_new=max_new), hit.rht_kv_attention(*args, **c.signs()))


@pytest.mark.parametrize("kw", [{"window": -1}, {"window": -2 ** 64 + 5}, {"max_new": 0}, {"max_new": -2 ** 64 + 1},
                                {"window": 5, "causal": False}])
def test_refused(kw):
    c = Cache(115, [90], 1, 64, 4, 16).fill()
    q, _ = heads(c.r, 2, 2, 64, torch.bfloat16)
    with pytest.raises(hit.HitError):
        hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu_of([2])).cuda(), **c.signs(), **kw)
