"""Padded calls of the rotated key/value cache: rows of tokens that belong to no sequence are zero where the binding makes
the output, whatever its memory held, and as they were where the caller gives it."""
import numpy as np
import pytest
import torch

import hadamard_incoherence_transforms_b200 as hit
from tests._kv import Cache, heads
from tests.test_gpu_kv import DT, cu_of

pytestmark = pytest.mark.gpu


def soil(shape, dtype):
    """Leaves memory of the results' size full of NaN for the allocator to hand out again."""
    x = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("d,bits", [(64, 4), (128, 8), (256, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,first,behind", [([1, 2], 0, 5), ([1, 2], 3, 0), ([90, 3], 70, 300), ([0, 0], 4, 9)])
def test_rows_of_no_sequence_are_zero(d, bits, dtype, new, first, behind):
    c = Cache(101, [120, 40], 2, d, bits, 16).fill()
    cu = cu_of(new, first)
    n = int(cu[-1]) + behind
    own = np.zeros(n, dtype=bool)
    own[first:int(cu[-1])] = True
    q, _ = heads(c.r, n, 6, d, DT[dtype])
    t, cud, signs = c.on(), torch.from_numpy(cu).cuda(), c.signs()
    given = torch.full((n, 6, d), 5.0, device="cuda", dtype=DT[dtype])
    hit.rht_kv_attention(q, *t, cud, **signs, out=given)
    assert (given.cpu()[torch.from_numpy(~own)] == 5.0).all()
    for max_new in (None, max(1, *new)):
        soil((n, 6, d), DT[dtype])
        got = hit.rht_kv_attention(q, *t, cud, **signs, max_new=max_new).cpu()
        assert (got[torch.from_numpy(~own)] == 0).all()
        assert torch.equal(got[torch.from_numpy(own)], given.cpu()[torch.from_numpy(own)]) or max_new is not None
    soil((n, 2, d), DT[dtype])
    k, v = hit.rht_kv_read(*t, cud, n, d, **signs, out_dtype=DT[dtype])
    base = torch.full((n, 2, d), 5.0, device="cuda", dtype=DT[dtype])
    _, v2 = hit.rht_kv_read(*t, cud, n, d, **signs, k_out=base)
    for x in (k, v, v2):
        assert (x.cpu()[torch.from_numpy(~own)] == 0).all() and torch.isfinite(x).all()
    assert (base.cpu()[torch.from_numpy(~own)] == 5.0).all()
    assert torch.equal(base.cpu()[torch.from_numpy(own)], k.cpu()[torch.from_numpy(own)]) and torch.equal(v, v2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_without_sequences_are_zero(dtype):
    c = Cache(103, [20], 3, 128, 4, 16).fill()
    t = c.on()
    t[4], t[5] = t[4][:0], t[5][:0]
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, _ = heads(c.r, 700, 6, 128, DT[dtype])
    soil((700, 6, 128), DT[dtype])
    assert (hit.rht_kv_attention(q, *t, cu) == 0).all()
    soil((700, 3, 128), DT[dtype])
    k, v = hit.rht_kv_read(*t, cu, 700, 128, out_dtype=DT[dtype])
    assert (k == 0).all() and (v == 0).all()


def test_replay_with_fewer_tokens():
    """A captured decoding step replayed with other lengths and fewer tokens: the rows left over are zero."""
    c = Cache(105, [60, 70, 80], 2, 64, 8, 16).fill()
    t, signs = c.on(), c.signs()
    cu = torch.from_numpy(cu_of([1, 1, 1])).cuda()
    q, _ = heads(c.r, 3, 4, 64, torch.float32)
    full = hit.rht_kv_attention(q, *t, cu, **signs, max_new=1)
    hit.rht_kv_read(*t, cu, 3, 64, **signs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = hit.rht_kv_attention(q, *t, cu, **signs, max_new=1)
        k, v = hit.rht_kv_read(*t, cu, 3, 64, **signs)
    g.replay()
    assert torch.equal(out, full)
    cu.copy_(torch.from_numpy(cu_of([1, 0, 0])))
    g.replay()
    assert torch.equal(out[0], full[0]) and (out[1:] == 0).all() and (k[1:] == 0).all() and (v[1:] == 0).all()
