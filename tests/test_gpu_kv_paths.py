"""The rotated key/value cache where its kernels split, join, mask and rescale: many sequences, short ones beside
prompts, scores and values that grow along the cache, narrow strides, shared pages, caches beyond 2^31 bytes."""
import numpy as np
import pytest
import torch

import hadamard_incoherence_transforms_b200 as hit
from hadamard_incoherence_transforms_b200 import _lib, api
from oracle import kvcache as kc
from tests._kv import U32, UBF, Cache, check_attention, heads
from tests.test_gpu_kv import DT, check_append, cu_of

pytestmark = pytest.mark.gpu


def attend_both(c, new, g, dtype=torch.bfloat16, causal=True, window=0, scale=None, out=None, max_new=None):
    cu = cu_of(new)
    q, q64 = heads(c.r, int(cu[-1]), c.hk * g, c.d, dtype)
    scale = c.d ** -0.5 if scale is None else scale
    want, size = kc.attention(q64, c.k, c.v, c.table, cu, c.lens, c.bits, c.k_signs, c.v_signs, scale, causal, window)
    got = hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), causal=causal, window=window,
                               sm_scale=scale, out=out, max_new=max_new)
    return got, want, size


@pytest.mark.parametrize("seqs,most,g,d", [(33, 3, 2, 64), (40, 90, 2, 64), (140, 5, 4, 128), (140, 80, 1, 64),
                                           (300, 3, 1, 64), (700, 2, 2, 64)])
def test_many_sequences(seqs, most, g, d):
    """More sequences than a warp's lanes and than a block's threads, empty ones among them, short ones and (where
    most * g > 64) prompts in one call."""
    r = np.random.RandomState(seqs + most)
    new = [int(x) for x in r.randint(0, most + 1, seqs)]
    new[0] = new[-1] = most
    lens = [n + int(r.choice([0, 1, 30, 130])) for n in new]
    c = Cache(seqs, lens, 1, d, 4, 16).fill()
    got, want, size = attend_both(c, new, g)
    check_attention(got, want, size, torch.bfloat16)
    cu = cu_of(new)
    k, _ = heads(c.r, int(cu[-1]), 1, d, torch.bfloat16)
    t, cud = c.on(), torch.from_numpy(cu).cuda()
    k64, before = k.double().cpu().numpy(), [x.cpu().numpy() for x in t[:4]]
    hit.rht_kv_append(k, k, *t, cud, **c.signs())
    after = [x.cpu().numpy() for x in t[:4]]
    check_append(c, before, after, (k64, k64), cu, {}, "bf16")
    _, v = hit.rht_kv_read(*t, cud, int(cu[-1]), d, **c.signs(), out_dtype=torch.float32)
    for i, (s, p) in enumerate(kc.places(cu, c.lens, int(cu[-1]))):
        ref = kc.unrotate(kc.held(after[2], after[3], c.table, s, [p], 0, 4)[0][0], c.v_signs)
        assert (np.abs(v[i, 0].double().cpu().numpy() - ref) <= (np.log2(d) + 3) * U32 * np.linalg.norm(ref)).all()


@pytest.mark.parametrize("new,lens,g,window,causal,d,bits", [
    ([600], [900], 2, 200, True, 64, 4),
    ([513, 40, 1, 300], [513, 1000, 700, 301], 4, 0, True, 128, 4),
    ([129, 700], [2000, 700], 1, 129, True, 128, 8),
    ([260, 65], [1500, 400], 3, 0, False, 64, 8),
    ([300, 40, 1, 129], [1400, 900, 300, 129], 2, 0, True, 256, 8),
    ([257, 500], [700, 500], 1, 200, True, 256, 4),
    ([90], [2000], 5, 0, False, 256, 8),
    ([70, 66, 68, 90, 64, 65, 1], [70, 500, 131, 90, 64, 257, 900], 1, 0, True, 128, 4),
])
def test_prompts_over_several_blocks(new, lens, g, window, causal, d, bits):
    c = Cache(sum(new), lens, 2, d, bits, 32).fill()
    got, want, size = attend_both(c, new, g, causal=causal, window=window)
    check_attention(got, want, size, torch.bfloat16)


@pytest.mark.parametrize("new,g", [(1, 2), (3, 1), (70, 2), (300, 1)])
@pytest.mark.parametrize("up", [True, False])
def test_scores_that_grow_along_the_cache(new, g, up):
    """Scores from 0 to 60, the largest last (every block raises the reference of its rows) or first.  Every key is the
    same vector times a factor and the queries lie along it, so sum|q k| is the score: its error is at most 4 u_h 60
    of a probability, and 1 / sqrt(128) of that as a root mean square over independent roundings (1.5e-3 twice, beside the
    3.9e-3 of probability, value and result)."""
    n, d = 700, 128
    c = Cache(41, [n], 1, d, 8, 16).fill()
    code, w, _ = kc.quantize(c.r.randn(d), 8)
    code = np.asarray(code).reshape(d)
    base = float(np.asarray(w).reshape(()))
    held = code * base
    for p in range(n):
        page, i = kc.slot(c.table, c.pages, c.page, 0, p)
        c.k[0][page, 0, i] = kc.pack(code[None], 8)[0]
        c.k[1][page, 0, i] = base * ((p + 1) if up else (n - p)) / n
    cu = cu_of([new])
    one = kc.unrotate(held, c.k_signs) * (60 / (held @ held))
    q64 = np.repeat(np.repeat(one[None, None], new, 0), g, 1).astype(np.float32)
    want, size = kc.attention(q64.astype(np.float64), c.k, c.v, c.table, cu, c.lens, 8, c.k_signs, c.v_signs, 1.0)
    got = hit.rht_kv_attention(torch.from_numpy(q64).cuda(), *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), sm_scale=1.0)
    check_attention(got, want, size, torch.float32)


@pytest.mark.parametrize("new,g,d", [(1, 4, 64), (40, 4, 64), (80, 4, 256)])
@pytest.mark.parametrize("kind", ["up", "down", "mixed", "first"])
def test_values_of_very_different_size(new, g, d, kind):
    """Value scales that grow or fall by 2^4 every 100 positions, ones that differ by 2^16 from neighbour to
    neighbour, and a first position of next to nothing that takes nearly all of the weight."""
    n = 900
    c = Cache(43, [n], 1, d, 8, 16).fill()
    for p in range(n):
        page, i = kc.slot(c.table, c.pages, c.page, 0, p)
        e = {"up": 4 * (p // 100) - 16, "down": 16 - 4 * (p // 100), "mixed": int(c.r.randint(-8, 9)),
             "first": -9 if p == 0 else 0}[kind]
        c.v[1][page, :, i] *= 2.0 ** e
        if kind == "first" and p == 0:
            c.k[1][page, :, i] *= 6.0
    got, want, size = attend_both(c, [new], g, torch.float32)
    check_attention(got, want, size, torch.float32, kind)


@pytest.mark.parametrize("new,g", [([1, 2], 2), ([1, 1], 16), ([70, 40], 2)])
@pytest.mark.parametrize("page", [4, 64])
@pytest.mark.parametrize("left", [1e30, 3e38, np.inf, np.nan])
def test_slots_that_hold_no_position(new, g, page, left):
    """What a page was left with behind a sequence's end says nothing about the values before it."""
    c = Cache(45, [75, 130], 1, 64, 4, page).fill()
    for scales in (c.k[1], c.v[1]):
        scales[np.isnan(scales)] = left
    got, want, size = attend_both(c, new, g, torch.float32)
    check_attention(got, want, size, torch.float32)


@pytest.mark.parametrize("new", [[2, 1], [50, 3]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_narrow_strides(new, dtype, d):
    """Heads that begin at multiples of 16 bytes and not of 32: results in strided tensors, whose gaps stay."""
    c = Cache(47, [150, 70], 2, d, 4, 16).fill()
    n, pad = sum(new), 16 // DT[dtype].itemsize
    base = torch.full((n, 8, d + pad), 5.0, device="cuda", dtype=DT[dtype])
    got, want, size = attend_both(c, new, 4, DT[dtype], out=base[..., :d])
    check_attention(got, want, size, DT[dtype])
    assert (base[..., d:] == 5.0).all()
    cu = torch.from_numpy(cu_of(new)).cuda()
    plain = hit.rht_kv_read(*c.on(), cu, n, d, **c.signs(), out_dtype=DT[dtype])
    ko, vo = (torch.full((n, 2, d + pad), 5.0, device="cuda", dtype=DT[dtype]) for _ in range(2))
    hit.rht_kv_read(*c.on(), cu, n, d, **c.signs(), k_out=ko[..., :d], v_out=vo[..., :d])
    assert torch.equal(ko[..., :d], plain[0]) and torch.equal(vo[..., :d], plain[1])
    assert (ko[..., d:] == 5.0).all() and (vo[..., d:] == 5.0).all()


def test_read_of_keys_or_values_alone():
    c = Cache(53, [40], 2, 128, 4, 16).fill()
    t = c.on()
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    both = hit.rht_kv_read(*t, cu, 40, 128, **c.signs())
    s = c.signs()
    kv = api._kv(128, 0, 40, *t, cu, s["k_signs"], s["v_signs"])
    for which in (0, 1):
        out = torch.zeros(40, 2, 128, device="cuda", dtype=torch.bfloat16)
        at = [None, None]
        at[which] = out.data_ptr()
        _lib.call("rht_kv_read", kv, *at, 40, 256, 128, 256, 128, 1, torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out, both[which])


@pytest.mark.parametrize("new", [[1, 1], [40, 30]])
def test_shared_pages_and_output_in_the_queries_place(new):
    """Two sequences on the same pages; the result replaces the queries; a workspace full of garbage."""
    c = Cache(59, [200, 180], 2, 128, 4, 16).fill()
    c.table[1, :10] = c.table[0, :10]
    cu = cu_of(new)
    q, q64 = heads(c.r, int(cu[-1]), 8, 128, torch.bfloat16)
    want, size = kc.attention(q64, c.k, c.v, c.table, cu, c.lens, 4, c.k_signs, c.v_signs, 128 ** -0.5)
    need = _lib.load().rht_kv_workspace_bytes(int(cu[-1]), 8, 2, 128, max(new))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    t, cud = c.on(), torch.from_numpy(cu).cuda()
    for _ in range(2):
        x = q.clone()
        got = hit.rht_kv_attention(x, *t, cud, **c.signs(), max_new=max(new), out=x, workspace=ws)
        assert got.data_ptr() == x.data_ptr()
        check_attention(got, want, size, torch.bfloat16)


@pytest.mark.parametrize("page", [1, 2, 8, 65536])
@pytest.mark.parametrize("new", [2, 70])
def test_page_sizes(page, new):
    c = Cache(61, [100, 130], 1, 64, 4, page, spare=1).fill()
    got, want, size = attend_both(c, [new, 1], 1)
    check_attention(got, want, size, torch.bfloat16)


@pytest.mark.parametrize("new", [1, 40])
def test_cache_beyond_2_31_bytes(new):
    """Codes of more than 2^31 bytes, the pages in use at the far end."""
    d, hk, page, bits = 256 if new == 1 else 128, 8, 64, 8
    c = Cache(67, [150], hk, d, bits, page).fill()
    pages = (1 << 31) // (hk * page * d) + 8
    small = c.on()
    t = [torch.zeros((pages,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda") for x in small[:4]]
    for x, y in zip(t, small):
        x[pages - c.pages:] = y
    table = torch.where(small[4] >= 0, small[4] + (pages - c.pages), small[4])
    args = (*t, table, small[5])
    cu = cu_of([new])
    q, q64 = heads(c.r, new, 2 * hk, d, torch.bfloat16)
    want, size = kc.attention(q64, c.k, c.v, c.table, cu, c.lens, bits, c.k_signs, c.v_signs, d ** -0.5)
    cud = torch.from_numpy(cu).cuda()
    check_attention(hit.rht_kv_attention(q, *args, cud, **c.signs()), want, size, torch.bfloat16)
    plain = hit.rht_kv_read(*small, cud, new, d, **c.signs())
    far = hit.rht_kv_read(*args, cud, new, d, **c.signs())
    assert all(torch.equal(x, y) for x, y in zip(plain, far))
    k, _ = heads(c.r, new, hk, d, torch.bfloat16)
    hit.rht_kv_append(k, k, *small, cud, **c.signs())
    hit.rht_kv_append(k, k, *args, cud, **c.signs())
    for x, y in zip(t, small):
        tail = x[pages - c.pages:]
        assert torch.equal(torch.nan_to_num(tail.float(), nan=-1.0), torch.nan_to_num(y.float(), nan=-1.0))


def test_two_streams_at_once():
    """Calls on two streams that run side by side, each with its own workspace, give what they give alone."""
    c = Cache(71, [900, 300], 2, 128, 4, 16).fill()
    t, signs = c.on(), c.signs()
    q, _ = heads(c.r, 200, 8, 128, torch.bfloat16)
    q1, _ = heads(c.r, 2, 8, 128, torch.bfloat16)
    cu, cu1 = (torch.from_numpy(cu_of(x)).cuda() for x in ([150, 50], [1, 1]))
    want = hit.rht_kv_attention(q, *t, cu, **signs), hit.rht_kv_attention(q1, *t, cu1, **signs, max_new=1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(hit.rht_kv_attention(q, *t, cu, **signs))
                got[i].append(hit.rht_kv_attention(q1, *t, cu1, **signs, max_new=1))
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(y, want[j % 2]) for j, y in enumerate(x))


@pytest.mark.parametrize("d,g", [(64, 2), (128, 1), (256, 2)])
@pytest.mark.parametrize("window", [0, 20])
def test_prompts_with_missing_pages_and_tokens_before_the_start(d, g, window):
    """Long chunks of which a part lies before position 0 (rows of 0), pages that are not there in the middle, a
    sequence of which nothing exists, and tokens of no sequence around them."""
    c = Cache(73, [300, 90, 150, 40], 1, d, 4, 16).fill()
    c.table[0, 3:7] = c.pages + 5
    c.table[0, 9] = -1
    c.table[2, :] = -1
    c.lens[1] = 30                       # 90 tokens, 60 of them before the sequence's start
    cu = cu_of([140, 90, 130, 40], first=3)
    n = int(cu[-1]) + 2
    q, q64 = heads(c.r, n, g, d, torch.bfloat16)
    want, size = kc.attention(q64, c.k, c.v, c.table, cu, c.lens, 4, c.k_signs, c.v_signs, d ** -0.5, True, window)
    out = torch.full((n, g, d), 5.0, device="cuda", dtype=torch.bfloat16)
    hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), window=window, out=out)
    assert (out[:3] == 5.0).all() and (out[-2:] == 5.0).all()
    check_attention(out, want, size, torch.bfloat16)
    assert (out[3 + 140:3 + 140 + 60] == 0).all() and (out[3 + 230:3 + 360] == 0).all()
