"""GPU parity of the rotated key/value cache: appending, attention and reading against the float64 oracle."""
import numpy as np
import pytest
import torch

import hadamard_incoherence_transforms_b200 as hit
from oracle import kvcache as kc
from tests._kv import U32, UBF, Cache, check_attention, heads

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rope_args(r, d, kind, tokens, share=1.0):
    """(keyword arguments of a call, keyword arguments of the oracle)"""
    if kind == "none":
        return {}, {}
    n = int(d * share) // 2
    f = (10000.0 ** (-np.arange(n) / n)).astype(np.float32)
    call, ref = {"inv_freq": torch.from_numpy(f).cuda()}, {"inv_freq": f}
    if kind.startswith("inter"):
        call["interleaved"] = ref["interleaved"] = True
    if kind.endswith("axes"):
        pos = r.randint(0, 5000, (3, tokens)).astype(np.int32)
        axis = r.randint(0, 3, n).astype(np.int8)
        call |= {"positions": torch.from_numpy(pos).cuda(), "rope_axis": torch.from_numpy(axis).cuda()}
        ref |= {"positions": pos, "axis": axis}
    return call, ref


def cu_of(n, first=0):
    return np.concatenate([[first], first + np.cumsum(n)]).astype(np.int32)


def check_append(c, before, after, x, cu, ref, dtype):
    """Codes equal wherever the quotient is not within its error of a rounding border, scales within their error;
    every other byte of the cache as it was.  The kernel's u is off by (log2 d + 12) half steps of fp32 of |u|_2 at
    most: one for each Hadamard stage and the normalisation, the rest for the turn (sine and cosine to 4 half steps)."""
    qmax = 2 ** (c.bits - 1) - 1
    tokens = x[0].shape[0]
    touched = np.zeros((c.pages, c.page), dtype=bool)
    for t, (s, p) in enumerate(kc.places(cu, c.lens, tokens)):
        at = None if s is None else kc.slot(c.table, c.pages, c.page, s, p)
        if at is None:
            continue
        touched[at] = True
        for name, dense, signs, codes, scales in (("k", x[0], c.k_signs, after[0], after[1]),
                                                  ("v", x[1], c.v_signs, after[2], after[3])):
            y = dense[t]
            if name == "k" and "inv_freq" in ref:
                y = kc.rope(y, kc.angles(ref["inv_freq"], p, t, ref.get("positions"), ref.get("axis")),
                            ref.get("interleaved", False))
            u = kc.rotate(y, signs)
            q, w, quot = kc.quantize(u, c.bits)
            top = np.abs(u).max(-1)
            off = (np.log2(c.d) + 12) * U32 * np.linalg.norm(u, axis=-1) / np.where(top > 0, top, 1.0)
            got_q, got_w = kc.unpack(codes[at[0], :, at[1]], c.bits), scales[at[0], :, at[1]].astype(np.float64)
            bad = ~(np.abs(got_w - w) <= (off + 2 * U32) * w) & ~(np.isnan(w) & np.isnan(got_w))
            assert not bad.any(), (name, t, got_w, w)
            border = np.abs(quot - np.floor(quot) - 0.5) <= ((2 * off + 4 * U32) * qmax)[:, None]
            wrong = (got_q != q) & ~border
            assert not wrong.any(), (name, t, np.argwhere(wrong)[:3])
            assert (np.abs(got_q - q) <= 1).all()
    for a, b in zip(before, after):
        np.testing.assert_array_equal(a.transpose(0, 2, 1, *range(3, a.ndim))[~touched],
                                      b.transpose(0, 2, 1, *range(3, b.ndim))[~touched])


APPENDS = [
    # d, bits, dtype, hk, page, rope, share, new tokens, lens (new ones included)
    (128, 4, "bf16", 8, 16, "half", 1.0, [1], [1]),
    (128, 4, "bf16", 8, 64, "half", 1.0, [1, 1, 1], [700, 1, 33]),
    (128, 8, "f32", 3, 32, "inter", 1.0, [5, 0, 40], [5, 9, 111]),
    (64, 4, "f32", 1, 1, "half", 0.5, [17, 2], [20, 2]),
    (64, 8, "bf16", 5, 128, "inter-axes", 0.5, [130, 61], [130, 300]),
    (256, 4, "bf16", 2, 16, "half-axes", 1.0, [31, 9], [47, 9]),
    (256, 8, "f32", 1, 32, "none", 1.0, [3], [3]),
    (128, 4, "bf16", 2, 16, "half", 0.25, [700, 320], [701, 1000]),  # several tokens per CTA
    (128, 8, "bf16", 40, 16, "half", 1.0, [4], [4]),
]


@pytest.mark.parametrize("d,bits,dtype,hk,page,rope,share,new,lens", APPENDS)
def test_append(d, bits, dtype, hk, page, rope, share, new, lens):
    c = Cache(d + bits + sum(new), lens, hk, d, bits, page)
    cu = cu_of(new)
    call, ref = rope_args(c.r, d, rope, int(cu[-1]), share)
    k, k64 = heads(c.r, int(cu[-1]), hk, d, DT[dtype], pad=8, gap=16)
    v, v64 = heads(c.r, int(cu[-1]), hk, d, DT[dtype])
    t = c.on()
    before = [x.cpu().numpy() for x in t[:4]]
    hit.rht_kv_append(k, v, *t, torch.from_numpy(cu).cuda(), **c.signs(), **call)
    check_append(c, before, [x.cpu().numpy() for x in t[:4]], (k64, v64), cu, ref, dtype)


def test_append_far_positions():
    """Angles of positions beyond 2^24 keep their digits."""
    c = Cache(3, [2], 1, 64, 8, 16)
    cu, pos = cu_of([2]), np.array([2 ** 31 - 2, 123456789], dtype=np.int32)
    f = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    k, k64 = heads(c.r, 2, 1, 64, torch.float32)
    v, v64 = heads(c.r, 2, 1, 64, torch.float32)
    t = c.on()
    before = [x.cpu().numpy() for x in t[:4]]
    hit.rht_kv_append(k, v, *t, torch.from_numpy(cu).cuda(), **c.signs(), inv_freq=torch.from_numpy(f).cuda(),
                      positions=torch.from_numpy(pos).cuda())
    check_append(c, before, [x.cpu().numpy() for x in t[:4]], (k64, v64), cu, {"inv_freq": f, "positions": pos}, "f32")


def test_append_leaves_out_what_has_no_place():
    """Tokens before cu[0] and behind the last sequence, positions before 0, behind the table and in bad pages."""
    c = Cache(5, [40, 3, 20], 2, 64, 4, 16)
    c.table[0, 1] = c.pages      # positions 16 .. 31 of sequence 0: a page that is not there
    c.table[2, 0] = -1
    c.lens[1] = -2               # all of sequence 1's tokens lie before its start
    cu = cu_of([35, 2, 20], first=3)
    k, k64 = heads(c.r, 70, 2, 64, torch.bfloat16)
    v, v64 = heads(c.r, 70, 2, 64, torch.bfloat16)
    t = c.on()
    before = [x.cpu().numpy() for x in t[:4]]
    hit.rht_kv_append(k, v, *t, torch.from_numpy(cu).cuda(), **c.signs())
    check_append(c, before, [x.cpu().numpy() for x in t[:4]], (k64, v64), cu, {}, "bf16")


def test_append_zero_tiny_huge_and_not_finite():
    c = Cache(7, [8], 1, 64, 4, 16)
    cu = cu_of([8])
    k, _ = heads(c.r, 8, 1, 64, torch.float32)
    v, _ = heads(c.r, 8, 1, 64, torch.float32)
    for j, f in enumerate([0.0, 1e-38, 1e-44, 1e36, float("inf"), float("nan")]):
        k[j] = f if f in (0.0, float("inf")) or f != f else k[j] * f
        if f != f or f == float("inf"):
            k[j, 0, 1:] = 1.0
    t = c.on()
    before = [x.cpu().numpy() for x in t[:4]]
    hit.rht_kv_append(k, v, *t, torch.from_numpy(cu).cuda(), **c.signs())
    page, table = t[0].cpu().numpy(), c.table
    scales = t[1].cpu().numpy()[table[0, 0], 0]
    q = kc.unpack(page[table[0, 0], 0], 4)
    assert scales[0] == 0.0 and (q[0] == 0).all()
    assert np.isnan(scales[4]) and np.isnan(scales[5]) and (q[4:6] == 0).all()
    for j in (1, 3):
        u = kc.rotate(k[j, 0].double().cpu().numpy(), c.k_signs)
        assert abs(scales[j] - np.abs(u).max() / 7) <= 1e-5 * scales[j] and (np.abs(q[j]).max() == 7)
    assert (np.abs(q[2]) <= 7).all() and np.isfinite(scales[2])


READS = [
    (64, 4, "f32", 3, 16, [5, 0, 40], [5, 9, 111]),
    (64, 8, "bf16", 1, 1, [7], [7]),
    (128, 4, "bf16", 8, 64, [1, 333], [90, 333]),
    (128, 8, "f32", 2, 128, [129], [400]),
    (256, 4, "f32", 2, 32, [31, 9], [47, 9]),
    (256, 8, "bf16", 1, 16, [3], [3]),
    (128, 4, "f32", 1, 16, [900, 650], [901, 650]),
]


@pytest.mark.parametrize("d,bits,dtype,hk,page,new,lens", READS)
def test_read(d, bits, dtype, hk, page, new, lens):
    """The rotation back is off by (log2 d + 3) half steps of fp32 of the vector's norm, then rounded once."""
    c = Cache(d + bits, lens, hk, d, bits, page).fill()
    cu = cu_of(new)
    n = int(cu[-1])
    k, v = hit.rht_kv_read(*c.on(), torch.from_numpy(cu).cuda(), n, d, **c.signs(), out_dtype=DT[dtype])
    for got, (codes, scales), signs in ((k, c.k, c.k_signs), (v, c.v, c.v_signs)):
        got = got.double().cpu().numpy()
        for t, (s, p) in enumerate(kc.places(cu, c.lens, n)):
            for h in range(hk):
                ref = kc.unrotate(kc.held(codes, scales, c.table, s, [p], h, bits)[0][0], signs)
                off = (np.log2(d) + 3) * U32 * np.linalg.norm(ref) + (UBF if dtype == "bf16" else 0) * np.abs(ref)
                assert (np.abs(got[t, h] - ref) <= off).all()


def test_read_of_what_has_no_place():
    """Zeros where a position does not exist; rows of no sequence, and the gaps between strided rows, as they were."""
    c = Cache(11, [40, 20], 2, 64, 8, 16).fill()
    c.table[0, 1] = c.pages + 3
    cu = cu_of([43, 4], first=2)
    base = torch.full((60, 2, 72), 7.0, device="cuda")
    k, v = hit.rht_kv_read(*c.on(), torch.from_numpy(cu).cuda(), 60, 64, **c.signs(), k_out=base[..., :64],
                           v_out=torch.full((60, 2, 64), 7.0, device="cuda"))
    places = kc.places(cu, c.lens, 60)
    for t, (s, p) in enumerate(places):
        if s is None:
            assert (k[t] == 7.0).all() and (v[t] == 7.0).all()
        elif kc.slot(c.table, c.pages, 16, s, p) is None:
            assert (k[t] == 0.0).all() and (v[t] == 0.0).all()
        else:
            assert np.isfinite(k[t].cpu().numpy()).all() and (k[t] != 7.0).any()
    assert (base[..., 64:] == 7.0).all()


ATTENDS = [
    # d, bits, hk, g, page, new, lens, causal, window, rope
    (128, 4, 2, 4, 16, [1], [1], True, 0, "half"),
    (128, 4, 2, 4, 64, [1, 1, 1], [700, 1, 130], True, 0, "half"),
    (128, 8, 1, 8, 32, [1, 0, 1], [257, 9, 64], True, 0, "inter"),
    (64, 4, 3, 1, 16, [1, 2], [65, 300], True, 0, "none"),
    (64, 8, 1, 5, 1, [3, 1], [50, 20], True, 7, "half"),
    (64, 8, 2, 7, 128, [5, 4, 1], [129, 4, 1], True, 0, "inter-axes"),
    (256, 4, 1, 3, 16, [1, 2], [77, 513], True, 0, "half"),
    (256, 8, 2, 2, 32, [9], [40], False, 0, "none"),
    (128, 4, 1, 16, 16, [2], [200], True, 100, "half"),
    (128, 4, 1, 40, 16, [1], [200], True, 0, "half"),
    (128, 8, 2, 4, 16, [33, 7], [33, 200], True, 0, "half"),
    (128, 4, 2, 1, 64, [130, 5, 0, 1], [300, 5, 7, 400], True, 0, "half"),
    (64, 4, 1, 4, 16, [70], [150], False, 0, "half-axes"),
    (64, 8, 2, 2, 32, [200], [200], True, 33, "half"),
    (256, 8, 1, 2, 64, [100, 65], [100, 300], True, 0, "inter"),
    (128, 8, 1, 1, 16, [257], [300], True, 0, "none"),
]


@pytest.mark.parametrize("d,bits,hk,g,page,new,lens,causal,window,rope", ATTENDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention(d, bits, hk, g, page, new, lens, causal, window, rope, dtype):
    c = Cache(d + bits + g, lens, hk, d, bits, page).fill()
    cu = cu_of(new)
    call, ref = rope_args(c.r, d, rope, int(cu[-1]))
    q, q64 = heads(c.r, int(cu[-1]), hk * g, d, DT[dtype], pad=8, gap=8)
    want, size = kc.attention(q64, c.k, c.v, c.table, cu, c.lens, bits, c.k_signs, c.v_signs, d ** -0.5, causal, window,
                              **ref)
    t, cud = c.on(), torch.from_numpy(cu).cuda()
    got = hit.rht_kv_attention(q, *t, cud, **c.signs(), **call, causal=causal, window=window)
    check_attention(got, want, size, DT[dtype], "default")
    again = hit.rht_kv_attention(q, *t, cud, **c.signs(), **call, causal=causal, window=window)
    assert torch.equal(got, again)  # no order of atomics in it
    # a tight bound on the new tokens, and one that is wrong, give right results too
    for m in (max(new), 1):
        check_attention(hit.rht_kv_attention(q, *t, cud, **c.signs(), **call, causal=causal, window=window, max_new=m),
                        want, size, DT[dtype], f"max_new {m}")


@pytest.mark.parametrize("length", [112, 100, 150])
def test_attention_masked_rows_and_missing_pages(length):
    """Rows that see nothing are 0, missing pages are not seen, tokens of no sequence are left as they were.  Sequence
    0 was filled up to position 100: rows that see the unfilled ones (NaN scales) are NaN; of length 150, its last
    positions are behind the table."""
    c = Cache(13, [100, 3, 60], 2, 128, 8, 16).fill()
    c.table[0, 2] = c.pages
    c.table[2, :] = -1
    c.lens[0] = length
    cu = cu_of([5, 6, 2], first=1)
    q, q64 = heads(c.r, 17, 8, 128, torch.bfloat16)
    want, size = kc.attention(q64, c.k, c.v, c.table, cu, c.lens, 8, c.k_signs, c.v_signs, 0.1)
    out = torch.full((17, 8, 128), 5.0, device="cuda", dtype=torch.bfloat16)
    hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), sm_scale=0.1, out=out)
    own = np.array([s is not None for s, _ in kc.places(cu, c.lens, 17)])
    assert (out.cpu()[torch.from_numpy(~own)] == 5.0).all()
    nan = own & np.isnan(want).all(-1).all(-1)
    assert nan.sum() == (0 if length == 100 else 5)
    assert torch.isnan(out.cpu()[torch.from_numpy(nan)]).all()
    check_attention(out, want, size, torch.bfloat16)
    assert (want[6:9] == 0).all() and (out[6:9] == 0).all() and (out[12:14] == 0).all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_attention_scales(scale):
    """A scale of zero is a plain average; a negative one and a very sharp one."""
    c = Cache(17, [90], 1, 64, 4, 16).fill()
    cu = cu_of([4])
    q, q64 = heads(c.r, 4, 2, 64, torch.float32)
    want, size = kc.attention(q64, c.k, c.v, c.table, cu, c.lens, 4, c.k_signs, c.v_signs, scale)
    got = hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), sm_scale=scale)
    check_attention(got, want, size, torch.float32)


@pytest.mark.parametrize("new", [1, 70])
def test_attention_large_and_small_queries(new):
    """Queries beyond fp16's range and below its smallest step: the power of two goes by the row."""
    c = Cache(19, [90], 1, 64, 8, 16).fill()
    cu = cu_of([new])
    q, q64 = heads(c.r, new, 4, 64, torch.float32)
    f = torch.tensor([1e6, 1e-9, 1.0, 0.0], device="cuda")[:, None]
    q, q64 = (q * f).contiguous(), q64 * f.cpu().numpy()
    for scale in (1e-6, 0.125):
        want, size = kc.attention(q64.astype(np.float32), c.k, c.v, c.table, cu, c.lens, 8, c.k_signs, c.v_signs, scale)
        got = hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), sm_scale=scale)
        sel = [1, 2, 3] if scale > 1e-3 else [0, 1, 2, 3]
        check_attention(got[:, sel], want[:, sel], size[:, sel], torch.float32, f"scale {scale}")


@pytest.mark.parametrize("new", [1, 40])
def test_attention_not_finite_only_where_seen(new):
    """A poisoned key or value reaches the rows that see it and no other."""
    for which in (0, 1):
        c = Cache(23, [90, 90], 1, 64, 4, 16).fill()
        at = kc.slot(c.table, c.pages, 16, 0, 60)
        (c.k, c.v)[which][1][at[0], 0, at[1]] = np.nan
        cu = cu_of([new, new])
        q, _ = heads(c.r, 2 * new, 2, 64, torch.float32)
        got = hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs()).cpu()
        pos = np.array([p for _, p in kc.places(cu, c.lens, 2 * new)])
        sees = (np.arange(2 * new) < new) & (pos >= 60)
        assert torch.isnan(got[torch.from_numpy(sees)]).all()
        assert torch.isfinite(got[torch.from_numpy(~sees)]).all()


def test_append_attend_and_read_together():
    """A prompt in two chunks and then single tokens, as a model would run them: attention over what was appended
    equals plain attention over the vectors read back."""
    d, hk, g, page = 128, 2, 4, 16
    c = Cache(29, [150, 61], hk, d, 8, page)
    t = c.on()
    f = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    rope = {"inv_freq": torch.from_numpy(f).cuda()}
    have = [0, 0]
    for new in ([100, 30], [47, 29], [1, 1], [1, 1], [1, 0]):
        have = [a + b for a, b in zip(have, new)]
        cu = cu_of(new)
        n = int(cu[-1])
        lens = torch.tensor(have, dtype=torch.int32).cuda()
        args = (*t[:5], lens, torch.from_numpy(cu).cuda())
        k, _ = heads(c.r, n, hk, d, torch.bfloat16)
        v, _ = heads(c.r, n, hk, d, torch.bfloat16)
        q, q64 = heads(c.r, n, hk * g, d, torch.bfloat16)
        hit.rht_kv_append(k, v, *args, **c.signs(), **rope)
        out = hit.rht_kv_attention(q, *args, **c.signs(), **rope, max_new=max(new))
        whole = cu_of(have)
        kk, vv = hit.rht_kv_read(*t[:5], lens, torch.from_numpy(whole).cuda(), int(whole[-1]), d, **c.signs(),
                                 out_dtype=torch.float32)
        for s in range(2):
            ks, vs = (x[whole[s]:whole[s + 1]].double().cpu().numpy() for x in (kk, vv))
            for i in range(new[s]):
                row, p = int(cu[s]) + i, have[s] - new[s] + i
                for h in range(hk * g):
                    x = kc.rope(q64[row, h], p * f.astype(np.float64), False)
                    z = ks[:p + 1, h // g] @ x * d ** -0.5
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    ref = w @ vs[:p + 1, h // g]
                    bound = (4 * 2.0 ** -11 * (np.abs(kc.rotate(ks[:p + 1, h // g], c.k_signs))
                                               @ np.abs(kc.rotate(x, c.k_signs))).max() * d ** -0.5 + 2 * UBF + 2.0 ** -14)
                    bound = bound * (w @ np.linalg.norm(vs[:p + 1, h // g], axis=1)) + UBF * np.linalg.norm(ref)
                    assert np.linalg.norm(out[row, h].double().cpu().numpy() - ref) <= bound
    # values and keys of the cache stand for what went in, to the codes' half step
    assert torch.isfinite(kk).all()


def test_graph_capture_other_stream_and_repeat():
    """Two captured graphs and eager calls on a side stream give the eager results; nothing is kept between calls."""
    c = Cache(31, [300, 90], 2, 128, 4, 16).fill()
    cu = torch.from_numpy(cu_of([3, 40])).cuda()
    t = c.on()
    q, _ = heads(c.r, 43, 8, 128, torch.bfloat16)
    q1, _ = heads(c.r, 2, 8, 128, torch.bfloat16)
    cu1 = torch.from_numpy(cu_of([1, 1])).cuda()
    want, want1 = hit.rht_kv_attention(q, *t, cu, **c.signs()), hit.rht_kv_attention(q1, *t, cu1, max_new=1, **c.signs())
    signs = c.signs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            a, b = hit.rht_kv_attention(q, *t, cu, **signs), hit.rht_kv_attention(q1, *t, cu1, max_new=1, **signs)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, want) and torch.equal(b, want1)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((hit.rht_kv_attention(q, *t, cu, **signs), hit.rht_kv_attention(q1, *t, cu1, max_new=1, **signs)))
        graphs.append(g)
    for g in (*graphs, *graphs):
        g.replay()
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, want1)


def test_empty_calls():
    c = Cache(37, [5], 1, 64, 4, 16).fill()
    t = c.on()
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 2, 64, device="cuda")
    assert hit.rht_kv_attention(q, *t, zero).shape == (0, 2, 64)
    hit.rht_kv_append(q[:, :1], q[:, :1], *t, zero)
    k, v = hit.rht_kv_read(*t, zero, 0, 64)
    assert k.shape == v.shape == (0, 1, 64)
    # sequences without tokens, tokens without a sequence, a cache without pages
    out = torch.full((3, 2, 64), 9.0, device="cuda")
    hit.rht_kv_attention(torch.ones(3, 2, 64, device="cuda"), *t, zero, out=out)
    assert (out == 9.0).all()
    none = [x[:0] for x in t[:4]]
    got = hit.rht_kv_attention(torch.ones(3, 2, 64, device="cuda"), *none, *t[4:],
                               torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    assert (got == 0).all()
