"""The rotated key/value cache where scales lie far apart: what a row does not see, or gives no weight to, must cost it
no digits."""
import numpy as np
import pytest
import torch

import hadamard_incoherence_transforms_b200 as hit
from oracle import kvcache as kc
from tests._kv import U32, UH, Cache
from tests.test_gpu_kv import cu_of

pytestmark = pytest.mark.gpu


def set_scale(c, which, s, positions, value, code=None):
    """Scale (and, if given, the code of every element) of keys (0) or values (1) of sequence s at the positions."""
    codes, scales = (c.k, c.v)[which]
    for p in positions:
        page, i = kc.slot(c.table, c.pages, c.page, s, p)
        scales[page, :, i] = value
        if code is not None:
            codes[page, :, i] = kc.pack(np.full((1, c.d), code), c.bits)[0]


def attention(q, c, cu, window):
    """The oracle's result, and for every row sum p |v| and the sum that a unit of relative error of the scores costs:
    a probability off by p_j (e_j - sum p e), e_j = sum_i |q_i k_ji|, moves the result by at most
    sum_j p_j e_j |v_j| + (sum p e) (sum p |v|)."""
    with np.errstate(invalid="ignore", over="ignore"):
        want, _ = kc.attention(q, c.k, c.v, c.table, cu, c.lens, c.bits, c.k_signs, c.v_signs, c.d ** -0.5, True, window)
    tokens, heads_, _ = q.shape
    value, spread = np.zeros((tokens, heads_)), np.zeros((tokens, heads_))
    g = heads_ // c.hk
    for t, (s, p) in enumerate(kc.places(cu, c.lens, tokens)):
        see = np.array(list(kc.visible(p, int(c.lens[s]), True, window)))
        for h in range(heads_):
            k, v = (kc.held(x[0], x[1], c.table, s, see, h // g, c.bits)[0] for x in (c.k, c.v))
            x = kc.rotate(q[t, h], c.k_signs) * c.d ** -0.5
            w = np.exp(k @ x - (k @ x).max())
            w /= w.sum()
            e, n = np.abs(k) @ np.abs(x), np.linalg.norm(v, axis=1)
            value[t, h] = w @ n
            spread[t, h] = (w * e) @ n + (w @ e) * value[t, h]
    return want, value, spread


def check_rows(got, ref, rows, positions):
    """fp32 results of the rows within the worst case of the roundings.  Query and key are rounded to fp16, u_h each: a
    score is off by 2 u_h sum|q k|.  Probability and value are rounded to fp16, u_h each.  A probability (times its value's
    scale) below fp16's normal range is off by 2^-25 where the row's largest is 2^4 or more, and scales of a block that are
    worked on together lie within 2^12: 2^-17 for a position.  fp32 sums: 2^-14."""
    want, value, spread = (x[rows] for x in ref)
    got = got.double().cpu().numpy()[rows]
    assert np.isfinite(want).all() and np.isfinite(got).all()
    err = np.linalg.norm(got - want, axis=-1)
    bound = 2 * UH * spread + (2 * UH + 2.0 ** -14 + positions * 2.0 ** -17) * value + U32 * np.linalg.norm(want, axis=-1)
    assert (err <= bound).all(), f"{(err / np.maximum(bound, 1e-300)).max():.2f} of the bound"


def run(c, new, g, window=0, q64=None):
    cu = cu_of(new)
    if q64 is None:
        q64 = c.r.randn(int(cu[-1]), c.hk * g, c.d)
    q = torch.from_numpy(q64).float().cuda()
    ref = attention(q.double().cpu().numpy(), c, cu, window)
    return hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), window=window), ref


SIZES = [(64, 8), (128, 4), (256, 8), (256, 4)]


@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("left", [1e30, 3e38, 1e-30])
@pytest.mark.parametrize("which", [(0,), (1,), (0, 1)])
def test_prompts_do_not_see_what_lies_before_the_window(d, bits, left, which):
    """Pages before the window may hold anything finite by now."""
    c = Cache(81, [700], 1, d, bits, 16).fill()
    for w in which:
        set_scale(c, w, 0, range(700 - 200 - 150 + 1), left)
    got, ref = run(c, [200], 2, window=150)
    check_rows(got, ref, np.arange(200), 150)


@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("left", [1e30, 3e38, 1e-30])
@pytest.mark.parametrize("which", [(0,), (1,), (0, 1)])
def test_prompts_do_not_see_later_tokens(d, bits, left, which):
    """Nor do the rows of the same tile, or of another half of it."""
    c = Cache(83, [250], 1, d, bits, 16).fill()
    for w in which:
        set_scale(c, w, 0, range(238, 250), left)
    got, ref = run(c, [200], 1)
    check_rows(got, ref, np.arange(238 - 50), 250)


@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("left", [1e30, 1e-30])
def test_drafted_tokens_do_not_see_later_ones(d, bits, left):
    c = Cache(85, [300], 1, d, bits, 16).fill()
    for w in (0, 1):
        set_scale(c, w, 0, [299], left)
    got, ref = run(c, [4], 4)
    check_rows(got, ref, np.arange(3), 300)


@pytest.mark.parametrize("new,g", [(1, 4), (4, 4), (100, 2)])
@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("at", [[3], [400], [3, 130, 131, 400], list(range(128, 256))])
@pytest.mark.parametrize("big", [2.0 ** 25, 2.0 ** 60])
def test_large_values_without_weight(new, g, d, bits, at, big):
    """Positions with values 2^25 (and 2^60) times as large as the others', and e^-120 of their weight: the others are
    the result, with 2^60 too (e^-120 is 2^-173)."""
    c = Cache(87, [600], 1, d, bits, 16).fill()
    x = c.r.randn(d)
    q64 = 0.2 * c.r.randn(new, g, d) + x
    code, w, _ = kc.quantize(-kc.rotate(x, c.k_signs)[None], bits)
    held = (code * w[:, None])[0]
    worst = (kc.rotate(q64, c.k_signs) @ held).max() * d ** -0.5  # the weakest score of a unit scale, negative
    assert worst < 0
    for p in at:
        page, i = kc.slot(c.table, c.pages, c.page, 0, p)
        c.k[0][page, :, i] = kc.pack(code, bits)[0]
        c.k[1][page, :, i] = float(w[0]) * 120 / -worst
        c.v[1][page, :, i] *= big
    got, ref = run(c, [new], g, q64=q64)
    check_rows(got, ref, np.arange(new), 600)


@pytest.mark.parametrize("new,g", [(1, 4), (100, 2)])
@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("at", [3, 400])
def test_a_key_of_nothing_with_a_large_scale(new, g, d, bits, at):
    """Codes of zero under a scale of 1e30: a score of 0 beside all others, whose keys keep their digits."""
    c = Cache(89, [600], 1, d, bits, 16).fill()
    set_scale(c, 0, 0, [at], 1e30, 0)
    got, ref = run(c, [new], g)
    check_rows(got, ref, np.arange(new), 600)


@pytest.mark.parametrize("new,g", [(1, 4), (100, 2)])
@pytest.mark.parametrize("d,bits", SIZES)
def test_neighbours_of_any_size(new, g, d, bits):
    """Keys' and values' scales that differ by up to 2^40 from neighbour to neighbour, values of nothing among them."""
    c = Cache(91, [600], 1, d, bits, 16).fill()
    for p in range(600):
        page, i = kc.slot(c.table, c.pages, c.page, 0, p)
        c.k[1][page, :, i] *= 2.0 ** int(c.r.randint(-40, 1))
        c.v[1][page, :, i] *= 2.0 ** int(c.r.randint(-20, 21)) if p % 7 else 0.0
    got, ref = run(c, [new], g)
    check_rows(got, ref, np.arange(new), 600)


@pytest.mark.parametrize("new,g", [(1, 4), (100, 2)])
@pytest.mark.parametrize("d,bits", SIZES)
def test_values_of_nothing(new, g, d, bits):
    """All values are zero vectors, or all but the last of the weight."""
    c = Cache(93, [300], 1, d, bits, 16).fill()
    set_scale(c, 1, 0, range(300), 0.0)
    got, ref = run(c, [new], g)
    assert (got == 0).all()
    set_scale(c, 1, 0, [7], 0.5)
    got, ref = run(c, [new], g)
    check_rows(got, ref, np.arange(new), 300)
