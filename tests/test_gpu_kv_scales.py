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
    """Causal attention in float64, and for every row sum p |v| and the sum that a unit of relative error of the scores
    costs: a probability off by p_j (e_j - sum p e), e_j = sum_i |q_i k_ji|, moves the result by at most
    sum_j p_j e_j |v_j| + (sum p e) (sum p |v|).  Last, what is lost where fp16 holds probabilities whose largest is 2^4
    or more: 2^-25 of each, or all of a smaller one."""
    tokens, n, _ = q.shape
    want, (value, spread, lost) = np.zeros(q.shape), (np.zeros((tokens, n)) for _ in range(3))
    x = kc.rotate(q, c.k_signs) * c.d ** -0.5
    for s, length in enumerate(c.lens):
        t = np.arange(cu[s], cu[s + 1])
        pos = int(length) - len(t) + np.arange(len(t))
        j = np.arange(int(length))
        hide = (j > pos[:, None]) | ((j <= pos[:, None] - window) if window else False)
        for h in range(n):
            k, v = (kc.held(y[0], y[1], c.table, s, j, h // (n // c.hk), c.bits)[0] for y in (c.k, c.v))
            z = np.where(hide, -np.inf, x[t, h] @ k.T)
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            e, size = np.where(hide, 0.0, np.abs(x[t, h]) @ np.abs(k).T), np.linalg.norm(v, axis=1)
            want[t, h] = kc.unrotate(p @ v, c.v_signs)
            value[t, h] = p @ size
            spread[t, h] = (p * e) @ size + (p * e).sum(1) * value[t, h]
            lost[t, h] = np.minimum(p, 2.0 ** -29 * p.max(1, keepdims=True)) @ size
    return want, value, spread, lost


def check_rows(got, ref, rows, positions):
    """fp32 results of the rows within the worst case of the roundings.  Query and key are rounded to fp16, u_h each: a
    score is off by 2 u_h sum|q k|.  Probability and value are rounded to fp16, u_h each, and below fp16's normal
    range a probability loses what `lost` counts, a product of probability and scale (few rows) 2^-29 of the row's
    largest.  A small scale is itself off by up to 2^-13 (2^-25 where it is 2^-12), fp32 sums by 2^-14."""
    want, value, spread, lost = (x[rows] for x in ref)
    got = got.double().cpu().numpy()[rows]
    assert np.isfinite(want).all() and np.isfinite(got).all()
    err = np.linalg.norm(got - want, axis=-1)
    bound = 2 * UH * spread + (2 * UH + 2.0 ** -13 + 2.0 ** -14 + positions * 2.0 ** -29) * value + lost
    bound += U32 * np.linalg.norm(want, axis=-1)
    assert (err <= bound).all(), f"{(err / np.maximum(bound, 1e-300)).max():.2f} of the bound"


def run(c, new, g, window=0, q64=None):
    cu = cu_of(new)
    if q64 is None:
        q64 = c.r.randn(int(cu[-1]), c.hk * g, c.d)
    q = torch.from_numpy(q64).float().cuda()
    ref = attention(q.double().cpu().numpy(), c, cu, window)
    return hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), window=window), ref


ROWS = [(100, 2), (65, 1), (1, 4), (4, 4)]  # new tokens, query heads of a key head: more than 64 rows, and few
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


@pytest.mark.parametrize("new,g", ROWS)
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


@pytest.mark.parametrize("new,g", ROWS)
@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("at", [3, 400])
def test_a_key_of_nothing_with_a_large_scale(new, g, d, bits, at):
    """Codes of zero under a scale of 1e30: a score of 0 beside all others, whose keys keep their digits."""
    c = Cache(89, [600], 1, d, bits, 16).fill()
    set_scale(c, 0, 0, [at], 1e30, 0)
    got, ref = run(c, [new], g)
    check_rows(got, ref, np.arange(new), 600)


@pytest.mark.parametrize("new,g", ROWS)
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


@pytest.mark.parametrize("new,g", ROWS)
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


@pytest.mark.parametrize("new,g", ROWS)
@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("steps", [(60, -60, 0), (-60, 60, -60), (0, -60, -60, -120, 60), (0, None, 0), (None, -40, None, 40)])
@pytest.mark.parametrize("light", [None, 0, 1, -1])
def test_values_that_go_up_and_down_by_blocks(new, g, d, bits, steps, light):
    """Blocks of 128 values, each 2^step times the usual size (None: zero vectors), all of the same weight, or one block
    with e^-60 of it: neither the way up nor the way down loses or overflows anything."""
    c = Cache(95, [128 * len(steps) + 100], 1, d, bits, 16).fill()
    x = c.r.randn(d)
    q64 = 0.2 * c.r.randn(new, g, d) + x
    code, w, _ = kc.quantize(-kc.rotate(x, c.k_signs)[None], bits)
    worst = (kc.rotate(q64, c.k_signs) @ (code * w[:, None])[0]).max() * d ** -0.5
    for i, step in enumerate(steps):
        for p in range(128 * i, 128 * i + 128):
            page, k = kc.slot(c.table, c.pages, c.page, 0, p)
            c.v[1][page, :, k] *= 0.0 if step is None else 2.0 ** step
            if light is not None and i == light % len(steps):
                c.k[0][page, :, k] = kc.pack(code, bits)[0]
                c.k[1][page, :, k] = float(w[0]) * 60 / -worst
    got, ref = run(c, [new], g, q64=q64)
    check_rows(got, ref, np.arange(new), 128 * len(steps) + 100)


@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("down", [6, 9, 14, 18])
def test_prompts_with_a_first_token_of_small_values(d, bits, down):
    """A first position with most of the weight and values 2^-6 to 2^-18 of the others'."""
    c = Cache(97, [600], 1, d, bits, 16).fill()
    x = c.r.randn(d)
    q64 = 0.2 * c.r.randn(100, 2, d) + x
    code, w, _ = kc.quantize(kc.rotate(x, c.k_signs)[None], bits)
    page, i = kc.slot(c.table, c.pages, c.page, 0, 0)
    c.k[0][page, :, i] = kc.pack(code, bits)[0]
    c.k[1][page, :, i] = w
    c.v[1][page, :, i] *= 2.0 ** -down
    got, ref = run(c, [100], 2, q64=q64)
    check_rows(got, ref, np.arange(100), 600)
