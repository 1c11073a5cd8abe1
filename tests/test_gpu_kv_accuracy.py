"""How many digits attention over the rotated cache keeps: bounds that go by fp16's half step u_h = 2^-11 for query, key,
probability and value, tight enough that one of them in bf16 (2^-8) fails."""
import numpy as np
import pytest
import torch

import hadamard_incoherence_transforms_b200 as hit
from oracle import kvcache as kc
from tests._kv import U32, UBF, UH, Cache, heads
from tests.test_gpu_kv import cu_of

pytestmark = pytest.mark.gpu
FORMS = [(1, 4), (7, 5), (90, 2), (300, 1)]  # new tokens, query heads of a key head: few rows, and prompts
SIZES = [(64, 8), (64, 4), (128, 4), (128, 8), (256, 8), (256, 4)]


def few(new, g, d):
    return new * g <= (32 if d == 256 else 64)


@pytest.mark.parametrize("new,g", FORMS)
@pytest.mark.parametrize("d,bits", SIZES)
def test_one_visible_position_gives_its_value(new, g, d, bits):
    """With a window of 1 a row's result is its own position's value u (rotated): code times scale, rounded once, by the
    product of the scale with the probability (2^4 to 2^-19) or of the code with the scale.  Element by element
    that is u_h |u_i|; the scale's second part and the quotient by the sum add 2^-6 of it, and the rotation back (log2 d + 3) half
    steps of fp32 of |u| to each element, sqrt(d) times that after the turn back to the rotated basis."""
    c = Cache(121, [new + 37], 2, d, bits, 16).fill()
    cu = cu_of([new])
    q, _ = heads(c.r, new, 2 * g, d, torch.float32)
    out = hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), window=1).double().cpu().numpy()
    for h in range(2 * g):
        u, _ = kc.held(*c.v, c.table, 0, np.arange(37, 37 + new), h // g, bits)
        err = np.abs(kc.rotate(out[:, h], c.v_signs) - u)
        norm = np.linalg.norm(u, axis=1, keepdims=True)
        bound = UH * (1 + 2.0 ** -6) * np.abs(u) + np.sqrt(d) * (np.log2(d) + 3) * U32 * norm
        assert (err <= bound).all(), (err / bound).max()


def reference(q, c, cu, scale):
    """Causal attention in float64, and for every row the sum of (p_j |v_j|)^2, and that of (p_j |v_j|)^2 (s_j + sum p s) with
    s_j = sum_i (q_i k_ji)^2 scale^2."""
    want, square, score = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    x = kc.rotate(q, c.k_signs) * scale
    for s, length in enumerate(c.lens):
        t = np.arange(cu[s], cu[s + 1])
        hide = np.arange(int(length)) > (int(length) - len(t) + np.arange(len(t)))[:, None]
        for h in range(q.shape[1]):
            k, v = (kc.held(y[0], y[1], c.table, s, np.arange(int(length)), h // (q.shape[1] // c.hk), c.bits)[0]
                    for y in (c.k, c.v))
            z = np.where(hide, -np.inf, x[t, h] @ k.T)
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            want[t, h] = kc.unrotate(p @ v, c.v_signs)
            size, one = (v ** 2).sum(1), np.where(hide, 0.0, x[t, h] ** 2 @ (k ** 2).T)
            square[t, h] = p ** 2 @ size
            score[t, h] = (p ** 2 * one) @ size + (p * one).sum(1) * square[t, h]
    return want, square, score


def over_root_mean_square(err, want, square, score, is_few, out_dtype):
    n = 1 if is_few else 2
    mean = UH ** 2 / 3 * n * (square + score).sum() + 2.0 ** -30 * square.sum()
    if out_dtype == torch.bfloat16:
        mean += UBF ** 2 / 3 * (want ** 2).sum()
    return np.sqrt((err ** 2).sum() / mean)


@pytest.mark.parametrize("new,g", FORMS)
@pytest.mark.parametrize("d,bits", SIZES)
@pytest.mark.parametrize("sharp", [0.1, 0.7])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_error_of_the_whole_result(new, g, d, bits, sharp, out_dtype):
    """Roundings are independent and at most u, so their root mean square is at most u / sqrt(3).  A row's error is the sum
    over positions of p v times: one rounding for each operand that is rounded (few rows: the product of probability
    and value's scale; prompts: probability and value), and the score's error less its mean over the row, whose
    squares are s_j and at most sum p s for each of query (few rows) or query and key (prompts).  Twice the root of that
    sum over all rows, with a bf16 result's own roundings beside it and 2^-15 of the values for fp32 sums and the
    exponentials."""
    c = Cache(123 + d + bits, [new + 250, 200], 2, d, bits, 32).fill()
    cu = cu_of([new, 1])
    q, _ = heads(c.r, new + 1, 2 * g, d, torch.float32)
    scale = sharp * d ** -0.5
    q64 = q.double().cpu().numpy()
    want, square, score = reference(q64, c, cu, scale)
    out = torch.empty(q.shape, dtype=out_dtype, device="cuda")
    hit.rht_kv_attention(q, *c.on(), torch.from_numpy(cu).cuda(), **c.signs(), sm_scale=scale, out=out)
    err = out.double().cpu().numpy() - want
    for rows, is_few in ((slice(0, new), few(new, g, d)), (slice(new, new + 1), few(1, g, d))):
        ratio = over_root_mean_square(err[rows], want[rows], square[rows], score[rows], is_few, out_dtype)
        assert ratio <= 2, f"{ratio:.2f} of the root mean square"
