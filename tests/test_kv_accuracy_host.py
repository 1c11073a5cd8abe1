"""The bounds on attention's error over the rotated cache tell fp16 operands from bf16 ones: roundings planted in the
float64 oracle (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import kvcache as kc
from tests._kv import Cache
from tests.test_gpu_kv import cu_of
from tests.test_gpu_kv_accuracy import few, over_root_mean_square, reference


def to(x, kind):
    return x if kind is None else torch.from_numpy(np.ascontiguousarray(x)).to(kind).double().numpy()


H, B = torch.float16, torch.bfloat16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_as,k_as,p_as,v_as,sharp,fits", [
    (H, H, H, H, 0.1, True), (H, H, H, H, 0.7, True), (H, H, B, H, 0.1, False), (H, H, H, B, 0.1, False),
    (B, H, H, H, 0.7, False), (H, B, H, H, 0.7, False)])
def test_prompts(q_as, k_as, p_as, v_as, sharp, fits, d):
    new, g = 90, 2
    c = Cache(131 + d, [new + 250], 2, d, 8, 32).fill()
    q = np.random.RandomState(d).randn(new, 2 * g, d)
    scale = sharp * d ** -0.5
    want, square, score = reference(q, c, cu_of([new]), scale)
    err = np.zeros_like(want)
    length = new + 250
    hide = np.arange(length) > (250 + np.arange(new))[:, None]
    for h in range(2 * g):
        k, v = (kc.held(y[0], y[1], c.table, 0, np.arange(length), h // g, 8)[0] for y in (c.k, c.v))
        x = to(kc.rotate(q[:, h], c.k_signs) * scale, q_as)
        z = np.where(hide, -np.inf, x @ to(k, k_as).T)
        p = np.exp(z - z.max(1, keepdims=True)) * 16
        err[:, h] = kc.unrotate(to(p, p_as) @ to(v, v_as) / p.sum(1, keepdims=True), c.v_signs) - want[:, h]
    assert not few(new, g, d)
    assert (over_root_mean_square(err, want, square, score, False, torch.float32) <= 2) == fits
