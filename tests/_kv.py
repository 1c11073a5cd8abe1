"""Small caches for the rotated key/value tests: a random page order, and garbage (random codes, NaN scales) in
every slot that no position uses."""
import numpy as np
import torch

from oracle import kvcache as kc

U32 = 2.0 ** -24  # half a step of fp32, bf16 and fp16, relative
UBF = 2.0 ** -8
UH = 2.0 ** -11


class Cache:
    def __init__(self, seed, lens, hk=2, d=64, bits=4, page=16, spare=2, extra_cols=1):
        r = np.random.RandomState(seed)
        self.r, self.hk, self.d, self.bits, self.page = r, hk, d, bits, page
        self.lens = np.asarray(lens, dtype=np.int32)
        per = [-(-max(int(n), 0) // page) for n in lens]
        self.pages = sum(per) + spare
        order = r.permutation(self.pages)
        self.table = np.full((len(lens), max(per + [0]) + extra_cols), -7, dtype=np.int32)
        at = 0
        for s, m in enumerate(per):
            self.table[s, :m] = order[at:at + m]
            at += m
        shape = (self.pages, hk, page)
        self.k, self.v = [(r.randint(0, 256, shape + (d * bits // 8,)).astype(np.uint8),
                           np.full(shape, np.nan, dtype=np.float32)) for _ in range(2)]
        self.k_signs, self.v_signs = (r.choice([-1, 1], d).astype(np.int8) for _ in range(2))

    def fill(self, spread=0.3):
        """Every position of every sequence holds a quantized normal vector."""
        for s, n in enumerate(self.lens):
            for p in range(int(n)):
                at = kc.slot(self.table, self.pages, self.page, s, p)
                if at is None:
                    continue
                for codes, scales in (self.k, self.v):
                    q, w, _ = kc.quantize(self.r.randn(self.hk, self.d) * np.exp(spread * self.r.randn(self.hk, 1)),
                                          self.bits)
                    codes[at[0], :, at[1]] = kc.pack(q, self.bits)
                    scales[at[0], :, at[1]] = w
        return self

    def on(self, dev="cuda"):
        """The tensors of a call, without cu: k_codes, k_scales, v_codes, v_scales, page_table, lens."""
        t = [torch.from_numpy(np.array(x)).to(dev) for x in (*self.k, *self.v, self.table, self.lens)]
        return t

    def signs(self, dev="cuda"):
        return {"k_signs": torch.from_numpy(self.k_signs).to(dev), "v_signs": torch.from_numpy(self.v_signs).to(dev)}


def heads(r, tokens, h, d, dtype, dev="cuda", pad=0, gap=0):
    """[tokens, h, d] normals as a strided view (pad extra elements between heads, gap between tokens), and float64."""
    x = torch.from_numpy(r.randn(tokens, h * (d + pad) + gap)).to(dtype)
    host = x[:, :h * (d + pad)].view(tokens, h, d + pad)[..., :d] if pad == 0 else \
        x[:, :h * (d + pad)].reshape(tokens, h, d + pad)[..., :d]
    x = x.to(dev)
    view = x.as_strided((tokens, h, d), (h * (d + pad) + gap, d + pad, 1))
    return view, host.double().numpy()


def check_attention(got, ref, size, dtype, what=""):
    """Error of every output vector within the worst case of the roundings that the kernels make.
    Query and key (its code times its scale) are each rounded to fp16, half a step u_h relative per element: a product
    is off by 2 u_h, a score by at most 2 u_h * sum|q k|, and a probability by twice its score's error (one for itself, one
    for the sum it is divided by): 4 u_h * sum|q k|.  Probability and value (code times scale) are each rounded to
    bf16: a term p v is off by 2 u_b.  The result's own rounding adds u_b or u_32; fp32 sums are far below these (2^-14 of
    the total covers thousands of terms).  (Few query rows keep keys and values exact and stay within half of it.)
    Over the whole tensor the roundings are independent: uniform errors have 1 / sqrt(3) of their bound as root mean
    square, and three roundings of u_b (probability, value, result) make sqrt(3 / 3) u_b = 3.9e-3; 8e-3 is twice that."""
    got = got.double().cpu().numpy()
    mine = ~np.isnan(ref).all(-1)
    assert np.isfinite(got[mine]).all(), what
    err = np.linalg.norm(got - ref, axis=-1)[mine]
    score, value = size[mine, 0], size[mine, 1]
    bound = (4 * UH * score + 2 * UBF + 2.0 ** -14) * value + (UBF if dtype == torch.bfloat16 else U32) * np.linalg.norm(
        ref[mine], axis=-1)
    worst = (err / np.maximum(bound, 1e-30)).max() if err.size else 0.0
    assert (err <= bound).all(), f"{what}: {worst:.2f} of the bound"
    norm = np.linalg.norm(ref[mine])
    if norm > 0:
        rel = np.linalg.norm(err) / norm
        assert rel <= 8e-3, f"{what}: relative error {rel:.2e}"
