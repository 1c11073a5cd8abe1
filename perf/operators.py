"""The rotated key/value cache's operators: what is measured of them, and their plain forms.

A paged cache holds keys and values as Hadamard-rotated low-bit codes with one
fp32 scale per head vector.  `rht_kv_append` puts new tokens in (rotary
positions, rotation, quantization), `rht_kv_attention` attends from a chunk of
new tokens (or one) over the cache, `rht_kv_read` gives cached vectors back as
dense rows.  Sequence s owns tokens cu[s] .. cu[s + 1] of a call; they are the
last ones of its lens[s] positions.

`run` computes one pass in elementary torch operations, or, where `own` is
true, with the package's kernels.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# The cases.  Keys: op, bits, d (head size), hk (key/value heads), g (query heads
# per key head), page
# (tokens per page), seqs, new_lo .. new_hi (new tokens of a sequence), ctx_lo ..
# ctx_hi (tokens cached before them), axes, pairs and rot (rotary positions: axes,
# half-split or interleaved pairs, share of the head that turns).
# ---------------------------------------------------------------------------
def _case(name, op, **kw):
    c = {"name": name, "op": op, "bits": 4, "d": 128, "hk": 8, "g": 4, "page": 64, "seqs": 1, "new_lo": 1, "new_hi": 1,
         "ctx_lo": 0, "ctx_hi": 0, "axes": 1, "pairs": "half", "rot": 1.0, "dtype": "bf16", "causal": True, "window": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token goes into the cache: launch latency is all there is
        _case("append_one", "append", ctx_lo=700, ctx_hi=700),
        # a serving batch's next tokens, 8-bit codes
        _case("append_batch", "append", bits=8, seqs=64, ctx_lo=100, ctx_hi=8000),
        # prompts of several users admitted together
        _case("append_prompts", "append", seqs=5, new_lo=700, new_hi=2400, ctx_hi=500),
        # image tokens: three position axes, interleaved pairs, fp32 projections, small pages, one head per query head
        _case("append_image", "append", bits=8, d=64, hk=40, g=1, page=16, seqs=3, new_lo=500, new_hi=1100, ctx_hi=90,
              axes=3, pairs="inter", dtype="f32"),
        # a few short sequences handed to another consumer
        _case("read_short", "read", bits=8, d=64, seqs=3, new_lo=90, new_hi=333, page=16, dtype="f32"),
        # whole long sequences read back
        _case("read_long", "read", seqs=4, new_lo=6000, new_hi=9000),
        # decoding for one user
        _case("decode_one", "attend", ctx_lo=1237, ctx_hi=1237),
        # decoding for a serving batch of ragged lengths
        _case("decode_batch", "attend", seqs=64, ctx_lo=300, ctx_hi=8000),
        # decoding over two very long documents, 8-bit codes, eight query heads per key head
        _case("decode_long", "attend", bits=8, g=8, hk=4, seqs=2, ctx_lo=120000, ctx_hi=131000, page=128),
        # checking a few drafted tokens per sequence, sliding window, odd group of query heads
        _case("verify_draft", "attend", bits=8, d=64, g=5, seqs=16, new_lo=3, new_hi=6, ctx_lo=50, ctx_hi=4000,
              window=1000, page=16),
        # a chunk of a long prompt over what is cached of it
        _case("chunk_long", "attend", new_lo=4096, new_hi=4096, ctx_lo=12000, ctx_hi=12000),
        # prompts of several users, ragged, some nearly new, one head per query head
        _case("chunk_ragged", "attend", bits=8, hk=40, g=1, seqs=6, new_lo=1, new_hi=900, ctx_hi=3000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attend", "attend", "attend"])
    kw = {"bits": rng.choice([4, 8]), "d": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
          "hk": rng.choice([1, 2, 4, 5, 8, 16]), "g": rng.choice([1, 2, 3, 4, 5, 7, 8])}
    row = kw["hk"] * kw["d"]  # values of a token's keys; no drawn case costs more than the largest listed ones
    if op != "read":
        kw["axes"] = rng.choice([1, 1, 2, 3])
        kw["pairs"] = rng.choice(["half", "inter"])
        kw["rot"] = rng.choice([1.0, 1.0, 0.5])
    if op == "append":
        seqs = _log(rng, 1, 64)
        n = _log(rng, 1, max(2, min(4000, 7000000 // (seqs * row))))
        kw.update(seqs=seqs, new_lo=max(1, n // 3), new_hi=n, ctx_hi=_log(rng, 1, 2000), dtype=rng.choice(["bf16", "f32"]))
    elif op == "read":
        seqs = _log(rng, 1, 16)
        n = _log(rng, 20, min(9000, 25000000 // (seqs * row)))
        kw.update(seqs=seqs, new_lo=max(1, n // 2), new_hi=n, dtype=rng.choice(["bf16", "f32"]))
    elif rng.random() < 0.5:  # single tokens, or a few
        seqs = _log(rng, 1, 64)
        c = _log(rng, 64, max(65, min(130000, 120000000 // (seqs * row))))
        kw.update(seqs=seqs, new_lo=1, new_hi=rng.choice([1, 1, 1, 2, 5]), ctx_lo=c // 4, ctx_hi=c,
                  window=rng.choice([0, 0, 0, 777]))
    else:  # chunks
        seqs = _log(rng, 1, 6)
        c = _log(rng, 1, 6000)
        n = _log(rng, 20, max(21, min(2400, 90000000 // (row * kw["g"] * seqs * (1 + c // 400)))))
        causal = rng.random() < 0.8
        kw.update(seqs=seqs, new_lo=max(1, n // 2), new_hi=n, ctx_hi=c, causal=causal,
                  window=rng.choice([0, 0, 300]) if causal else 0)
    c = _case("", op, **kw)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and total length of each sequence.  They go by the case, so that a seed changes values, not sizes."""
    r = np.random.RandomState(97 + case["seqs"] + 3 * case["new_hi"] + 7 * case["ctx_hi"])
    n = r.randint(case["new_lo"], case["new_hi"] + 1, case["seqs"])
    ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, case["seqs"])
    return n.astype(np.int64), (n + ctx).astype(np.int64)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _heads(gen, tokens, heads, d, dtype):
    """Projections as a model has them: a few channels of each head are far larger than the rest."""
    x = torch.randn(tokens, heads, d, generator=gen, device=DEV)
    loud = torch.rand(heads, d, generator=gen, device=DEV) < 0.03
    x = x * torch.where(loud, 6.0, 0.8)
    return x.to(torch.float32 if dtype == "f32" else torch.bfloat16)


def _filled(gen, pages, hk, page, d, bits, spread):
    """Codes and scales of rotated vectors (near normal after the rotation)."""
    qmax = 2 ** (bits - 1) - 1
    codes = torch.empty(pages, hk, page, d * bits // 8, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, hk, page, device=DEV)
    step = max(1, (1 << 26) // (hk * page * d))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        y = torch.randn(b - a, hk, page, d, generator=gen, device=DEV)
        s = y.abs().amax(-1, keepdim=True) / qmax
        u = (torch.round(y / s) + (qmax + 1)).to(torch.uint8)
        codes[a:b] = u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)
        scales[a:b] = s[..., 0] * torch.exp(spread * torch.randn(b - a, hk, page, generator=gen, device=DEV))
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * (seed + 1) % (1 << 40))
    n, lens = _lengths(case)
    d, hk, page, bits, seqs = case["d"], case["hk"], case["page"], case["bits"], case["seqs"]
    tokens = int(n.sum())
    per = [-(-int(x) // page) for x in lens]
    cols = max(per) + 1
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(seqs, cols, dtype=torch.int32, device=DEV)
    at = 0
    for s, m in enumerate(per):
        table[s, :m] = order[at:at + m]
        at += m
    st = {"case": case, "tokens": tokens, "n_max": int(n.max()), "l_max": int(lens.max()), "page_table": table,
          "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
          "cu": torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)}
    if case["op"] == "append":
        st["k_codes"], st["k_scales"] = (torch.zeros(pages, hk, page, d * bits // 8, dtype=torch.uint8, device=DEV),
                                         torch.zeros(pages, hk, page, device=DEV))
        st["v_codes"], st["v_scales"] = torch.zeros_like(st["k_codes"]), torch.zeros_like(st["k_scales"])
        st["k"] = _heads(gen, tokens, hk, d, case["dtype"])
        st["v"] = _heads(gen, tokens, hk, d, case["dtype"])
    else:
        st["k_codes"], st["k_scales"] = _filled(gen, pages, hk, page, d, bits, 0.2)
        st["v_codes"], st["v_scales"] = _filled(gen, pages, hk, page, d, bits, 0.5)
        if case["op"] == "attend":
            st["q"] = _heads(gen, tokens, hk * case["g"], d, case["dtype"])
    for key in ("k_signs", "v_signs"):
        st[key] = torch.randint(0, 2, (d,), generator=gen, device=DEV, dtype=torch.int8) * 2 - 1
    st["inv_freq"] = st["positions"] = st["rope_axis"] = None
    if case["op"] != "read":
        pairs = int(d * case["rot"]) // 2
        st["inv_freq"] = (10000.0 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)).float()
        if case["axes"] > 1:  # pair j turns by axis j mod axes; time runs on, height and width are small
            p = torch.randint(0, 80, (case["axes"], tokens), generator=gen, device=DEV, dtype=torch.int32)
            p[0] = torch.arange(tokens, device=DEV, dtype=torch.int32) // 50 + 400
            st["positions"] = p
            st["rope_axis"] = (torch.arange(pairs, device=DEV) % case["axes"]).to(torch.int8)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _hadamard(d):
    i = torch.arange(d, device=DEV)
    bits = i[:, None] & i[None, :]
    odd = torch.zeros_like(bits)
    odd = odd ^ bits
    odd = odd ^ (odd >> 4)
    odd = odd ^ (odd >> 2)
    odd = odd ^ (odd >> 1)
    return 1.0 - 2.0 * (odd & 1).float()


def _turn(x, pos, st):
    """Rotary positions: pos int64 [tokens]; angles in 64 bits."""
    f = st["inv_freq"]
    m = f.numel()
    if st["positions"] is None:
        p = pos[:, None].double()
    else:
        p = st["positions"].double().t()[:, st["rope_axis"].long()]
    a = p * f.double()
    c, s = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    out = x.clone()
    if st["case"]["pairs"] == "half":
        u, w = x[..., :m], x[..., m:2 * m]
        out[..., :m], out[..., m:2 * m] = u * c - w * s, u * s + w * c
    else:
        u, w = x[..., 0:2 * m:2], x[..., 1:2 * m:2]
        out[..., 0:2 * m:2], out[..., 1:2 * m:2] = u * c - w * s, u * s + w * c
    return out


def _quantize(y, bits):
    qmax = 2 ** (bits - 1) - 1
    s = y.abs().amax(-1) / qmax
    t = y / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    u = (torch.round(t).clamp(-qmax, qmax) + (qmax + 1)).to(torch.uint8)
    return (u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)), s


def _values(codes, scales, bits):
    if bits == 8:
        q = codes.float() - 128.0
    else:
        q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0
    return q * scales[..., None]


def _places(st):
    """Sequence, position, page and offset of every token of the call."""
    cu, lens = st["cu"].long(), st["lens"].long()
    t = torch.arange(st["tokens"], device=DEV)
    s = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[s] - (cu[s + 1] - cu[s]) + t - cu[s]
    page = st["case"]["page"]
    return s, pos, st["page_table"][s, pos // page].long(), pos % page


def _plain_read(st, dtype):
    c = st["case"]
    _, _, page, off = _places(st)
    h = _hadamard(c["d"]) / math.sqrt(c["d"])
    out = {}
    for n in ("k", "v"):
        y = _values(st[n + "_codes"][page, :, off], st[n + "_scales"][page, :, off], c["bits"])
        out[n] = ((y @ h) * st[n + "_signs"].float()).to(dtype)
    return out


def _plain_append(st):
    c = st["case"]
    _, pos, page, off = _places(st)
    h = _hadamard(c["d"]) / math.sqrt(c["d"])
    for n in ("k", "v"):
        x = st[n].float()
        x = _turn(x, pos, st) if n == "k" else x
        codes, s = _quantize((x * st[n + "_signs"].float()) @ h, c["bits"])
        st[n + "_codes"][page, :, off] = codes
        st[n + "_scales"][page, :, off] = s


def _plain_attend(st):
    c = st["case"]
    d, hk, g, seqs = c["d"], c["hk"], c["g"], c["seqs"]
    s, pos, _, _ = _places(st)
    h = _hadamard(d) / math.sqrt(d)
    q = (_turn(st["q"].float(), pos, st) * st["k_signs"].float()) @ h
    i = torch.arange(st["tokens"], device=DEV) - st["cu"].long()[s]
    nm = st["n_max"]
    qp = torch.zeros(seqs, nm, hk, g, d, device=DEV)
    qp[s, i] = q.view(-1, hk, g, d)
    pp = torch.full((seqs, nm), -1, device=DEV, dtype=torch.int64)
    pp[s, i] = pos
    need = -(-st["l_max"] // c["page"])
    table = st["page_table"][:, :need].long()
    k = _values(st["k_codes"][table], st["k_scales"][table], c["bits"])  # [seqs, pages, hk, page, d]
    k = k.transpose(1, 2).reshape(seqs, hk, need * c["page"], d)
    x = qp.permute(0, 2, 3, 1, 4).reshape(seqs, hk, g * nm, d) @ k.transpose(-1, -2) / math.sqrt(d)
    del k
    j = torch.arange(need * c["page"], device=DEV)
    seen = (j < st["lens"].long()[:, None, None]).expand(seqs, nm, -1)
    if c["causal"]:
        seen = seen & (j <= pp[..., None])
    if c["window"]:
        seen = seen & (j > pp[..., None] - c["window"])
    x = x.view(seqs, hk, g, nm, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > float("-inf"), top, torch.zeros_like(top))).exp_()
    total = x.sum(-1, keepdim=True)
    v = _values(st["v_codes"][table], st["v_scales"][table], c["bits"])
    v = v.transpose(1, 2).reshape(seqs, hk, need * c["page"], d)
    o = x.reshape(seqs, hk, g * nm, -1) @ v
    o = o.view(seqs, hk, g, nm, d) / torch.where(total > 0, total, torch.ones_like(total))
    o = (o @ h) * st["v_signs"].float()
    return o.permute(0, 3, 1, 2, 4)[s, i].reshape(st["tokens"], hk * g, d).to(st["q"].dtype)


def _own(st):
    import hadamard_incoherence_transforms_b200 as hit

    c = st["case"]
    cache = (st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["page_table"], st["lens"], st["cu"])
    signs = {"k_signs": st["k_signs"], "v_signs": st["v_signs"]}
    rope = {"inv_freq": st["inv_freq"], "interleaved": c["pairs"] == "inter", "positions": st["positions"],
            "rope_axis": st["rope_axis"]}
    if c["op"] == "attend":
        return {"out": hit.rht_kv_attention(st["q"], *cache, **signs, **rope, causal=c["causal"], window=c["window"],
                                            max_new=st["n_max"])}
    if c["op"] == "append":
        hit.rht_kv_append(st["k"], st["v"], *cache, **signs, **rope)
    k, v = hit.rht_kv_read(*cache, rows=st["tokens"], head_dim=c["d"], **signs,
                           out_dtype=torch.float32 if c["op"] == "read" and c["dtype"] == "f32" else torch.bfloat16)
    return {"k": k, "v": v}


def run(st):
    """One pass.  An append gives back what the cache then stands for at the new tokens (bf16 rows)."""
    if own:
        return _own(st)
    c = st["case"]
    if c["op"] == "attend":
        return {"out": _plain_attend(st)}
    if c["op"] == "append":
        _plain_append(st)
    return _plain_read(st, torch.float32 if c["op"] == "read" and c["dtype"] == "f32" else torch.bfloat16)


def work(case):
    n, lens = _lengths(case)
    d, hk, g = case["d"], case["hk"], case["g"]
    tokens = int(n.sum())
    e = 4 if case["dtype"] == "f32" else 2
    vector = d * case["bits"] // 8 + 4
    if case["op"] == "append":  # read k and v, write and read back codes and scales, write bf16 rows
        return {"bytes": 2 * tokens * hk * (d * e + 2 * vector + 2 * d), "flops": 2 * tokens * hk * 2 * d * (math.log2(d) + 4)}
    if case["op"] == "read":
        return {"bytes": 2 * tokens * hk * (vector + d * e), "flops": 2 * tokens * hk * d * (math.log2(d) + 2)}
    keys = pairs = 0
    for a, b in zip(n.tolist(), lens.tolist()):
        if not case["causal"]:
            keys, pairs = keys + b, pairs + a * b
            continue
        pos = np.arange(b - a, b)
        first = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros_like(pos)
        keys, pairs = keys + b - int(first[0]), pairs + int((pos - first + 1).sum())
    return {"bytes": 2 * keys * hk * vector + 2 * tokens * hk * g * d * e, "flops": 4 * d * hk * g * pairs}


# ---------------------------------------------------------------------------
# The definition in 64 bits, one sequence after another
# ---------------------------------------------------------------------------
def _rotation64(d):
    m = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    while m.shape[0] < d:
        m = torch.cat([torch.cat([m, m], 1), torch.cat([m, -m], 1)], 0)
    return m / math.sqrt(d)


def _positions64(st, s, n, length):
    """Angles [n, pairs] of the new tokens of sequence s."""
    f = st["inv_freq"].double()
    a = int(st["cu"][s])
    if st["positions"] is None:
        return torch.outer(torch.arange(length - n, length, device=DEV, dtype=torch.float64), f)
    p = st["positions"][:, a:a + n].double()
    return torch.stack([p[int(x)] for x in st["rope_axis"].tolist()], 1) * f


def _roped64(x, angle, pairs):
    m = angle.shape[1]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.clone()
    if pairs == "half":
        z = torch.complex(x[..., :m].contiguous(), x[..., m:2 * m].contiguous()) * turn
        y[..., :m], y[..., m:2 * m] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :2 * m].reshape(*x.shape[:-1], m, 2).contiguous()) * turn
        y[..., :2 * m] = torch.view_as_real(z).flatten(-2)
    return y


def _held64(st, name, s, length, first=0):
    """What the cache holds of sequence s, positions first .. length: [hk, positions, d], rotated."""
    c = st["case"]
    ids = st["page_table"][s, :-(-length // c["page"])].long()
    u = st[name + "_codes"][ids].transpose(0, 1).flatten(1, 2)[:, first:length].to(torch.int32)
    w = st[name + "_scales"][ids].transpose(0, 1).flatten(1, 2)[:, first:length].double()
    if c["bits"] == 4:
        u = torch.stack([u % 16, u // 16], 3).flatten(2)
    return (u.double() - 2 ** (c["bits"] - 1)) * w[..., None]


def exact(case, seed):
    st = prepare(case, seed)
    n, lens = _lengths(case)
    d, hk, g, bits = case["d"], case["hk"], case["g"], case["bits"]
    rot = _rotation64(d)
    k_out, v_out, o_out = [], [], []
    for s in range(case["seqs"]):
        m, length, a = int(n[s]), int(lens[s]), int(st["cu"][s])
        if case["op"] == "read":
            for name, out in (("k", k_out), ("v", v_out)):
                y = _held64(st, name, s, length, length - m)
                out.append((torch.matmul(y, rot) * st[name + "_signs"].double()).transpose(0, 1))
        elif case["op"] == "append":
            for name, out in (("k", k_out), ("v", v_out)):
                x = st[name][a:a + m].double()
                x = _roped64(x, _positions64(st, s, m, length), case["pairs"]) if name == "k" else x
                y = torch.matmul(x * st[name + "_signs"].double(), rot)
                step = y.abs().max(-1, keepdim=True).values / (2 ** (bits - 1) - 1)
                y = torch.round(y / step) * step
                out.append(torch.matmul(y, rot) * st[name + "_signs"].double())
        else:
            x = _roped64(st["q"][a:a + m].double(), _positions64(st, s, m, length), case["pairs"])
            x = torch.matmul(x * st["k_signs"].double(), rot)
            k, v = _held64(st, "k", s, length), _held64(st, "v", s, length)
            at = torch.arange(length - m, length, device=DEV)[:, None]
            j = torch.arange(length, device=DEV)[None]
            hide = torch.zeros(m, length, dtype=torch.bool, device=DEV)
            if case["causal"]:
                hide |= j > at
            if case["window"]:
                hide |= at - j >= case["window"]
            o = torch.empty(m, hk * g, d, dtype=torch.float64, device=DEV)
            for h in range(hk * g):
                w = torch.softmax((x[:, h] @ k[h // g].t() / math.sqrt(d)).masked_fill(hide, -math.inf), -1)
                o[:, h] = torch.matmul(w @ v[h // g], rot) * st["v_signs"].double()
            o_out.append(o)
    if case["op"] == "attend":
        return {"out": torch.cat(o_out)}
    return {"k": torch.cat(k_out), "v": torch.cat(v_out)}
