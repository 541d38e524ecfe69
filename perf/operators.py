"""Cases of the decode-attention operators, their plain forms and their calls.

The operators: rotary positions (moe_rope), rotating and writing a step's keys and values into a paged cache
(moe_kv_append), the attention of one new token per sequence over that cache (moe_attn_decode), and copying pages of it in
every layer (moe_kv_copy_pages).  `own` picks between the library's calls and elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch, rotated apart from the cache: a launch's latency
        {"name": "rope_step", "op": "rope", "T": 32, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "layout": "half",
         "scaling": "none", "far": 8000},
        # a long prompt's queries and keys, half of each head rotated, positions far beyond the trained length
        {"name": "rope_prompt", "op": "rope", "T": 16383, "hq": 32, "hkv": 8, "d": 128, "rot": 64, "layout": "interleaved",
         "scaling": "yarn", "far": 1000000},
        # one sequence's new token: the smallest call of a decode step
        {"name": "append_one", "op": "append", "T": 1, "seqs": 1, "start": 5000, "hq": 32, "hkv": 8, "d": 128, "page": 64,
         "kv": "bf16", "rot": 128, "layout": "half", "scaling": "none"},
        # a decode step of a large batch into an 8-bit cache
        {"name": "append_step_e4m3", "op": "append", "T": 256, "seqs": 256, "start": 4000, "hq": 32, "hkv": 8, "d": 128,
         "page": 64, "kv": "e4m3", "rot": 128, "layout": "half", "scaling": "none"},
        # three prompts written at once into an 8-bit cache, after a shared prefix that ends inside a page
        {"name": "append_prompt_e4m3", "op": "append", "T": 16000, "seqs": 3, "start": 77, "hq": 32, "hkv": 8, "d": 128,
         "page": 32, "kv": "e4m3", "rot": 128, "layout": "half", "scaling": "linear"},
        # one chat of ordinary length: latency
        {"name": "attn_one", "op": "attn", "B": 1, "len": 1000, "hq": 32, "hkv": 8, "d": 128, "page": 64, "kv": "bf16",
         "out": "bf16", "window": 0, "cap": 0.0},
        # a served batch of ragged lengths
        {"name": "attn_batch", "op": "attn", "B": 64, "len": 8000, "hq": 32, "hkv": 8, "d": 128, "page": 64, "kv": "bf16",
         "out": "bf16", "window": 0, "cap": 0.0},
        # a larger served batch over an 8-bit cache, eight query heads to a key head
        {"name": "attn_batch_e4m3", "op": "attn", "B": 128, "len": 8000, "hq": 64, "hkv": 8, "d": 128, "page": 32,
         "kv": "e4m3", "out": "f32", "window": 0, "cap": 0.0},
        # two long documents: few rows, so the work is split along the cache
        {"name": "attn_long", "op": "attn", "B": 2, "len": 131071, "hq": 32, "hkv": 8, "d": 128, "page": 64, "kv": "bf16",
         "out": "bf16", "window": 0, "cap": 0.0},
        # a local layer: a sliding window, capped scores, small heads that share nothing, small pages
        {"name": "attn_window", "op": "attn", "B": 48, "len": 20000, "hq": 16, "hkv": 16, "d": 64, "page": 16, "kv": "bf16",
         "out": "bf16", "window": 1000, "cap": 30.0},
        # a beam step: a few forked last pages copied in all 40 layers
        {"name": "copy_fork", "op": "copy", "pairs": 8, "layers": 40, "hkv": 8, "d": 128, "page": 16, "kv": "e4m3"},
        # compaction of a fragmented pool, a group of layers at a time
        {"name": "copy_compact", "op": "copy", "pairs": 512, "layers": 8, "hkv": 8, "d": 128, "page": 64, "kv": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 6, 8, 8, 12, 16, 24])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice(["bf16", "e4m3"])
    if kv == "e4m3":
        d = {80: 96}.get(d, d)
    pos = {"rot": rng.choice([d, d, d // 32 * 16]), "layout": rng.choice(["half", "interleaved"]),
           "scaling": rng.choice(["none", "linear", "ntk", "yarn"])}
    heads = {"hq": hkv * group, "hkv": hkv, "d": d}
    op = rng.choice(["rope", "append", "append", "attn", "attn", "attn", "copy"])
    if op == "rope":
        most = 16383 * 40 * 128 // ((heads["hq"] + hkv) * d)
        return {"op": op, "T": _log(rng, 1, most), **heads, **pos, "far": _log(rng, 100, 1000000)}
    if op == "append":
        most = 16000 * 48 * 128 // ((heads["hq"] + 2 * hkv) * d)
        t = _log(rng, 1, min(most, 16000))
        seqs = t if t <= 300 and rng.random() < 0.7 else min(t, rng.randint(1, 8))
        return {"op": op, "T": t, "seqs": seqs, "start": _log(rng, 1, 8000), **heads, "page": page, "kv": kv, **pos}
    if op == "attn":
        # keys of the batch in all heads, at most those of the largest listed case; fewer where many query heads share one
        most = 2 * 131071 * 8 * 128 // (hkv * d) // (1 if group <= 8 else 4)
        batch = _log(rng, 1, 256)
        length = _log(rng, 1, max(2, min(131071, most // batch)))
        return {"op": op, "B": batch, "len": length, **heads, "page": page, "kv": kv, "out": rng.choice(["bf16", "f32"]),
                "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "cap": rng.choice([0.0, 0.0, 30.0, 50.0])}
    layers = rng.randint(1, 40)
    page_bytes = 2 * hkv * page * d * (2 if kv == "bf16" else 1)
    most = max(2, min(512, 8 * 512 * 262144 // (layers * page_bytes)))
    return {"op": op, "pairs": _log(rng, 1, most), "layers": layers, "hkv": hkv, "d": d, "page": page, "kv": kv}


def _lens(batch, longest):
    """Ragged lengths of a batch, from the case alone: 10 to 100 % of the longest; now and then one key, or none."""
    got = []
    for i in range(batch):
        f = (i * 2654435761 + 40503) % (1 << 32) / (1 << 32)
        n = longest if i == 0 else int(longest * (0.1 + 0.9 * f))
        got.append(1 if i % 13 == 7 else 0 if i % 29 == 11 else n)
    return got


def _tokens(c):
    """(sequence, position) of each token of an append: one to a sequence at its own length, or whole runs after `start`."""
    t = np.arange(c["T"], dtype=np.int64)
    if c["T"] == c["seqs"]:
        return t, np.maximum(np.array(_lens(c["seqs"], c["start"]), np.int64), 1) - 1
    seq = t * c["seqs"] // c["T"]
    first = -(-seq * c["T"] // c["seqs"])
    return seq, c["start"] + t - first


def _frequencies(c):
    """f_i in radians a position, in 64 bits, and the factor on cos and sin: base 10000, scaled to four times the length."""
    r, base, factor, trained = c["rot"], 10000.0, 4.0, 8192
    i = np.arange(r // 2, dtype=np.float64)
    if c["scaling"] == "ntk":
        base *= factor ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "yarn":
        at = [r * math.log(trained / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ---------------------------------------------------------------- inputs

class _Handle:
    """A library handle that lives as long as the state that holds it."""

    def __init__(self, c, pages, seqs, row, hq=None):
        import fp4_block_scaled_gb300 as moe

        self.moe = moe
        self.h = None
        cfg = moe.kv_config(hq or c["hq"], c["hkv"], c["d"], c.get("page", 16), pages, seqs, row,
                            kv_dtype=moe.MOE_KV_E4M3_UE8M0 if c.get("kv") == "e4m3" else moe.MOE_KV_BF16,
                            out_dtype=moe.MOE_OUT_F32 if c.get("out") == "f32" else moe.MOE_OUT_BF16)
        self.h = moe.moe_kv_create(cfg, 0)

    def __del__(self):
        if self.h is not None:
            self.moe.moe_kv_destroy(self.h)


def _rope(c, dev):
    if not own:
        return None
    import fp4_block_scaled_gb300 as moe

    kind = {"none": moe.MOE_ROPE_SCALE_NONE, "linear": moe.MOE_ROPE_SCALE_LINEAR, "ntk": moe.MOE_ROPE_SCALE_NTK,
            "yarn": moe.MOE_ROPE_SCALE_YARN}[c["scaling"]]
    turns, factor = moe.moe_rope_table(c["rot"], 10000.0, kind, 4.0, 8192)
    table = torch.from_numpy(turns.view(np.int64)).to(dev)
    return moe.rope(table, c["rot"], moe.MOE_ROPE_HALF if c["layout"] == "half" else moe.MOE_ROPE_INTERLEAVED, factor), table


def _scale_byte(amax):
    """The least k with amax <= 448 * 2^k, as the byte k + 127; 127 for a row of zeros."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, k.clamp(-126, 127) + 127, 127).to(torch.uint8)


def _quantize(x):
    """float rows [..., d] -> E4M3 codes and ue8m0 scale bytes, one a row."""
    s = _scale_byte(x.abs().amax(-1))
    codes = (x * torch.exp2(127.0 - s.float())[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), s


def _values(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(scales.float() - 127.0)[..., None]


def _pool(c, pages, g, dev, layers=None):
    """A pool's contents: keys and values of N(0, 1), and their scales in an 8-bit cache."""
    shape = (() if layers is None else (layers,)) + (pages, c["hkv"], c["page"], c["d"])
    k, v = (torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16) for _ in range(2))
    if c["kv"] == "bf16":
        return {"k": k, "v": v}
    (kc, ks), (vc, vs) = _quantize(k.float()), _quantize(v.float())
    return {"k": kc, "v": vc, "ks": ks, "vs": vs}


def _struct(p, layer=None):
    import fp4_block_scaled_gb300 as moe

    pick = (lambda t: t) if layer is None else (lambda t: t[layer])
    return moe.kv_pool(pick(p["k"]), pick(p["v"]), *([pick(p["ks"]), pick(p["vs"])] if "ks" in p else []))


def _table(lens, page, spare, rng, dev):
    """A page table whose sequences hold pages scattered over the pool; -1 behind a sequence's last page."""
    need = [-(-n // page) for n in lens]
    total = sum(need)
    row = max(1, max(need))
    ids = rng.permutation(total + spare)[:total].astype(np.int32)
    table = np.full((len(lens), row), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).to(dev), total + spare, row


def prepare(case, seed):
    c, dev = case, torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": c}
    if c["op"] in ("rope", "append"):
        f, m = _frequencies(c)
        s["f"], s["m"] = torch.from_numpy(f).to(dev), m
        s["rope"] = _rope(c, dev)
        # the projections of a step lie in one row: q, then k, then v
        heads = c["hq"] + (1 if c["op"] == "rope" else 2) * c["hkv"]
        qkv = torch.randn((c["T"], heads, c["d"]), generator=g, device=dev, dtype=torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + c["hkv"]], qkv[:, c["hq"] + c["hkv"]:]
        s["q_out"] = torch.zeros((c["T"], c["hq"], c["d"]), device=dev, dtype=torch.bfloat16)
    if c["op"] == "rope":
        s["pos"] = torch.from_numpy(rng.integers(0, c["far"], c["T"]).astype(np.int32)).to(dev)
        s["k_out"] = torch.zeros((c["T"], c["hkv"], c["d"]), device=dev, dtype=torch.bfloat16)
        if own:
            s["h"] = _Handle(c, 1, 1, 1)
    elif c["op"] == "append":
        seq, pos = _tokens(c)
        lens = np.zeros(c["seqs"], np.int64)
        np.maximum.at(lens, seq, pos + 1)
        s["table"], pages, row = _table(lens.tolist(), c["page"], 3, rng, dev)
        s["seq"], s["pos"] = (torch.from_numpy(a.astype(np.int32)).to(dev) for a in (seq, pos))
        s["pool"] = _pool(c, pages, g, dev)
        if own:
            s["h"], s["struct"] = _Handle(c, pages, c["seqs"], row), _struct(s["pool"])
    elif c["op"] == "attn":
        lens = _lens(c["B"], c["len"])
        s["table"], pages, row = _table(lens, c["page"], 3, rng, dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["pool"] = _pool(c, pages, g, dev)
        s["q"] = 1.5 * torch.randn((c["B"], c["hq"], c["d"]), generator=g, device=dev, dtype=torch.bfloat16)
        if own:
            s["h"], s["struct"] = _Handle(c, pages, c["B"], row), _struct(s["pool"])
            s["out"] = torch.empty((c["B"], c["hq"], c["d"]), device=dev,
                                   dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16)
            s["lse"] = torch.empty((c["B"], c["hq"]), device=dev, dtype=torch.float32)
    else:
        pages = 2 * c["pairs"]
        s["pool"] = _pool(c, pages, g, dev, layers=c["layers"])
        order = rng.permutation(pages).astype(np.int32)         # which pages are kept, which are free
        s["pairs"] = torch.from_numpy(np.stack([order[:c["pairs"]], order[c["pairs"]:]], 1)).to(dev)
        if own:
            s["h"] = _Handle(c, pages, 1, 1, hq=c["hkv"])
            s["structs"] = [_struct(s["pool"], i) for i in range(c["layers"])]
    return s


# ---------------------------------------------------------------- one pass

def _rotate(x, cos, sin, c):
    r, x = c["rot"], x.float()
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


def _angles(s):
    a = s["pos"].double()[:, None] * s["f"][None, :]
    return (torch.cos(a) * s["m"]).float()[:, None, :], (torch.sin(a) * s["m"]).float()[:, None, :]


def _pool_out(p):
    """A pool as the values that its bytes stand for."""
    if "ks" not in p:
        return {"k": p["k"], "v": p["v"]}
    return {"k": p["k"].view(torch.float8_e4m3fn), "v": p["v"].view(torch.float8_e4m3fn),
            "ks": p["ks"].view(torch.float8_e8m0fnu), "vs": p["vs"].view(torch.float8_e8m0fnu)}


def _plain_append(s):
    c, p = s["case"], s["pool"]
    cos, sin = _angles(s)
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c))
    k, v = _rotate(s["k"], cos, sin, c), s["v"]
    at, off = s["table"][s["seq"].long(), s["pos"].long() // c["page"]].long(), s["pos"].long() % c["page"]
    if c["kv"] == "e4m3":
        (k, ks), (v, vs) = _quantize(k.float()), _quantize(v.float())
        p["ks"][at, :, off], p["vs"][at, :, off] = ks, vs
    p["k"][at, :, off], p["v"][at, :, off] = k, v
    return {"q": s["q_out"], **_pool_out(p)}


def _plain_attention(s):
    c, p = s["case"], s["pool"]
    B, hkv, d, n = c["B"], c["hkv"], c["d"], s["table"].shape[1] * c["page"]
    at = s["table"].clamp(min=0).long()

    def rows(name):
        x = p[name][at].float() if c["kv"] == "bf16" else _values(p[name][at], p[name + "s"][at])
        return x.transpose(1, 2).reshape(B, hkv, n, d)

    q = s["q"].float().view(B, hkv, c["hq"] // hkv, d)
    score = torch.matmul(q, rows("k").transpose(2, 3)) * d ** -0.5
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    j, length = torch.arange(n, device=q.device), s["lens"].long()[:, None]
    seen = j < length
    if c["window"]:
        seen = seen & (j >= length - c["window"])
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w / total.clamp(min=1e-30), rows("v"))
    lse = torch.where(total > 0, torch.log(total) + top, -math.inf)
    return {"out": out.reshape(B, c["hq"], d).to(torch.float32 if c["out"] == "f32" else torch.bfloat16),
            "lse": lse.reshape(B, c["hq"])}


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "rope":
            cos, sin = _angles(s)
            return {"q": _rotate(s["q"], cos, sin, c), "k": _rotate(s["k"], cos, sin, c)}
        if c["op"] == "append":
            return _plain_append(s)
        if c["op"] == "attn":
            return _plain_attention(s)
        src, dst = s["pairs"].long().unbind(1)
        for t in s["pool"].values():
            t[:, dst] = t[:, src]
        return _pool_out(s["pool"])
    moe, h, stream = s["h"].moe, s["h"].h, torch.cuda.current_stream()
    if c["op"] == "rope":
        moe.moe_rope(h, s["rope"][0], s["pos"], c["T"], q=s["q"], q_out=s["q_out"], k=s["k"], k_out=s["k_out"],
                     ldq=s["q"].stride(0), ldk=s["k"].stride(0), stream=stream)
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "append":
        moe.moe_kv_append(h, s["struct"], s["k"], s["v"], s["pos"], s["table"], c["T"], seq=s["seq"], rope=s["rope"][0],
                          q=s["q"], q_out=s["q_out"], ldq=s["q"].stride(0), ldk=s["k"].stride(0), ldv=s["v"].stride(0),
                          stream=stream)
        return {"q": s["q_out"], **_pool_out(s["pool"])}
    if c["op"] == "attn":
        moe.moe_attn_decode(h, s["struct"], s["q"], s["lens"], s["table"], c["B"], s["out"], lse=s["lse"],
                            softcap=c["cap"], window=c["window"], stream=stream)
        return {"out": s["out"], "lse": s["lse"]}
    moe.moe_kv_copy_pages(h, s["structs"], s["pairs"], c["pairs"], stream=stream)
    return _pool_out(s["pool"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    row = c["d"] * 2 if c.get("kv", "bf16") == "bf16" else c["d"] + 1          # bytes of a cached row
    if c["op"] == "rope":
        n = c["T"] * (c["hq"] + c["hkv"])
        return {"bytes": 4 * n * c["d"] + 4 * c["T"], "flops": 3 * n * c["rot"]}
    if c["op"] == "append":
        n = c["T"] * c["hkv"]
        return {"bytes": 4 * c["T"] * c["hq"] * c["d"] + 2 * n * (2 * c["d"] + row) + 8 * c["T"],
                "flops": 3 * c["T"] * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "attn":
        keys = sum(min(n, c["window"] or n) for n in _lens(c["B"], c["len"]))
        io = c["B"] * c["hq"] * (c["d"] * (2 + (4 if c["out"] == "f32" else 2)) + 4)
        return {"bytes": 2 * keys * c["hkv"] * row + io, "flops": 4 * keys * c["hq"] * c["d"]}
    return {"bytes": 4 * c["pairs"] * c["layers"] * c["hkv"] * c["page"] * row, "flops": 0}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _turned(x, s, c):
    """Each pair as a complex number times m e^{i p f}."""
    r, x = c["rot"], x.double()
    z = x[..., :r].reshape(*x.shape[:-1], 2, r // 2).transpose(-1, -2) if c["layout"] == "half" else \
        x[..., :r].reshape(*x.shape[:-1], r // 2, 2)
    turn = torch.polar(torch.full_like(s["f"], s["m"]).expand(c["T"], -1), torch.outer(s["pos"].double(), s["f"]))
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None, :])
    z = (z.transpose(-1, -2) if c["layout"] == "half" else z).reshape(*x.shape[:-1], r)
    return torch.cat([z, x[..., r:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return {"q": _turned(s["q"], s, c), "k": _turned(s["k"], s, c)}
    if c["op"] == "append":
        got = {"q": _turned(s["q"], s, c), "k": None, "v": None}
        if c["kv"] == "e4m3":
            return {**got, "ks": None, "vs": None}
        k, v, turned = s["pool"]["k"].double(), s["pool"]["v"].double(), _turned(s["k"], s, c)
        pos = s["pos"].long()
        slot = s["table"][s["seq"].long()].gather(1, (pos // c["page"])[:, None])[:, 0].long() * c["page"] + pos % c["page"]
        for pool, x in ((k, turned), (v, s["v"].double())):
            flat = pool.transpose(1, 2).reshape(-1, c["hkv"], c["d"]).index_copy(0, slot, x)
            pool.copy_(flat.view(-1, c["page"], c["hkv"], c["d"]).transpose(1, 2))
        return {**got, "k": k, "v": v}
    if c["op"] == "copy":
        return None
    hkv, d = c["hkv"], c["d"]
    out = torch.zeros((c["B"], c["hq"], d), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((c["B"], c["hq"]), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_lens(c["B"], c["len"])):
        if n == 0:
            continue
        first = max(0, n - c["window"]) if c["window"] else 0
        pages = s["table"][b, first // c["page"]:-(-n // c["page"])].long()
        lo = first - first // c["page"] * c["page"]
        for h in range(hkv):
            def rows(name):
                x = s["pool"][name][pages, h].reshape(-1, d)[lo:lo + n - first]
                if c["kv"] == "bf16":
                    return x.double()
                byte = s["pool"][name + "s"][pages, h].reshape(-1)[lo:lo + n - first]
                return x.view(torch.float8_e4m3fn).double() * torch.pow(2.0, byte.double() - 127.0)[:, None]

            at = slice(h * (c["hq"] // hkv), (h + 1) * (c["hq"] // hkv))
            z = (s["q"][b, at].double() @ rows("k").T) / math.sqrt(d)
            if c["cap"]:
                z = torch.tanh(z / c["cap"]) * c["cap"]
            out[b, at], lse[b, at] = torch.softmax(z, -1) @ rows("v"), torch.logsumexp(z, -1)
    return {"out": out, "lse": lse}
