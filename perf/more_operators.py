"""Cases of the norm and of the 4-bit product, their plain forms and their calls.

The operators: root-mean-square norm with the residual's addition and quantised outputs (moe_rms_norm), quantisation to E2M1
or E4M3 with power-of-two scales and back (moe_mx_quant, moe_mx_values), and the product of rows with E2M1 weights
(moe_linear). `own` picks between the library's calls and elementary torch operations.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one sequence's new token between two blocks of a layer, the residual in fp32: a launch's latency
        {"name": "norm_one", "op": "norm", "T": 1, "n": 4096, "x": "bf16", "res": "f32", "codes": "none", "out": True},
        # a decode step of a batch: bf16 rows for the router and 8-bit ones for the projections
        {"name": "norm_step_e4m3", "op": "norm", "T": 128, "n": 4096, "x": "bf16", "res": "f32", "codes": "e4m3", "out": True},
        # a norm without a residual over rows whose last block of 128 is half full
        {"name": "norm_odd_e4m3", "op": "norm", "T": 4099, "n": 2880, "x": "f32", "res": "none", "codes": "e4m3", "out": True},
        # a long prompt, the residual in bf16
        {"name": "norm_prompt_e4m3", "op": "norm", "T": 16384, "n": 4096, "x": "bf16", "res": "bf16", "codes": "e4m3",
         "out": True},
        # a batch's rows as 4 bits hold them
        {"name": "quant_rows_e2m1", "op": "quant", "T": 77, "n": 2880, "codes": "e2m1"},
        # a projection's weights quantised at load time, and read back to see what was lost
        {"name": "quant_weights_e2m1", "op": "quant", "T": 16384, "n": 4096, "codes": "e2m1"},
        # one token's queries, keys and values (32 + 8 + 8 heads of 128): the smallest product, bound by the weights
        {"name": "linear_one_e2m1", "op": "linear", "T": 1, "k": 4096, "n": 6144, "codes": "e2m1", "y": "bf16"},
        # a decode step's output projection in 8 bits
        {"name": "linear_step_e4m3", "op": "linear", "T": 64, "k": 4096, "n": 4096, "codes": "e4m3", "y": "bf16"},
        # a ragged batch through a reduction that ends inside a block, sums kept in fp32
        {"name": "linear_odd_e4m3", "op": "linear", "T": 333, "k": 2880, "n": 4099, "codes": "e4m3", "y": "f32"},
        # the norm ahead of the attention and the projection of what it wrote, a decode step of 16 sequences
        {"name": "norm_linear_e2m1", "op": "block", "T": 16, "k": 4096, "n": 6144, "x": "bf16", "res": "f32", "codes": "e2m1",
         "y": "bf16"},
        # a long prompt's projections: bound by the tensor cores
        {"name": "linear_prompt_e2m1", "op": "linear", "T": 16384, "k": 4096, "n": 6144, "codes": "e2m1", "y": "bf16"},
        {"name": "linear_prompt_e4m3", "op": "linear", "T": 8191, "k": 4096, "n": 5760, "codes": "e4m3", "y": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "linear", "linear", "linear", "block"])
    codes = rng.choice(["e2m1", "e4m3"])
    if op == "quant":
        n = 32 * _log(rng, 1, 256)
        return {"op": op, "T": _log(rng, 1, min(16384, 16384 * 4096 // n)), "n": n, "codes": codes}
    if op == "norm":
        n = 32 * _log(rng, 1, 256)
        res, out = rng.choice(["none", "bf16", "f32", "f32"]), rng.choice([("none", True), ("e4m3", True), ("e4m3", False)])
        return {"op": op, "T": _log(rng, 1, min(16384, 16384 * 4096 // n)), "n": n, "x": rng.choice(["bf16", "f32"]),
                "res": res, "codes": out[0], "out": out[1] or res == "none"}
    k, n = 32 * _log(rng, 2, 256), _log(rng, 64, 12288)
    case = {"op": op, "T": _log(rng, 1, max(2, min(16384, 16384 * 4096 * 6144 // (n * k), 16384 * 6144 // n, 16384 * 4096 // k))),
            "k": k, "n": n}
    if op == "block":
        case.update(x=rng.choice(["bf16", "f32"]), res=rng.choice(["bf16", "f32"]))
    return {**case, "codes": codes, "y": rng.choice(["bf16", "bf16", "f32"])}


# ---------------------------------------------------------------- inputs

class _Handle:
    """A library handle that lives as long as the state that holds it."""

    def __init__(self, max_tokens, max_in):
        import fp4_block_scaled_gb300 as moe

        self.moe, self.h = moe, None
        self.h = moe.moe_lin_create(moe.lin_config(max_tokens, max_in), 0)
        self.modes = {"e4m3": moe.MOE_ACT_E4M3_UE8M0_128, "e2m1": moe.MOE_ACT_E2M1_UE8M0_32, "none": moe.MOE_ACT_BF16}
        self.types = {"bf16": moe.MOE_OUT_BF16, "f32": moe.MOE_OUT_F32, "none": moe.MOE_OUT_BF16}

    def __del__(self):
        if self.h is not None:
            self.moe.moe_lin_destroy(self.h)


def _activations(shape, g, dev):
    """Rows as they leave a block: N(0, 1), a few channels several times as large, rows of unlike size."""
    x = torch.randn(shape, generator=g, device=dev)
    channel = 1.0 + 7.0 * (torch.rand(shape[1], generator=g, device=dev) < 0.01).float()
    return x.mul_(channel).mul_(torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device=dev)))


def _code_buffers(T, n, codes, dev):
    width, block = (n // 2, 32) if codes == "e2m1" else (n, 128)
    return (torch.zeros((T, width), device=dev, dtype=torch.uint8),
            torch.zeros((T, -(-n // block)), device=dev, dtype=torch.uint8))


def prepare(case, seed):
    c, dev = case, torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s, T = {"case": c}, c["T"]
    width = c["k"] if c["op"] in ("linear", "block") else c["n"]
    x = _activations((T, width), g, dev)
    s["x"] = x.to(TYPES[c.get("x", "bf16")])
    if c["op"] in ("norm", "block"):
        s["weight"] = (1.0 + 0.2 * torch.randn(width, generator=g, device=dev)).to(torch.bfloat16)
        s["res"] = None
        if c["res"] != "none":
            s["res"] = (3.0 * _activations((T, width), g, dev)).to(TYPES[c["res"]])
    if c["op"] in ("linear", "block"):
        w = torch.randn((c["n"], c["k"]), generator=g, device=dev) * c["k"] ** -0.5
        s["w"], s["ws"] = _quantize_e2m1(w.to(torch.bfloat16).float())
    if own:
        s["h"] = h = _Handle(T, width)
        moe = h.moe
        if c["codes"] != "none":
            s["codes"], s["scales"] = _code_buffers(T, width, c["codes"], dev)
        if c["op"] in ("norm", "block"):
            s["norm"] = moe.norm(s["weight"], width, EPS, h.types[c["x"]], h.types[c["res"]])
            s["res_out"] = None if s["res"] is None else torch.empty_like(s["res"])
            s["out"] = torch.empty((T, width), device=dev, dtype=torch.bfloat16) if c.get("out") else None
        if c["op"] == "quant":
            s["values"] = torch.empty((T, width), device=dev, dtype=torch.bfloat16)
        if c["op"] in ("linear", "block"):
            s["packed"] = torch.empty(moe.moe_linear_packed_bytes(c["n"], c["k"]), device=dev, dtype=torch.uint8)
            moe.moe_linear_pack(h.h, s["w"], s["ws"], c["n"], c["k"], s["packed"], stream=torch.cuda.current_stream())
            s["linear"] = moe.linear(s["packed"], c["n"], c["k"])
            s["y"] = torch.empty((T, c["n"]), device=dev, dtype=TYPES[c["y"]])
    return s


# ---------------------------------------------------------------- one pass

def _scale_byte(amax, top, exponent):
    """The least k with amax <= top * 2^exponent * 2^k (top in [1, 2)), as the byte k + 127; 127 for a block of zeros."""
    m, e = torch.frexp(amax)
    k = torch.where(2 * m <= top, e - 1 - exponent, e - exponent)
    return torch.where(amax > 0, k.clamp(-126, 127) + 127, 127).to(torch.uint8)


def _blocks(x, size):
    """Rows as blocks of `size`, zeros behind a row's end."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % size)).unflatten(-1, (-1, size))


def _power(byte):
    """2^(byte - 127) for a byte in [1, 254], from its bits: exact, where exp2 need not be."""
    return (byte.int() << 23).view(torch.float32)


def _quantize_e4m3(x):
    """float rows [T, n] -> E4M3 codes and one scale byte for 128 elements."""
    b = _blocks(x, 128)
    s = _scale_byte(b.abs().amax(-1), 1.75, 8)
    codes = (b * _power(254 - s)[..., None]).to(torch.float8_e4m3fn)
    return codes.flatten(-2)[..., :x.shape[-1]].contiguous(), s


def _values_e4m3(codes, s):
    b = _blocks(codes.float(), 128) * _power(s)[..., None]
    return b.flatten(-2)[..., :codes.shape[-1]]


def _quantize_e2m1(x):
    """float rows [T, n] -> E2M1 codes, two to a byte, the even element in the low bits, and one scale byte for 32 elements."""
    b = x.unflatten(-1, (-1, 32))
    s = _scale_byte(b.abs().amax(-1), 1.5, 2)
    a = b * _power(254 - s)[..., None]
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
            + 8 * torch.signbit(a).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, s


def _values_e2m1(codes, s):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _power(s)[..., None]).flatten(-2)


def _fake(x, codes):
    """What is left of bf16 rows after their quantisation, in fp32, and the scale bytes."""
    q, s = _quantize_e4m3(x.float()) if codes == "e4m3" else _quantize_e2m1(x.float())
    return (_values_e4m3 if codes == "e4m3" else _values_e2m1)(q, s), s


def _plain_norm(s):
    c, got = s["case"], {}
    row = s["x"].float()
    if s["res"] is not None:
        got["res"] = (row + s["res"].float()).to(s["res"].dtype)
        row = got["res"].float()
    u = row * torch.rsqrt(row.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    return u.to(torch.bfloat16), got


def _plain_linear(x, s):
    values, _ = _fake(x, s["case"]["codes"])
    return torch.matmul(values, _values_e2m1(s["w"], s["ws"]).T).to(TYPES[s["case"]["y"]])


def _plain(s):
    c = s["case"]
    if c["op"] == "quant":
        values, scales = _fake(s["x"], c["codes"])
        return {"values": values.to(torch.bfloat16), "scales": scales.view(torch.float8_e8m0fnu)}
    if c["op"] == "linear":
        return {"y": _plain_linear(s["x"], s)}
    u, got = _plain_norm(s)
    if c["op"] == "block":
        return {**got, "y": _plain_linear(u, s)}
    if c["out"]:
        got["out"] = u
    if c["codes"] == "e4m3":
        codes, scales = _quantize_e4m3(u.float())
        got.update(codes=codes, scales=scales.view(torch.float8_e8m0fnu))
    return got


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain(s)
    moe, h, stream = s["h"].moe, s["h"].h, torch.cuda.current_stream()
    mode = s["h"].modes[c["codes"]]
    if c["op"] == "quant":
        moe.moe_mx_quant(h, s["x"], c["T"], c["n"], mode, s["codes"], s["scales"], stream=stream)
        moe.moe_mx_values(h, mode, s["codes"], s["scales"], c["T"], c["n"], moe.MOE_OUT_BF16, s["values"], stream=stream)
        return {"values": s["values"], "scales": s["scales"].view(torch.float8_e8m0fnu)}
    if c["op"] == "linear":
        moe.moe_linear(h, s["linear"], mode, s["x"], c["T"], s["y"], s["h"].types[c["y"]], stream=stream)
        return {"y": s["y"]}
    moe.moe_rms_norm(h, s["norm"], s["x"], c["T"], residual=s["res"], residual_out=s["res_out"], out=s["out"], act_mode=mode,
                     codes=s.get("codes"), scales=s.get("scales"), stream=stream)
    got = {} if s["res"] is None else {"res": s["res_out"]}
    if c["op"] == "block":
        moe.moe_linear(h, s["linear"], mode, s["codes"], c["T"], s["y"], s["h"].types[c["y"]], x_scales=s["scales"], stream=stream)
        return {**got, "y": s["y"]}
    if c["out"]:
        got["out"] = s["out"]
    if c["codes"] == "e4m3":
        got.update(codes=s["codes"].view(torch.float8_e4m3fn), scales=s["scales"].view(torch.float8_e8m0fnu))
    return got


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    T, size = c["T"], {"bf16": 2, "f32": 4, "none": 0}
    code_bytes = {"none": lambda n: 0, "e4m3": lambda n: n + -(-n // 128), "e2m1": lambda n: n // 2 + n // 32}[c["codes"]]
    if c["op"] == "quant":
        # rows in, codes and scales out; those in again, values out
        return {"bytes": T * (4 * c["n"] + 2 * code_bytes(c["n"])), "flops": 2 * T * c["n"]}
    norm = 0
    if c["op"] in ("norm", "block"):
        n = c["n"] if c["op"] == "norm" else c["k"]
        norm = T * (n * (size[c["x"]] + 2 * size[c["res"]]) + code_bytes(n)) + 2 * n
        if c["op"] == "norm":
            return {"bytes": norm + (2 * T * n if c["out"] else 0), "flops": 5 * T * n}
    k, n = c["k"], c["n"]
    rows = T * (2 * k if c["op"] == "linear" else code_bytes(k))
    return {"bytes": norm + rows + n * (k // 2 + k // 32) + T * n * size[c["y"]], "flops": 2 * T * n * k}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _two_to(k):
    return (k + 1023 << 52).view(torch.float64)


def _rounded(x, block, mantissa, least, most):
    """Rows of doubles rounded to a grid of `mantissa` bits behind the point and exponents from `least`, under each block's
    power of two: the least that brings the block's largest within `most`."""
    b = _blocks(x, block)
    amax = b.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(amax / most)).clamp(-126, 127).long()
    k = torch.where(amax > 0, k, 0)
    k = torch.where(amax > most * _two_to(k), k + 1, k)                      # log2's last bit
    k = torch.where((k > -126) & (amax > 0) & (amax <= most * _two_to(k - 1)), k - 1, k)
    a = b * _two_to(-k)
    _, e = torch.frexp(a)
    step = _two_to((e.long() - 1).clamp(min=least) - mantissa)
    v = (torch.round(a / step) * step).clamp(-most, most) * _two_to(k)
    return v.flatten(-2)[..., :x.shape[-1]], _two_to(k[..., 0])


def _grid(x, codes):
    return _rounded(x.double(), 128, 3, -6, 448.0) if codes == "e4m3" else _rounded(x.double(), 32, 1, 0, 6.0)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        values, scales = _grid(s["x"], c["codes"])
        return {"values": values, "scales": scales}
    got, x = {}, s["x"].double()
    if c["op"] in ("norm", "block"):
        if s["res"] is not None:
            got["res"] = x + s["res"].double()
            x = got["res"].to(s["res"].dtype).double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * s["weight"].double()
        if c["op"] == "norm":
            if c["out"]:
                got["out"] = x
            return {**got, **({"codes": None, "scales": None} if c["codes"] != "none" else {})}
        x = x.to(torch.bfloat16)
    values, _ = _grid(x, c["codes"])
    low, high = s["w"] & 15, s["w"] >> 4
    code = torch.stack([low, high], -1).flatten(-2).long()
    e, m = code >> 1 & 3, (code & 1).double()
    w = torch.where(e > 0, (1 + m / 2) * _two_to(e - 1), m / 2) * torch.where(code > 7, -1.0, 1.0)
    w = w * _two_to(s["ws"].long() - 127).repeat_interleave(32, -1)
    got["y"] = values @ w.T
    return got
