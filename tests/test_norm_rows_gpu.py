"""moe_rms_norm over more rows than there are CTAs, which then take rows in turn
and fetch the next ones ahead: every type, in place, every format of codes, rows
of up to 32768; what must not count in the choice of a kernel; repeats."""
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from lin_setup import MODE, TORCH, TYPE, code_buffers, handle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


def inputs(T, n, x_type, res, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + T * 1009 + n)
    x = (2.0 * torch.randn((T, n), generator=g, device="cuda")).to(TORCH[x_type])
    r = None if res == "none" else (5.0 * torch.randn((T, n), generator=g, device="cuda")).to(TORCH[res])
    return x, r, (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)


def norm64(row, w, eps):
    d = row.double()
    return d / torch.sqrt((d * d).mean(-1, keepdim=True) + eps) * w.double()


def close(out, want):
    """fp32: at most 32 squares a thread and ten sums of threads, halved by the root; four more roundings: together below 2^-19.
    Then half a step of bf16."""
    return bool(((out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -19) + 2.0 ** -133).all())


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("n", [288, 4096, 8192])
def test_the_type_of_an_absent_residual_counts_for_nothing(x_type, n):
    T = 3000
    x, _, w = inputs(T, n, x_type, "none")
    outs = []
    with handle() as h:
        for t in ("bf16", "f32"):
            outs.append(torch.zeros((T, n), dtype=torch.bfloat16, device="cuda"))
            moe.moe_rms_norm(h, moe.norm(w, n, 1e-6, TYPE[x_type], TYPE[t]), x, T, out=outs[-1])
    assert close(outs[0], norm64(x, w, 1e-6)) and torch.equal(*outs)


def turns(h, T, n, x_type, res, codes, in_place, eps=1e-5):
    """One call; every row and every code held to the formula; nothing behind the last row."""
    x, r, w = inputs(T, n, x_type, res)
    row = x.float() if r is None else (x.float() + r.float()).to(r.dtype)
    in_place = in_place and x_type == "bf16"
    out = torch.full((T + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    ro = None if r is None else torch.full((T + 1, n), 7.0, dtype=r.dtype, device="cuda")
    if in_place:                                                 # rows go over their own inputs
        out[:T].copy_(x)
        x = out
    if r is not None and (in_place or x_type == "f32"):
        ro[:T].copy_(r)
        r = ro
    q, s = code_buffers(T, n, codes) if codes != "none" else (None, None)
    d = moe.norm(w, n, eps, TYPE[x_type], TYPE["f32" if res == "f32" else "bf16"])
    moe.moe_rms_norm(h, d, x, T, residual=r, residual_out=ro, out=out, act_mode=MODE[codes], codes=q, scales=s)
    torch.cuda.synchronize()
    assert moe.moe_lin_status(h) == moe.MOE_OK
    assert close(out[:T], norm64(row, w, eps)) and torch.all(out[T] == 7.0)
    if ro is not None:
        assert torch.equal(ro[:T], row.to(ro.dtype)) and torch.all(ro[T] == 7.0)
    if codes != "none":
        q2, s2 = code_buffers(T, n, codes)
        moe.moe_mx_quant(h, out, T, n, MODE[codes], q2, s2)
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and torch.equal(s, s2)


TYPES = [(x, r) for x in ("bf16", "f32") for r in ("none", "bf16", "f32")]


@pytest.mark.parametrize("x_type,res", TYPES)
@pytest.mark.parametrize("T,n", [(9001, 64), (9001, 128), (4099, 288), (5003, 544), (3001, 4096), (1501, 8192), (801, 12000), (700, 16384)])
def test_rows_in_turn(x_type, res, T, n):
    """More rows than run at once, in every kernel form: a part of a warp, a warp, a CTA with one or two groups a thread."""
    with handle() as h:
        for codes, in_place in (("e4m3", True), ("e2m1", False), ("none", True)):
            turns(h, T, n, x_type, res, codes, in_place)


@pytest.mark.parametrize("x_type,res", TYPES)
@pytest.mark.parametrize("T,n", [(1, 16640), (400, 16640), (333, 20000), (500, 32768)])
def test_wide_rows_in_turn(x_type, res, T, n):
    """Four groups a thread."""
    with handle() as h:
        for codes, in_place in (("e4m3", False), ("e2m1", True), ("none", False)):
            turns(h, T, n, x_type, res, codes, in_place)


@pytest.mark.parametrize("T,n,x_type,res", [(3001, 4096, "bf16", "bf16"), (1201, 2880, "f32", "none"), (20000, 96, "bf16", "f32"), (400, 32768, "f32", "f32")])
def test_repeats_are_equal_bit_for_bit(T, n, x_type, res):
    """A call alone, and one of many that nothing waits between, others' rows before and behind it."""
    (x, r, w), (x2, r2, _) = inputs(T, n, x_type, res), inputs(T, n, x_type, res, 1)
    d = moe.norm(w, n, 1e-6, TYPE[x_type], TYPE["f32" if res == "f32" else "bf16"])

    def buffers():
        return [torch.zeros((T, n), dtype=torch.bfloat16, device="cuda"), None if r is None else torch.zeros_like(r), *code_buffers(T, n, "e4m3")]

    def call(h, x, r, b):
        moe.moe_rms_norm(h, d, x, T, residual=r, residual_out=b[1], out=b[0], act_mode=MODE["e4m3"], codes=b[2], scales=b[3])

    with handle() as h:
        want, got, other = buffers(), buffers(), buffers()
        call(h, x, r, want)
        torch.cuda.synchronize()
        for _ in range(10):
            for _ in range(4):
                call(h, x2, r2, other)
                call(h, x, r, got)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got) if a is not None)
            for b in got:
                if b is not None:
                    b.view(torch.uint8).fill_(0xEE if b.dtype == torch.uint8 else 0)


def test_rows_at_the_ends_of_fp32s_range():
    """Squares beyond fp32 make a row of zeros, squares that vanish leave eps alone; neighbours are as ever."""
    n = 4096
    x = torch.ones((5, n), device="cuda")
    x[1], x[3] = 1e20, 1e-25
    w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = torch.full((5, n), 7.0, dtype=torch.bfloat16, device="cuda")
    with handle() as h:
        moe.moe_rms_norm(h, moe.norm(w, n, 2.0 ** -20, TYPE["f32"], TYPE["f32"]), x, 5, out=out)
    assert not out[1].any() and close(out[3], x[3].double() * 2.0 ** 10)
    for t in (0, 2, 4):
        assert close(out[t], norm64(x[t:t + 1], w, 2.0 ** -20)[0])
