"""moe_mx_quant and moe_mx_values byte for byte against the search for the
nearest code, over blocks at every border of their rules."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from lin_setup import MODE, TORCH, TYPE, code_buffers, f64, handle
from oracle import lin as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


def rows(T, n, seed):
    """Values of bf16 over its whole range, blocks of zeros, of equal magnitudes, and of halves between codes."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, n)) * 2.0 ** rng.integers(-100, 100, (T, 1))
    for t in range(T):
        if t % 7 == 1:
            x[t] = 0.0 if t % 2 else -0.0
        if t % 7 == 3:
            x[t] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 448.0, 464.0, 1.0], n) * rng.choice([-1, 1], n)
        if t % 7 == 5:
            x[t] = rng.choice([3.0, 6.0, 6.03125, 7.0, 448.0, 450.0], 1) * 2.0 ** rng.integers(-120, 100)
        if t % 7 == 6:
            x[t] *= 2.0 ** -20 * 2.0 ** rng.integers(-10, 0, n)
    return torch.from_numpy(x).float().cuda().to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,n", [(1, 32), (3, 64), (15, 160), (40, 256), (29, 2880), (300, 128)])
def test_codes_scales_and_values(fmt, T, n):
    x = rows(T, n, T + n)
    q, s = code_buffers(T, n, fmt)
    with handle() as h:
        moe.moe_mx_quant(h, x, T, n, MODE[fmt], q, s)
        want = ol.quantise(f64(x), fmt)
        torch.cuda.synchronize()
        assert np.array_equal(s[:T].cpu().numpy(), want[1]) and np.array_equal(q[:T].cpu().numpy(), want[0])
        assert torch.all(q[T] == 0xEE) and torch.all(s[T] == 0xEE)
        v = ol.values(*want, fmt)
        for t in ("f32", "bf16"):
            out = torch.full((T + 1, n), 7.0, dtype=TORCH[t], device="cuda")
            moe.moe_mx_values(h, MODE[fmt], q, s, T, n, TYPE[t], out)
            torch.cuda.synchronize()
            got = f64(out[:T])
            normal = (np.abs(v) >= 2.0 ** -126) | (v == 0)      # below, a bf16 has fewer bits than a code
            assert np.array_equal(got[normal], v[normal]) and np.all(np.abs(got - v) <= 2.0 ** -133) and torch.all(out[T] == 7.0)
        assert moe.moe_lin_status(h) == moe.MOE_OK


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_values_of_every_code_and_scale(fmt):
    n = 256 if fmt == "e4m3" else 512
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(256, 1).cuda().contiguous()
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, n // (128 if fmt == "e4m3" else 32)).cuda().contiguous()
    out = torch.zeros((256, n), dtype=torch.float32, device="cuda")
    with handle() as h:
        moe.moe_mx_values(h, MODE[fmt], codes, scales, 256, n, TYPE["f32"], out)
        torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        want = ol.values(codes.cpu().numpy(), scales.cpu().numpy(), fmt).astype(np.float32)
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_blocks_that_are_not_finite(fmt):
    n, block = 384, 32 if fmt == "e2m1" else 128
    x = torch.ones((3, n), dtype=torch.bfloat16, device="cuda")
    x[0, 130], x[1, 0], x[2, n - 1] = float("nan"), float("inf"), -float("inf")
    q, s = code_buffers(3, n, fmt)
    out = torch.zeros((3, n), dtype=torch.float32, device="cuda")
    with handle() as h:
        moe.moe_mx_quant(h, x, 3, n, MODE[fmt], q, s)
        moe.moe_mx_values(h, MODE[fmt], q, s, 3, n, TYPE["f32"], out)
        torch.cuda.synchronize()
    for t, at in enumerate((130 // block, 0, (n - 1) // block)):
        bad = torch.zeros(n, dtype=torch.bool, device="cuda")
        bad[at * block:(at + 1) * block] = True
        assert torch.equal(torch.isnan(out[t]), bad) and torch.all(out[t][~bad] == 1.0)
        assert (s[t] == 255).nonzero().flatten().tolist() == [at]


def test_e4m3_codes_are_those_of_the_expert_layers_quantizer():
    x = rows(50, 288, 9)
    q, s = code_buffers(50, 288, "e4m3")
    q2, s2 = code_buffers(50, 288, "e4m3")
    ffn = moe.moe_ffn_create(moe.config(8, 256, 128, 2, 4), 0)
    with handle() as h:
        moe.moe_mx_quant(h, x, 50, 288, MODE["e4m3"], q, s)
        moe.moe_ffn_act_quant(ffn, x, 50, 288, q2, s2)
        torch.cuda.synchronize()
    moe.moe_ffn_destroy(ffn)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_refusals():
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    o = torch.ones((4, 64), dtype=torch.float32, device="cuda")
    q, s = code_buffers(4, 64, "e2m1")
    m = MODE["e2m1"]
    with handle() as h:
        def refused(f, *a, code=moe.MOE_ERR_INVALID_ARG):
            with pytest.raises(moe.MoeError) as e:
                f(h, *a)
            assert e.value.code == code, a
        for a in ((None, 2, 64, m, q, s), (x, -1, 64, m, q, s), (x, 2, 48, m, q, s), (x, 2, 0, m, q, s), (x, 2, 64, 0, q, s), (x, 2, 64, 3, q, s),
                  (x, 2, 64, m, None, s), (x, 2, 64, m, q, None), (x.data_ptr() + 8, 2, 64, m, q, s), (x, 2, 64, m, x, s), (x, 2, 64, m, q, x),
                  (x, 2, 64, m, q, q)):
            refused(moe.moe_mx_quant, *a)
        refused(moe.moe_mx_quant, x, 2 ** 24 + 1, 64, m, q, s, code=moe.MOE_ERR_UNSUPPORTED)
        refused(moe.moe_mx_quant, x, 1, 2 ** 20 + 32, m, q, s, code=moe.MOE_ERR_UNSUPPORTED)
        for a in ((0, q, s, 2, 64, 1, o), (m, None, s, 2, 64, 1, o), (m, q, None, 2, 64, 1, o), (m, q, s, -2, 64, 1, o), (m, q, s, 2, 63, 1, o),
                  (m, q, s, 2, 64, 2, o), (m, q, s, 2, 64, 1, None), (m, q, s, 2, 64, 1, o.data_ptr() + 4), (m, o, s, 2, 64, 1, o), (m, q, o, 2, 64, 1, o)):
            refused(moe.moe_mx_values, *a)
        moe.moe_mx_quant(h, None, 0, 64, m, None, None)
        moe.moe_mx_values(h, m, None, None, 0, 64, 1, None)
