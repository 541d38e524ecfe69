"""moe_rms_norm against its formula in fp64: widths of every kernel form, both
types of rows and residual, the codes of moe_mx_quant, rows that are not finite,
refusals."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from lin_setup import MODE, TORCH, TYPE, code_buffers, f64, handle, rand
from oracle import lin as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


def run(h, T, n, x_type="bf16", res="f32", codes="e4m3", weighted=True, in_place=False, eps=1e-6, seed=0, edit=None):
    rng = np.random.default_rng([T, n, seed])
    x = rand(rng, (T, n), 2.0).to(TORCH[x_type])
    w = (1 + 0.3 * rand(rng, (n,))).to(torch.bfloat16) if weighted else None
    r = None if res == "none" else rand(rng, (T, n), 5.0).to(TORCH[res])
    if edit:
        edit(x, r)
    ro = None if r is None else r.clone() if in_place else torch.full((T + 1, n), 7.0, dtype=r.dtype, device="cuda")
    out = torch.full((T + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    d = moe.norm(w, n, eps, TYPE[x_type], TYPE["bf16" if res == "none" else res])
    q = s = None
    if codes != "none":
        q, s = code_buffers(T, n, codes)
    moe.moe_rms_norm(h, d, x, T, residual=ro if in_place else r, residual_out=ro, out=out, act_mode=MODE[codes], codes=q, scales=s)
    torch.cuda.synchronize()
    assert moe.moe_lin_status(h) == moe.MOE_OK
    # nothing behind the last row
    assert torch.all(out[T] == 7.0) and (ro is None or in_place or torch.all(ro[T] == 7.0))
    assert codes == "none" or (torch.all(q[T] == 0xEE) and torch.all(s[T] == 0xEE))
    row = x.float()
    if r is not None:
        row = row + r.float()                                   # one rounding to fp32, and one to bf16
        row = row.to(r.dtype)
        assert torch.allclose(ro[:T], row, rtol=0, atol=0, equal_nan=True)
    want = ol.norm(f64(row), None if w is None else f64(w), eps)
    return dict(x=x, w=w, r=r, out=out[:T], q=q, s=s, want=want, d=d)


def check(h, g, T, n, codes):
    # fp32: 32 squares a thread and two trees of five, their root halves the error; four more
    # roundings; then half a step of bf16
    assert np.all(np.abs(f64(g["out"]) - g["want"]) <= np.abs(g["want"]) * (2.0 ** -8 + 2.0 ** -19) + 2.0 ** -133)
    if codes != "none":
        q, s = code_buffers(T, n, codes)
        moe.moe_mx_quant(h, g["out"].contiguous(), T, n, MODE[codes], q, s)
        torch.cuda.synchronize()
        assert torch.equal(q, g["q"]) and torch.equal(s, g["s"])


@pytest.mark.parametrize("n", [32, 96, 256, 288, 512, 1024, 1056, 2880, 4096, 4128, 8192, 12000, 16384, 32768])
@pytest.mark.parametrize("codes", ["e4m3", "e2m1"])
def test_widths(n, codes):
    with handle() as h:
        for T in (1, 5):
            check(h, run(h, T, n, codes=codes), T, n, codes)


@pytest.mark.parametrize("x_type", ["bf16", "f32"])
@pytest.mark.parametrize("res", ["none", "bf16", "f32"])
@pytest.mark.parametrize("codes", ["none", "e4m3", "e2m1"])
def test_types(x_type, res, codes):
    with handle() as h:
        for T, n in ((131, 224), (67, 2880)):
            check(h, run(h, T, n, x_type, res, codes), T, n, codes)
            check(h, run(h, T, n, x_type, res, codes, weighted=False, in_place=res != "none"), T, n, codes)


@pytest.mark.parametrize("n", [8, 24, 1000, 1032, 4104])
def test_widths_without_codes(n):
    with handle() as h:
        check(h, run(h, 6, n, codes="none"), 6, n, "none")


def test_outputs_are_optional_and_may_be_in_place():
    with handle() as h:
        T, n = 33, 1056
        g = run(h, T, n, codes="e2m1")
        q, s = code_buffers(T, n, "e2m1")
        moe.moe_rms_norm(h, g["d"], g["x"], T, residual=g["r"], act_mode=MODE["e2m1"], codes=q, scales=s)
        torch.cuda.synchronize()
        assert torch.equal(q, g["q"]) and torch.equal(s, g["s"])
        ro = torch.empty_like(g["r"])
        moe.moe_rms_norm(h, g["d"], g["x"], T, residual=g["r"], residual_out=ro)
        x = g["x"].clone()
        moe.moe_rms_norm(h, g["d"], x, T, residual=g["r"], out=x)
        torch.cuda.synchronize()
        assert torch.equal(ro, g["x"].float() + g["r"]) and torch.equal(x, g["out"])


def test_many_rows():
    with handle() as h:
        for T, n, res in ((70000, 64, "bf16"), (9000, 2880, "f32")):
            check(h, run(h, T, n, res=res), T, n, "e4m3")


@pytest.mark.parametrize("n", [256, 2880])
def test_rows_of_zeros_and_rows_that_are_not_finite(n):
    def edit(x, r):
        x[0], r[0] = 0.0, 0.0
        x[2, 5], x[3, n - 1] = float("nan"), float("inf")

    with handle() as h:
        with np.errstate(invalid="ignore"):
            g = run(h, 5, n, codes="e4m3", edit=edit)
        assert not g["out"][0].any()
        assert torch.isnan(g["out"][2]).all() and torch.isnan(g["out"][3, n - 1]) and not g["out"][3, :n - 1].any()
        for t in (1, 4):
            assert np.all(np.abs(f64(g["out"][t]) - g["want"][t]) <= np.abs(g["want"][t]) * (2.0 ** -8 + 2.0 ** -19))
        assert torch.all(g["s"][0] == 127) and torch.all(g["s"][2] == 255) and g["s"][3, -1] == 255 and torch.all(g["s"][3, :-1] == 127)
        assert not torch.any(g["s"][[1, 4]] == 255)
        # eps 0: a row of zeros has no norm
        z = run(h, 1, n, codes="none", eps=0.0, edit=lambda x, r: (x.zero_(), r.zero_()))
        assert torch.isnan(z["out"]).all()


def test_refusals():
    with handle() as h:
        n, T = 64, 2
        x = torch.ones((4, n), dtype=torch.bfloat16, device="cuda")
        r = torch.ones((4, n), dtype=torch.float32, device="cuda")
        w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
        o = torch.zeros((4, n), dtype=torch.bfloat16, device="cuda")
        q, s = code_buffers(4, n, "e4m3")

        def refused(d=moe.norm(w, n, 1e-6, TYPE["bf16"], TYPE["f32"]), x=x, T=T, code=moe.MOE_ERR_INVALID_ARG, **kw):
            kw = {**dict(residual=r, out=o), **kw}
            with pytest.raises(moe.MoeError) as e:
                moe.moe_rms_norm(h, d, x, T, **kw)
            assert e.value.code == code, kw
        coded = dict(act_mode=MODE["e4m3"], codes=q, scales=s)
        refused(T=-1), refused(x=None), refused(out=None), refused(residual=None, residual_out=r)
        refused(act_mode=3, codes=q, scales=s), refused(act_mode=MODE["e4m3"]), refused(**{**coded, "scales": None})
        refused(codes=q, scales=s)
        for bad in (moe.norm(w, 0, 1e-6), moe.norm(w, 60, 1e-6), moe.norm(w, -64, 1e-6), moe.norm(w, n, -1.0), moe.norm(w, n, float("nan")),
                    moe.norm(w, n, float("inf")), moe.norm(w, n, 1e-6, 2), moe.norm(w, n, 1e-6, 0, 5), moe.norm(w.data_ptr() + 2, n, 1e-6)):
            refused(d=bad)
        refused(d=moe.norm(None, 40, 1e-6), **coded)                                         # codes need whole blocks of 32
        refused(d=moe.norm(None, 32776, 1e-6), code=moe.MOE_ERR_UNSUPPORTED), refused(T=2 ** 24 + 1, code=moe.MOE_ERR_UNSUPPORTED)
        for name in ("residual", "out"):
            refused(**{name: (r if name == "residual" else o).data_ptr() + 8})
        refused(x=x.data_ptr() + 2)
        # outputs over inputs and over one another
        refused(out=x.data_ptr() + 16), refused(out=r), refused(residual_out=r.data_ptr() + 16), refused(residual_out=x)
        refused(residual_out=o, out=o), refused(**{**coded, "codes": o}), refused(**{**coded, "scales": q}), refused(**{**coded, "scales": w})
        refused(out=w), refused(d=moe.norm(w, n, 1e-6, TYPE["f32"], TYPE["f32"]), x=r, out=r, residual=None)
        moe.moe_rms_norm(h, moe.norm(w, n, 1e-6), None, 0)                                   # no rows: nothing is read
        assert moe.moe_lin_status(h) == moe.MOE_OK
