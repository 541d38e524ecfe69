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
