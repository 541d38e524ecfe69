"""moe_mx_quant and moe_mx_values over more elements than the quantiser's threads
hold at once (two loads a thread from 5 million): rows as the formulas give them,
and as calls of fewer rows do."""
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


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,n", [(200001, 32), (40007, 160), (3001, 2880), (1777, 4096), (7, 2 ** 20)])
def test_many_rows(fmt, T, n):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, n), generator=g, device="cuda") * torch.exp2(torch.randint(-30, 30, (T, 1), generator=g, device="cuda").float())
    x = x.to(torch.bfloat16)
    x[T // 3], x[T // 2, n // 2:] = 0.0, 0.0
    q, s = code_buffers(T, n, fmt)
    with handle() as h:
        moe.moe_mx_quant(h, x, T, n, MODE[fmt], q, s)
        torch.cuda.synchronize()
        assert torch.all(q[T] == 0xEE) and torch.all(s[T] == 0xEE)
        # rows from everywhere, byte for byte
        at = [0, T // 2, T - 1] if n > 5000 else sorted({0, 1, T // 3, T // 2, T - 1, *np.random.default_rng(T).integers(0, T, 40).tolist()})
        codes, scales = ol.quantise(f64(x[at]), fmt)
        assert np.array_equal(q[at].cpu().numpy(), codes) and np.array_equal(s[at].cpu().numpy(), scales)
        # every row, as calls of at most 2 million elements give it
        q1, s1 = code_buffers(T, n, fmt)
        per = max(1, 2 ** 21 // n)
        for r in range(0, T, per):
            rows = min(per, T - r)
            qa, sa = code_buffers(rows, n, fmt)
            moe.moe_mx_quant(h, x[r:r + rows].clone(), rows, n, MODE[fmt], qa, sa)
            q1[r:r + rows], s1[r:r + rows] = qa[:rows], sa[:rows]
        torch.cuda.synchronize()
        assert torch.equal(q, q1) and torch.equal(s, s1)
        for t in ("f32", "bf16"):
            out = torch.full((T + 1, n), 7.0, dtype=TORCH[t], device="cuda")
            moe.moe_mx_values(h, MODE[fmt], q, s, T, n, TYPE[t], out)
            torch.cuda.synchronize()
            assert np.array_equal(f64(out[at]), ol.values(codes, scales, fmt)) and torch.all(out[T] == 7.0)
        assert moe.moe_lin_status(h) == moe.MOE_OK
