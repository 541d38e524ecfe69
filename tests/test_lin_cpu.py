"""The formulas of the norms and projections against what pins them, and the
calls' refusals that need no handle (no GPU)."""
import ctypes
import os
import re

import numpy as np
import pytest

import fp4_block_scaled_gb300 as moe
import oracle
from conftest import ROOT
from oracle import lin as ol


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_lin.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_\w+)\s*\(", src)))
    assert names == sorted(moe.LIN_EXPORTS) and all(hasattr(moe.lib(), n) for n in names)


@pytest.mark.parametrize("fmt,n", [("e2m1", 32), ("e2m1", 160), ("e4m3", 128), ("e4m3", 160)])
def test_quantisation_is_that_of_the_expert_layers(fmt, n):
    rng = np.random.default_rng(n)
    x = ol.bf16_rne(rng.standard_normal((20, n)) * 2.0 ** rng.integers(-20, 20, (20, 1)))
    x[3] = 0.0
    x[4, ::3] = -0.0
    x[5, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]         # halfway between codes
    x[5, 8:] = 0.5
    codes, scales = ol.quantise(x, fmt)
    block = 32 if fmt == "e2m1" else 128
    for r in range(len(x)):
        if fmt == "e2m1":
            q, s = oracle.act_quant_e2m1(x[r])[:2]
            q = np.asarray(q).reshape(-1)
            q = q if q.size == n // 2 else (q[0::2] | q[1::2] << 4)
        else:
            q, s = oracle.act_quant_e4m3(x[r])[:2]
        assert np.array_equal(codes[r], np.asarray(q, np.uint8).reshape(-1)) and np.array_equal(scales[r], np.asarray(s, np.uint8).reshape(-1))
    v = ol.values(codes, scales, fmt)
    # half a step of the block's grid, of which the largest element has at least a quarter (E4M3: an eighth) of the range
    amax = np.repeat(np.abs(np.pad(x, ((0, 0), (0, -n % block)))).reshape(20, -1, block).max(-1), block, -1)[:, :n]
    assert np.all(np.abs(v - x) <= (amax / 3 if fmt == "e2m1" else np.maximum(np.abs(x) * 2.0 ** -4, amax * 2.0 ** -16)))


def test_bf16_rounding():
    x = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -30, -3.14159, 0.0, 1e-20])
    assert np.array_equal(ol.bf16_rne(x), [oracle.bf16_value(oracle.bf16_rne(float(v))) for v in x])


def test_packed_sizes():
    unit = 128 * 128 + 2 * 512
    for n, k, want in [(1, 32, 1), (128, 256, 1), (129, 256, 2), (6144, 4096, 48 * 16), (4099, 2880, 33 * 12)]:
        assert moe.moe_linear_packed_bytes(n, k) == want * unit
    for n, k in [(0, 32), (-1, 32), (8, 0), (8, 16), (8, 48), (8, -32), (8, 2 ** 20 + 32), (2 ** 24 + 1, 32)]:
        assert moe.moe_linear_packed_bytes(n, k) == 0


def test_null_handles_and_bad_configs_are_refused():
    L, bad = moe.lib(), moe.MOE_ERR_INVALID_ARG
    h = ctypes.c_void_p()
    for c in [moe.lin_config(-1, 0), moe.lin_config(0, -32), moe.lin_config(1, 33)]:
        assert L.moe_lin_create(ctypes.byref(h), ctypes.byref(c), 0) == bad and h.value is None
    for c in [moe.lin_config(2 ** 24 + 1, 32), moe.lin_config(1, 2 ** 20 + 32)]:
        assert L.moe_lin_create(ctypes.byref(h), ctypes.byref(c), 0) == moe.MOE_ERR_UNSUPPORTED
    assert L.moe_lin_create(None, ctypes.byref(moe.lin_config()), 0) == bad
    assert L.moe_lin_create(ctypes.byref(h), None, 0) == bad
    assert L.moe_lin_status(None, None) == bad
    d, w = moe.norm(None, 32, 1e-6), moe.linear(256, 8, 32)
    assert L.moe_rms_norm(None, ctypes.byref(d), 256, None, 0, None, None, 0, None, None, None) == bad
    assert L.moe_mx_quant(None, 256, 0, 32, 2, 512, 1024, None) == bad
    assert L.moe_mx_values(None, 2, 256, 512, 0, 32, 0, 1024, None) == bad
    assert L.moe_linear_pack(None, 256, 512, 8, 32, 1024, None) == bad
    assert L.moe_linear(None, ctypes.byref(w), 2, 256, None, 0, 512, 0, None) == bad
    L.moe_lin_destroy(None)
    words = (ctypes.c_int64 * 16)()
    assert L.moe_lin_call(7, ctypes.cast(words, ctypes.c_char_p)) == bad and L.moe_lin_call(0, None) == bad
    for op, at in ((0, 4), (1, 2), (2, 4), (3, 5)):             # a count that an int does not hold
        words = (ctypes.c_int64 * 16)()
        words[at] = 2 ** 31
        assert L.moe_lin_call(op, ctypes.cast(words, ctypes.c_char_p)) == bad
