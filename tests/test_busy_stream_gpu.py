"""Handles made and used while torch's default stream is busy: torch's other
streams do not wait for it, and nothing of a handle may."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from busy_stream import busy_default_stream
from kv_setup import Pool, handle
from moe_setup import Layer, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


@pytest.mark.parametrize("path,T", [("slot", 1), ("slot", 4), ("group", 20)])
def test_a_new_ffn_handle_works_at_once(path, T):
    """The counters of the layer kernels are zero when the handle is there."""
    L = Layer(E=16, H=1024, I=448, k=6, max_tokens=32, path=path)
    s = torch.cuda.Stream()
    try:
        x, idx, w = inputs(T, 16, 1024, 6, seed=3)
        want = L.run(x, idx, w)
        xd = torch.from_numpy(x.view(np.int16)).cuda()
        it, wt = torch.from_numpy(np.ascontiguousarray(idx, np.int32)).cuda(), torch.from_numpy(np.ascontiguousarray(w, np.float32)).cuda()
        y = torch.empty_like(want)
        for _ in range(3):
            y.fill_(float("nan"))
            with busy_default_stream():
                h = moe.moe_ffn_create(L.cfg, 0)
                for _ in range(3):
                    moe.moe_ffn_forward(h, xd, it, wt, L.es.table, y, T, stream=s)
                s.synchronize()
            assert moe.moe_ffn_status(h, s) == moe.MOE_OK
            moe.moe_ffn_destroy(h)
            assert torch.equal(y, want)
    finally:
        torch.cuda.synchronize()
        L.close()


def test_the_cache_status_is_read_and_cleared_on_its_stream():
    """Errors set right after a status call are kept, and it waits for its own
    stream alone."""
    D, page = 64, 16
    p = Pool(1, 1, page, D, "bf16", np.random.default_rng(0))
    x = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    good, bad = (torch.tensor([n], dtype=torch.int32, device="cuda") for n in (0, page))     # beyond the row
    tab = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    with handle(1, 1, D, page, 1, 1, 1) as h:
        def append(pos):
            moe.moe_kv_append(h, p.struct, x, x, pos, tab, 1, stream=s)
        append(good)
        assert moe.moe_kv_status(h, s) == moe.MOE_OK
        with busy_default_stream():
            for _ in range(50):
                append(bad)
                assert moe.moe_kv_status(h, s) == moe.MOE_ERR_BAD_INDEX
            append(good)
            assert moe.moe_kv_status(h, s) == moe.MOE_OK


def test_the_ffn_status_is_read_and_cleared_on_its_stream():
    L = Layer(E=8, H=256, I=128, k=2, max_tokens=2)
    s = torch.cuda.Stream()
    try:
        x, idx, w = inputs(1, 8, 256, 2, seed=1)
        xd, wt = torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(np.ascontiguousarray(w, np.float32)).cuda()
        good = torch.from_numpy(np.ascontiguousarray(idx, np.int32)).cuda()
        bad = torch.full_like(good, 99)                              # no such expert
        y = torch.zeros((1, 256), dtype=torch.float32, device="cuda")

        def run(it):
            moe.moe_ffn_forward(L.h, xd, it, wt, L.es.table, y, 1, stream=s)
        torch.cuda.synchronize()
        run(good)
        assert moe.moe_ffn_status(L.h, s) == moe.MOE_OK
        with busy_default_stream():
            for _ in range(50):
                run(bad)
                assert moe.moe_ffn_status(L.h, s) == moe.MOE_ERR_BAD_INDEX
            run(good)
            assert moe.moe_ffn_status(L.h, s) == moe.MOE_OK
    finally:
        torch.cuda.synchronize()
        L.close()
