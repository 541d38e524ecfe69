"""The norms' and projections' calls on streams and in graphs: first calls
captured, a packed layer's first product, handles at work at once, a handle made
beside a busy default stream, weights that change between calls."""
import time

import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from busy_stream import busy_default_stream
from lin_setup import MODE, TYPE, Weights, code_buffers, f64, handle, rand
from oracle import lin as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


class Step:
    """A norm with codes, the product of the codes, and the product of bf16 rows that the call quantises."""

    def __init__(self, h, T, K, N, fmt, seed):
        rng = np.random.default_rng(seed)
        self.T, self.K, self.N, self.fmt = T, K, N, fmt
        self.w = Weights(h, N, K, rng)
        self.x, self.res = rand(rng, (T, K)).to(torch.bfloat16), rand(rng, (T, K), 3.0)
        self.g = (1 + 0.2 * rand(rng, (K,))).to(torch.bfloat16)
        self.norm = moe.norm(self.g, K, 1e-5, TYPE["bf16"], TYPE["f32"])
        self.u, self.res_out = torch.zeros_like(self.x), torch.zeros_like(self.res)
        self.q, self.s = code_buffers(T, K, fmt)
        self.y, self.z = (torch.zeros((T, N), dtype=torch.float32, device="cuda") for _ in range(2))
        torch.cuda.synchronize()

    def run(self, h, st=None):
        m = MODE[self.fmt]
        moe.moe_rms_norm(h, self.norm, self.x, self.T, residual=self.res, residual_out=self.res_out, out=self.u, act_mode=m,
                         codes=self.q, scales=self.s, stream=st)
        moe.moe_linear(h, self.w.desc, m, self.q, self.T, self.y, TYPE["f32"], x_scales=self.s, stream=st)
        moe.moe_linear(h, self.w.desc, m, self.u, self.T, self.z, TYPE["f32"], stream=st)

    def check(self):
        T = self.T
        ref, total = ol.linear(ol.values(self.q[:T].cpu().numpy(), self.s[:T].cpu().numpy(), self.fmt), self.w.values())
        assert np.all(np.abs(f64(self.y) - ref) <= ol.linear_tolerance(self.K, total))
        assert torch.equal(self.y, self.z)
        want = ol.norm(f64(self.x.float() + self.res), f64(self.g), 1e-5)
        assert np.all(np.abs(f64(self.u) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -19))


SIZES = [(1, 1024, 768), (4, 4096, 384), (40, 2880, 500), (150, 512, 4096), (700, 1056, 520)]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_a_handles_first_calls_may_be_captured(fmt, T, K, N):
    st = torch.cuda.Stream()
    with handle(T, K) as h0:
        a = Step(h0, T, K, N, fmt, T)
        with handle(T, K) as h:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                a.run(h, st)
            assert not a.y.any()                                     # nothing ran yet
            for i in range(3):
                a.x.copy_(torch.randn_like(a.x))
                a.y.fill_(float("nan")), a.z.fill_(float("nan"))
                torch.cuda.synchronize()
                with torch.cuda.stream(st):
                    g.replay()
                st.synchronize()
                a.check()
            assert moe.moe_lin_status(h, st) == moe.MOE_OK


def test_handles_at_work_at_once():
    st = [torch.cuda.Stream() for _ in SIZES]
    hs = [moe.moe_lin_create(moe.lin_config(T, K), 0) for T, K, _ in SIZES]
    steps = [Step(h, *c, "e2m1" if i % 2 else "e4m3", i) for i, (h, c) in enumerate(zip(hs, SIZES))]
    for h, a in zip(hs, steps):
        a.run(h)
    torch.cuda.synchronize()
    want = [a.y.clone() for a in steps]
    for a in steps:
        a.check()
    for _ in range(10):
        for a in steps:
            a.y.zero_(), a.z.zero_()
        torch.cuda.synchronize()
        for _ in range(8):
            for h, a, s in zip(hs, steps, st):
                a.run(h, s)
        torch.cuda.synchronize()
        for a, y in zip(steps, want):
            assert torch.equal(a.y, y) and torch.equal(a.z, y)
    for h in hs:
        assert moe.moe_lin_status(h) == moe.MOE_OK
        moe.moe_lin_destroy(h)


def test_products_one_after_another_see_each_others_outputs():
    """A chain whose kernels overlap: each product's rows are what the one before wrote."""
    rng = np.random.default_rng(3)
    for T, fmt in ((1, "e2m1"), (3, "e4m3"), (16, "e2m1"), (60, "e4m3"), (300, "e2m1")):
        with handle(T, 512) as h:
            ws = [Weights(h, 512, 512, rng, 118, 121) for _ in range(6)]
            x = [rand(rng, (T, 512)).to(torch.bfloat16)] + [torch.zeros((T, 512), dtype=torch.bfloat16, device="cuda") for _ in ws]
            torch.cuda.synchronize()
            for _ in range(20):
                for w, a, b in zip(ws, x, x[1:]):
                    moe.moe_linear(h, w.desc, MODE[fmt], a, T, b, TYPE["bf16"])
            torch.cuda.synchronize()
            for w, a, b in zip(ws, x, x[1:]):
                y = torch.zeros_like(b)
                moe.moe_linear(h, w.desc, MODE[fmt], a, T, y, TYPE["bf16"])
                torch.cuda.synchronize()
                assert torch.equal(y, b) and y.any()
                q, s = ol.quantise(f64(a), fmt)
                ref, total = ol.linear(ol.values(q, s, fmt), w.values())
                tol = ol.linear_tolerance(512, total)
                assert np.all(np.abs(f64(b) - ref) <= tol + (np.abs(ref) + tol) * 2.0 ** -8)


@pytest.mark.parametrize("T", [1, 30, 700])
def test_weights_packed_or_copied_just_before(T):
    """The product reads weights before the kernel ahead of it is done: not before a packing or a copy is."""
    rng = np.random.default_rng(4)
    K, N = 2048, 1024
    with handle(T, K) as h:
        a, b = Weights(h, N, K, rng), Weights(h, N, K, rng)
        x = rand(rng, (T, K)).to(torch.bfloat16)
        want = []
        for w in (a, b):
            y = torch.zeros((T, N), dtype=torch.float32, device="cuda")
            moe.moe_linear(h, w.desc, MODE["e2m1"], x, T, y, TYPE["f32"])
            want.append(y)
        torch.cuda.synchronize()
        packed = torch.zeros_like(a.packed)
        d, y = moe.linear(packed, N, K), torch.zeros((T, N), dtype=torch.float32, device="cuda")
        st = torch.cuda.Stream()
        copies = [w.packed.clone() for w in (a, b)]
        u = torch.zeros_like(x)
        norm = moe.norm(None, K, 1e-6)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for i in range(30):
                w, k = (a, b)[i % 2], i % 2
                if i % 4 < 2:
                    moe.moe_linear_pack(h, *w.dev, N, K, packed, stream=st)
                else:
                    packed.copy_(copies[k])
                if i % 3 == 0:                                       # a kernel between that lets its dependents launch early
                    moe.moe_rms_norm(h, norm, x, T, out=u, stream=st)
                moe.moe_linear(h, d, MODE["e2m1"], x, T, y, TYPE["f32"], stream=st)
                got = y.clone()
                st.synchronize()
                assert torch.equal(got, want[k]), i


def test_a_new_handle_works_at_once_on_a_stream_beside_a_busy_default_one():
    T, K, N = 70, 1024, 384
    st = torch.cuda.Stream()
    with handle(T, K) as h0:
        a = Step(h0, T, K, N, "e4m3", 5)
        a.run(h0, st)
        torch.cuda.synchronize()
        for _ in range(2):
            a.y.fill_(float("nan")), a.z.fill_(float("nan"))
            with busy_default_stream():
                h = moe.moe_lin_create(moe.lin_config(T, K), 0)
                for _ in range(3):
                    a.run(h, st)
                st.synchronize()
                assert moe.moe_lin_status(h, st) == moe.MOE_OK
            moe.moe_lin_destroy(h)
            a.check()


@pytest.mark.parametrize("T,K,N", [(1, 4096, 6144), (16, 2048, 256), (100, 512, 30000), (150, 4096, 1024), (5000, 1056, 520)])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_waits_that_run_out_end_the_call(fmt, T, K, N):
    """A report that never comes: every wait that follows from it gives up, the call ends at once, says so, and the next
    one is right.  (One tile cut along K, two, tiles taken in turn, and pairs of CTAs.)"""
    rng = np.random.default_rng(6)
    with handle(T, K) as h:
        w = Weights(h, N, K, rng)
        x = rand(rng, (T, K)).to(torch.bfloat16)
        q, s = code_buffers(T, K, fmt)
        moe.moe_mx_quant(h, x, T, K, MODE[fmt], q, s)
        y, want = (torch.zeros((T, N), dtype=torch.float32, device="cuda") for _ in range(2))
        call = lambda out, **kw: moe.moe_linear(h, w.desc, MODE[fmt], kw.get("x", q), T, out, TYPE["f32"], x_scales=kw.get("s", s))  # noqa: E731
        call(want)
        assert moe.moe_lin_status(h) == moe.MOE_OK
        for kw in ({}, dict(x=x, s=None)):
            moe.moe_lin_test_set_wait(h, 1000000, True)
            t = time.perf_counter()
            call(y, **kw)
            assert moe.moe_lin_status(h) == moe.MOE_ERR_DEVICE_TIMEOUT
            assert time.perf_counter() - t < 1.0
            moe.moe_lin_test_set_wait(h, 0, False)
            for _ in range(2):
                y.fill_(float("nan"))
                call(y, **kw)
                assert moe.moe_lin_status(h) == moe.MOE_OK and torch.equal(y, want)
        with pytest.raises(moe.MoeError):
            moe.moe_lin_test_set_wait(h, 2000000001, False)
