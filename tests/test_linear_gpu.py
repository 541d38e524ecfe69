"""moe_linear against the fp64 product of what codes and scales stand for: one
token to many, features and reductions that fill no tile, both formats, both
output types, split and persistent forms, scales at their ends, refusals."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from lin_setup import MODE, TORCH, TYPE, Weights, code_buffers, f64, handle, rand
from oracle import lin as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


def rows(h, T, K, fmt, rng):
    """bf16 rows, and their codes and scales."""
    x = (rand(rng, (T, K)) * torch.exp2(torch.from_numpy(rng.integers(-3, 4, (T, 1))).float().cuda())).to(torch.bfloat16)
    q, s = code_buffers(T, K, fmt)
    moe.moe_mx_quant(h, x, T, K, MODE[fmt], q, s)
    torch.cuda.synchronize()
    return x, q[:T], s[:T]


def product(h, w, fmt, x, T, out="f32", scales=None):
    y = torch.full((T + 1, w.N), 7.0, dtype=TORCH[out], device="cuda")
    moe.moe_linear(h, w.desc, MODE[fmt], x, T, y, TYPE[out], x_scales=scales)
    torch.cuda.synchronize()
    assert moe.moe_lin_status(h) == moe.MOE_OK
    assert torch.all(y[T] == 7.0)
    return y[:T]


def check(y, q, s, w, fmt, out="f32", some=None):
    at = np.arange(len(y)) if some is None else np.asarray(some)
    ref, total = ol.linear(ol.values(q.cpu().numpy()[at], s.cpu().numpy()[at], fmt), w.values())
    tol = ol.linear_tolerance(w.K, total)
    if out == "bf16":
        tol = tol + (np.abs(ref) + tol) * 2.0 ** -8
    assert np.all(np.abs(f64(y)[at] - ref) <= tol)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T,K,N", [
    (1, 32, 1), (1, 64, 64), (2, 96, 127), (1, 256, 128), (3, 288, 129), (1, 4096, 640), (7, 2880, 384), (16, 4096, 1000), (17, 1024, 256),
    (33, 512, 257), (64, 2080, 4096), (100, 160, 130), (130, 2880, 384), (200, 4096, 512), (257, 4096, 128), (333, 2880, 4099), (800, 544, 96),
    (2000, 256, 1000), (4200, 64, 1), (4500, 96, 24), (4097, 1056, 258)])
def test_sizes(fmt, T, K, N):
    rng = np.random.default_rng([T, K, N])
    with handle(T, K) as h:
        w = Weights(h, N, K, rng)
        x, q, s = rows(h, T, K, fmt, rng)
        y = product(h, w, fmt, q, T, scales=s)
        check(y, q, s, w, fmt)
        # the quantisation inside the call, and the rounding of the output
        assert torch.equal(product(h, w, fmt, x, T), y)
        assert torch.equal(product(h, w, fmt, x, T, "bf16"), y.to(torch.bfloat16))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_token_counts_around_the_tiles(fmt):
    rng = np.random.default_rng(5)
    K, N = 512, 200
    with handle() as h:
        w = Weights(h, N, K, rng)
        _, q, s = rows(h, 600, K, fmt, rng)
        for T in (1, 8, 15, 16, 31, 32, 48, 63, 65, 127, 128, 129, 191, 192, 193, 383, 384, 385, 577):
            check(product(h, w, fmt, q, T, scales=s), q[:T], s[:T], w, fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("K,N", [(96, 40), (512, 200), (1440, 384), (4096, 1024), (2048, 30000)])
def test_few_bf16_rows_are_quantised_alike(fmt, K, N):
    """In the product's kernel or ahead of it: the codes' product bit for bit, whichever sizes take which."""
    rng = np.random.default_rng([K, N])
    with handle(20, K) as h:
        w = Weights(h, N, K, rng)
        x, q, s = rows(h, 20, K, fmt, rng)
        for T in (1, 2, 3, 4, 5, 7, 8, 9, 13, 15, 16, 17, 20):
            assert torch.equal(product(h, w, fmt, x, T), product(h, w, fmt, q, T, scales=s)), T


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T", [300, 4229])
def test_outputs_of_any_row_length(fmt, T):
    """Rows of y that begin on any element; on pairs of CTAs, which do not cut K, the same sums of each feature."""
    rng = np.random.default_rng(21)
    K, N = 160, 584
    with handle(20, K) as h:
        w = Weights(h, N, K, rng)
        _, q, s = rows(h, T, K, fmt, rng)
        whole = product(h, w, fmt, q, T, scales=s)
        check(whole, q, s, w, fmt)
        for n in (1, 3, 6, 31, 34, 66, 253, 255, 257, 260, 322, 513, 577, 578, 579, 580, 581, 582, 583):
            part = Weights(h, n, K, rng)
            part.codes, part.scales = w.codes[:n].copy(), w.scales[:n].copy()
            part.pack(h)
            for out in ("f32", "bf16"):
                y = product(h, part, fmt, q, T, out, scales=s)
                if T > 4096:
                    assert torch.equal(y, whole[:, :n].to(TORCH[out])), (n, out)
                else:
                    check(y, q, s, part, fmt, out)


@pytest.mark.parametrize("T", [1, 2, 5, 20, 300, 4229])
def test_rows_of_scales_of_any_length(T):
    """Rows of scales that begin on any byte: each keeps its own, up to the array's last."""
    rng = np.random.default_rng(22)
    N = 40
    with handle(20) as h:
        for K in (32, 64, 96, 128, 160, 224, 288, 480, 736, 1056):
            w = Weights(h, N, K, rng)
            q = torch.from_numpy(rng.integers(0, 256, (T, K // 2), dtype=np.uint8)).cuda()
            room = torch.full((T * (K // 32) + 64,), 255, dtype=torch.uint8, device="cuda")
            s = room[:T * (K // 32)].view(T, K // 32)
            s.copy_(torch.from_numpy(rng.integers(117, 124, (T, K // 32), dtype=np.uint8)))
            check(product(h, w, "e2m1", q, T, scales=s), q, s, w, "e2m1")
            # a scale of NaN at each end of every third row
            s[1::3, 0] = 255
            s[2::3, -1] = 255
            bad = torch.zeros(T, dtype=torch.bool, device="cuda")
            bad[1::3], bad[2::3] = True, True
            y = product(h, w, "e2m1", q, T, scales=s)
            assert torch.equal(torch.isnan(y), bad[:, None].expand(T, N)), K


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_repeats_are_equal_bit_for_bit(fmt):
    rng = np.random.default_rng(6)
    with handle() as h:
        for T, K, N in ((5, 4096, 512), (300, 1440, 700)):
            w = Weights(h, N, K, rng)
            _, q, s = rows(h, T, K, fmt, rng)
            y = product(h, w, fmt, q, T, scales=s)
            for _ in range(5):
                assert torch.equal(product(h, w, fmt, q, T, scales=s), y)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("T", [3, 150])
def test_scales_of_nan_stay_in_their_row_and_feature(fmt, T):
    rng = np.random.default_rng(7)
    K, N = 608, 300
    with handle() as h:
        w = Weights(h, N, K, rng)
        w.scales[170, 11] = 255
        w.pack(h)
        _, q, s = rows(h, T, K, fmt, rng)
        s[1, 2] = 255
        y = product(h, w, fmt, q, T, scales=s)
        bad = torch.zeros((T, N), dtype=torch.bool, device="cuda")
        bad[1], bad[:, 170] = True, True
        assert torch.equal(torch.isnan(y), bad)
        ref, total = ol.linear(np.nan_to_num(ol.values(q.cpu().numpy(), s.cpu().numpy(), fmt)), np.nan_to_num(w.values()))
        ok = ~bad.cpu().numpy()
        assert np.all(np.abs(f64(y) - ref)[ok] <= ol.linear_tolerance(K, total)[ok])


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_scales_far_from_one(fmt):
    """Bytes that would overflow or vanish alone and not in their product."""
    rng = np.random.default_rng(8)
    T, K, N = 20, 256, 128
    with handle() as h:
        for wl, xb in ((20, 230), (225, 25), (127, 127)):
            w = Weights(h, N, K, rng, wl, wl + 5)
            _, q, _ = rows(h, T, K, fmt, rng)
            s = torch.full((T, K // (32 if fmt == "e2m1" else 128)), xb, dtype=torch.uint8, device="cuda")
            check(product(h, w, fmt, q, T, scales=s), q, s, w, fmt)


def test_places_beyond_32_bits():
    rng = np.random.default_rng(9)
    T, K, N = 70001, 64, 32000                                   # 2.24e9 outputs
    with handle() as h:
        w = Weights(h, N, K, rng)
        _, q, s = rows(h, T, K, "e2m1", rng)
        y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        moe.moe_linear(h, w.desc, MODE["e2m1"], q, T, y, TYPE["bf16"], x_scales=s)
        torch.cuda.synchronize()
        assert moe.moe_lin_status(h) == moe.MOE_OK
        at = [0, 1, 33553, 67108, 67109, 70000]
        check(y[at], q[at], s[at], w, "e2m1", "bf16")


def test_long_reductions_and_many_features():
    rng = np.random.default_rng(10)
    with handle() as h:
        for T, K, N in ((2, 131072, 128), (1, 64, 100000)):
            for fmt in ("e2m1", "e4m3"):
                w = Weights(h, N, K, rng)
                _, q, s = rows(h, T, K, fmt, rng)
                check(product(h, w, fmt, q, T, scales=s), q, s, w, fmt)


def test_refusals():
    rng = np.random.default_rng(11)
    with handle(8, 64) as h:
        w = Weights(h, 100, 64, rng)
        x, q, s = rows(h, 9, 64, "e2m1", rng)
        y = torch.zeros((9, 100), dtype=torch.float32, device="cuda")

        def refused(desc=w.desc, mode=MODE["e2m1"], x=q, T=4, y=y, out=TYPE["f32"], scales=s, code=moe.MOE_ERR_INVALID_ARG):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_linear(h, desc, mode, x, T, y, out, x_scales=scales)
            assert e.value.code == code
        refused(mode=0), refused(mode=3), refused(out=2), refused(T=-1), refused(x=None), refused(y=None)
        refused(T=2 ** 24 + 1, code=moe.MOE_ERR_UNSUPPORTED)
        for d in (moe.linear(None, 100, 64), moe.linear(w.packed, 0, 64), moe.linear(w.packed, -5, 64), moe.linear(w.packed, 100, 48),
                  moe.linear(w.packed, 100, 0), moe.linear(w.packed.data_ptr() + 64, 100, 64)):
            refused(desc=d)
        refused(desc=moe.linear(w.packed, 100, 2 ** 20 + 32), code=moe.MOE_ERR_UNSUPPORTED)
        refused(x=q.data_ptr() + 8), refused(scales=s.data_ptr() + 4), refused(y=y.data_ptr() + 4)
        refused(y=q), refused(y=s), refused(y=w.packed)
        refused(x=x, scales=None, T=9)                              # more bf16 rows than the handle's workspace holds
        wide = Weights(h, 4, 96, rng)
        refused(desc=wide.desc, x=x, scales=None)
        moe.moe_linear(h, w.desc, MODE["e2m1"], None, 0, None, TYPE["f32"])
        for a in ((None, w.dev[1], 100, 64, w.packed), (w.dev[0], None, 100, 64, w.packed), (*w.dev, 0, 64, w.packed), (*w.dev, 100, 40, w.packed),
                  (*w.dev, 100, 64, None), (*w.dev, 100, 64, w.packed.data_ptr() + 16), (*w.dev, 100, 64, w.dev[0])):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_linear_pack(h, *a)
            assert e.value.code == moe.MOE_ERR_INVALID_ARG
        assert moe.moe_lin_status(h) == moe.MOE_OK


def test_a_failed_allocation_is_reported():
    moe.moe_ffn_test_fail_allocs(1)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_lin_create(moe.lin_config(4, 64), 0)
    moe.moe_ffn_test_fail_allocs(0)
    assert e.value.code == moe.MOE_ERR_OOM
