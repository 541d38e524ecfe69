"""The products' plans, on the host: they go by the figures of the handle's own
device, whatever other handles and threads do (no GPU)."""
import concurrent.futures as cf

import pytest

import fp4_block_scaled_gb300 as moe

E4M3, E2M1 = moe.MOE_ACT_E4M3_UE8M0_128, moe.MOE_ACT_E2M1_UE8M0_32
BF16, F32 = moe.MOE_OUT_BF16, moe.MOE_OUT_F32


def device(sms=152, pairs=None):
    """Figures of a device whose SMs lie in groups of 16 at most (clusters do not cross them)."""
    fit = [0, 0] + [sum(min(16, sms - g) // c for g in range(0, sms, 16)) for c in range(2, 9)]
    return moe.moe_lin_test_device(sms, pairs or fit[2], (moe.ctypes.c_int * 9)(*fit))


GB300 = moe.moe_lin_test_device(152, 76, (moe.ctypes.c_int * 9)(0, 0, 76, 46, 36, 28, 23, 15, 15))


def plan(dev, mode, T, N, K, out=BF16, bf16_rows=False):
    p = moe.moe_lin_test_plan(dev, mode, T, N, K, out, bf16_rows)
    return tuple(getattr(p, f) for f, _ in p._fields_)


SIZES = [(T, N, K) for T in (1, 7, 16, 40, 64, 130, 333, 1000, 3000, 9000) for N in (1, 200, 1024, 4099, 6144, 12288) for K in (32, 512, 2880, 4096, 8192)]


def test_a_plan_goes_by_its_own_devices_figures():
    """Handles of two devices, planning in turn and at once from many threads."""
    devs = [GB300, device(132), device(20), device(152, 40)]
    want = [[plan(d, m, *s) for m in (E4M3, E2M1) for s in SIZES] for d in devs]
    assert len({str(w) for w in want}) == len(devs)             # the figures count
    for i, s in enumerate(SIZES):                               # in turn
        for d, w in zip(devs, want):
            assert plan(d, E4M3, *s) == w[i]
    with cf.ThreadPoolExecutor(8) as ex:                        # at once
        jobs = [(w, ex.submit(lambda d=d: [plan(d, m, *s) for m in (E4M3, E2M1) for s in SIZES])) for _ in range(4) for d, w in zip(devs, want)]
        for w, j in jobs:
            assert j.result() == w


def test_refusals():
    for a in ((device(), 0, 1, 8, 32), (device(), E2M1, 0, 8, 32), (device(), E2M1, 1, 0, 32), (device(), E2M1, 1, 8, 48), (device(), E2M1, 1, 8, 32, 2),
              (moe.moe_lin_test_device(0, 1), E2M1, 1, 8, 32), (moe.moe_lin_test_device(1, 0), E2M1, 1, 8, 32)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_lin_test_plan(*a)
        assert e.value.code == moe.MOE_ERR_INVALID_ARG
    for a in ((2 ** 24 + 1, 8, 32), (1, 2 ** 24 + 1, 32), (1, 8, 2 ** 20 + 32)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_lin_test_plan(device(), E2M1, *a)
        assert e.value.code == moe.MOE_ERR_UNSUPPORTED


SM_SHARED, RESERVED = 228 * 1024, 1024       # of an SM, and of it for each CTA; a CTA takes at most 227 KB


def plans(dev):
    """The distinct plans over the range of sizes: every number of tokens up to a tile and around the tiles behind, features and
    reductions from one to many tiles and stages."""
    tokens = [*range(1, 200, 3), 16, 32, 64, 128, 192, *range(200, 1000, 37), *range(1000, 4400, 211), 5000, 16384, 70001]
    found = {}
    for m in (E4M3, E2M1):
        for N in (1, 129, 640, 1024, 2048, 4099, 6144, 12288, 40000):
            for K in (32, 256, 288, 512, 768, 1024, 1536, 2048, 2880, 4096, 8192, 32768):
                for T in tokens:
                    for out, bf16_rows in ((BF16, False), (F32, False), (BF16, True))[:3 if T <= 16 else 2]:
                        found.setdefault(plan(dev, m, T, N, K, out, bf16_rows), (m, T, N, K, out, bf16_rows))
    return found


@pytest.mark.parametrize("dev", [GB300, device(132), device(152, 70)], ids=["152", "132", "few_pairs"])
def test_shared_and_tensor_memory_of_every_plan(dev):
    """CTAs of clusters wait for one another's tensor memory without a limit of time, and those of two streams' products may
    meet on an SM.  Each has at least the share of its shared memory that it takes of the 512 columns, so that whatever fits the
    one fits the other; and none lies beside a pair's CTA, which takes every column, or beside a layer kernel's of 212 KB or
    more, which waits for its whole grid."""
    found = plans(dev)
    pairs = [p for p in found if p[0] == 0]
    split = [p for p in found if p[2] > 1]
    assert len(pairs) == 2 and len(split) > 100
    for p, at in found.items():
        tokens, tiles, cut, ring, smem, tmem = p
        assert 0 < smem <= 227 * 1024 and tmem in (32, 64, 128, 256, 512), at
        if tokens:
            assert tokens % 16 == 0 and tokens <= 192 and 3 <= ring <= 16 and 1 <= cut <= 8, at
        if cut > 1:
            assert (smem + RESERVED) * 512 >= SM_SHARED * tmem, at
            assert tiles * cut <= dev.sms
            for other in [q[4] for q in pairs] + [212 * 1024]:
                assert smem + other + 2 * RESERVED > SM_SHARED, at


@pytest.mark.parametrize("dev", [GB300, device(132)], ids=["152", "132"])
def test_clusters_run_at_once(dev):
    """A tile that is cut along K has a cluster of its own, and the costs by which it is cut count one round of them."""
    found = [(p, at) for p, at in plans(dev).items() if p[2] > 1]
    assert len(found) > 100
    for (tokens, tiles, cut, ring, smem, tmem), at in found:
        assert tiles <= dev.clusters[cut] * (SM_SHARED // (smem + RESERVED)), at
