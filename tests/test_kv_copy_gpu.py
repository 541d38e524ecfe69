"""Copying pages in every layer's pool: every byte of the pools, and what is
left out."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from kv_setup import Pool, handle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("pages,n,layers,hkv,page,D", [
    (2, 1, 1, 1, 16, 32), (40, 17, 3, 2, 16, 64), (9, 4, 70, 1, 32, 96), (300, 150, 2, 5, 48, 128), (6, 2, 2, 8, 1024, 128),
    (5, 2, 1, 3, 496, 96)])
def test_copies_every_byte_of_every_layer(pages, n, layers, hkv, page, D, kv):
    rng = np.random.default_rng(pages + layers)
    pools = [Pool(pages, hkv, page, D, kv, rng) for _ in range(layers)]
    before = [p.bytes() for p in pools]
    order = rng.permutation(pages).astype(np.int32)
    dst = order[:n]
    src = order[n:][rng.integers(0, pages - n, n)]                   # one page may be copied to several
    pairs = torch.from_numpy(np.stack([src, dst], 1)).cuda()
    with handle(hkv, hkv, D, page, pages, 1, 1, kv) as h:
        moe.moe_kv_copy_pages(h, [p.struct for p in pools], pairs, n)
        assert moe.moe_kv_status(h) == moe.MOE_OK
    for p, b in zip(pools, before):
        for name, got in p.bytes().items():
            want = b[name].copy()
            want[dst] = b[name][src]
            assert np.array_equal(got, want), name


def test_bad_pairs_are_left_out_and_self_copies_do_nothing():
    rng = np.random.default_rng(0)
    p = Pool(8, 2, 16, 64, "e4m3", rng)
    b = p.bytes()
    pairs = torch.tensor([[0, 1], [8, 2], [-1, 3], [4, 8], [4, -2], [5, 5], [6, 7]], dtype=torch.int32, device="cuda")
    with handle(2, 2, 64, 16, 8, 1, 1, "e4m3") as h:
        moe.moe_kv_copy_pages(h, [p.struct], pairs, 7)
        assert moe.moe_kv_status(h) == moe.MOE_ERR_BAD_INDEX
    for name, got in p.bytes().items():
        want = b[name].copy()
        want[1], want[7] = want[0], want[6]
        assert np.array_equal(got, want), name


def test_refusals():
    rng = np.random.default_rng(0)
    p = Pool(4, 1, 16, 32, "bf16", rng)
    pairs = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    with handle(1, 1, 32, 16, 4, 1, 1) as h:
        def refused(pools=(p.struct,), pairs=pairs, n=1):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_kv_copy_pages(h, list(pools), pairs, n)
            assert e.value.code == moe.MOE_ERR_INVALID_ARG
        refused(n=-1), refused(n=5), refused(pairs=None), refused(pairs=pairs.data_ptr() + 2)
        refused(pools=[moe.kv_pool(p.dev["k"], None)]), refused(pools=[p.struct, moe.kv_pool(p.dev["k"].data_ptr() + 4, p.dev["v"])])
        moe.moe_kv_copy_pages(h, [p.struct], None, 0)
        moe.moe_kv_copy_pages(h, [], None, 0)
        assert moe.moe_kv_status(h) == moe.MOE_OK
