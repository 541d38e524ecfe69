"""Attention of one token over the paged cache against fp64, at the lengths,
heads, pages and masks where it can go wrong."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from kv_setup import Pool, bf16_of, check_attention, f64, handle, table
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


def _run(lens, hq, hkv, D, page, kv="bf16", out="f32", scale=0.0, softcap=0.0, window=0, row=None, share=(), seed=0,
         extra=2, spread=0.0, edit=None, status=moe.MOE_OK, lse=True, check=True, qscale=1.5):
    rng = np.random.default_rng(seed + sum(lens) + D + hq)
    B = len(lens)
    row = row or max(1, max(-(-max(n, 0) // page) for n in lens))
    pages = sum(-(-max(n, 0) // page) for n in lens) + extra
    tab = table(lens, page, pages, row, rng, share)
    p = Pool(pages, hkv, page, D, kv, rng, spread=spread)
    if edit:
        edit(p, tab)
        p.upload()
    qb = bf16_of(qscale * rng.standard_normal((B, hq, D)))
    q = torch.from_numpy(qb).cuda()
    ld, td = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(tab).cuda()
    dt = torch.float32 if out == "f32" else torch.bfloat16
    o = torch.full((B + 1, hq, D), 5.0, dtype=dt, device="cuda")
    ls = torch.full((B + 1, hq), 5.0, dtype=torch.float32, device="cuda")
    with handle(hq, hkv, D, page, pages, B, row, kv, out) as h:
        for again in range(2):
            moe.moe_attn_decode(h, p.struct, q, ld, td, B, o, lse=ls if lse else None, scale=scale, softcap=softcap,
                                window=window)
            torch.cuda.synchronize()
            if again:
                assert torch.equal(o.view(torch.int16), keep.view(torch.int16)), "two runs differ"
            keep = o.clone()
        assert moe.moe_kv_status(h) == status
    assert torch.all(o[B] == 5.0) and torch.all(ls[B] == 5.0)        # behind the last sequence
    if check:
        check_attention(p, okv.bf16(qb), lens, tab, page, f64(o[:B]), f64(ls[:B]) if lse else None,
                        scale or D ** -0.5, softcap, window, out == "bf16")
    return f64(o[:B]), f64(ls[:B])


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (6, 2), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (24, 2), (40, 1), (10, 5)])
def test_heads_and_lengths(hq, hkv, kv):
    _run(LENS, hq, hkv, 128, 16, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_very_many_query_heads(kv):
    _run([0, 5, 40, 300], 512, 1, 64, 16, kv)
    _run([33, 1], 512, 512, 32, 16, kv)


@pytest.mark.parametrize("kv,D", [("bf16", d) for d in (16, 32, 48, 64, 80, 96, 112, 128)] +
                         [("e4m3", d) for d in (32, 64, 96, 128)])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (12, 1)])
def test_head_sizes(D, kv, hq, hkv):
    _run(LENS, hq, hkv, D, 32, kv, out="bf16")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 1024])
def test_pages(page, kv):
    _run([1, page - 1, page, page + 1, 3 * page + 5, 2 * page], 8, 2, 64, page, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[20000], [5000, 3, 0, 12345, 1], [4096] * 3], ids=["one", "ragged", "even"])
def test_long_caches_are_split_and_joined(lens, kv):
    _run(lens, 8, 2, 128, 64, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,D", [(8, 128), (32, 64)])
def test_fp32_outputs_of_long_rows_do_not_drift(hq, D, kv):
    """Rows of 6000 keys that one warp sums nearly alone (more rows than the
    machine has warps), against fp64 on the device.

    Bound on a row's relative norm: scores off by sqrt(D) 2^-24 of the products'
    size (scale sum |q k| is about 1.5 sqrt(D) 2 / pi < 11 here) and 2^-21, twice; weights
    2^-21; the tiles' sums added to the row's, 188 roundings at most, sqrt(188) 2^-24:
    below 2^-18 in all, where sums cut to 24 bits at every product of 16 keys
    would drift by up to 375 * 2^-24 = 2^-15.4."""
    B, n, hkv, page = 160, 6000, 8, 64
    row = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(D + hq)
    pages = 200                                                      # all sequences share them, in different orders
    k, v = (torch.randn((pages, hkv, page, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    v = v + 1.0                                                      # sums that grow
    tab = torch.stack([torch.randperm(pages, generator=g, device="cuda")[:row] for _ in range(B)]).to(torch.int32)
    q = (1.5 * torch.randn((B, hq, D), generator=g, device="cuda")).to(torch.bfloat16)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    if kv == "bf16":
        pool, kd, vd = moe.kv_pool(k, v), k.double(), v.double()
    else:
        kc, vc = k.float().to(torch.float8_e4m3fn), v.float().to(torch.float8_e4m3fn)
        s = torch.full((pages, hkv, page), 127, dtype=torch.uint8, device="cuda")
        pool, kd, vd = moe.kv_pool(kc, vc, s, s), kc.double(), vc.double()
    out = torch.empty((B, hq, D), dtype=torch.float32, device="cuda")
    with handle(hq, hkv, D, page, pages, B, row, kv, "f32") as h:
        moe.moe_attn_decode(h, pool, q, lens, tab, B, out)
        assert moe.moe_kv_status(h) == moe.MOE_OK
    worst = 0.0
    for b in range(0, B, 7):
        kb, vb = (x[tab[b].long()].transpose(0, 1).reshape(hkv, -1, D)[:, :n] for x in (kd, vd))
        z = q[b].double().view(hkv, hq // hkv, D) @ kb.transpose(1, 2) / D ** 0.5
        ref = (torch.softmax(z, -1) @ vb).view(hq, D)
        worst = max(worst, float(((out[b].double() - ref).norm(dim=-1) / ref.norm(dim=-1)).max()))
    assert worst <= 2.0 ** -18, worst


@pytest.mark.parametrize("hq", [8, 16])
def test_many_short_sequences(hq):
    _run([(i * 37) % 50 for i in range(300)], hq, 2, 64, 16)


def test_no_keys_at_all():
    out, lse = _run([0, 0, 0], 8, 2, 64, 16)
    assert not out.any() and np.isneginf(lse).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,D", [(16, 128), (48, 64)])
def test_short_rows_stay_whole_between_long_ones(hq, D, kv):
    """Enough short sequences that none of them is split, with long ones that
    are between them, at the ends and next to each other."""
    lens = [(i * 37) % 131 for i in range(330)]
    lens[0], lens[100], lens[101], lens[200], lens[329] = 3000, 2100, 129, 128, 2500
    _run(lens, hq, 4, D, 32, kv, window=0)


FEW = {  # rows with CTAs of their own, on both sides of what one takes; more rows than CTAs with little to do
    "two_heads": ([511, 512, 513, 1, 0, 1023, 1024, 1025, 256, 257], 2),
    "one_sequence": ([1300], 8),
    "past_a_warp": ([(i * 97) % 500 for i in range(40)] + [1030, 1024, 1025], 2),
    "most_rows": ([(i * 89) % 300 for i in range(147)] + [513, 0, 1040], 1),
    "between": ([(i * 37) % 60 for i in range(60)] + [700, 0, 33, 515, 1], 4),
    "between_in_a_warp": ([(i * 37) % 60 for i in range(29)] + [700, 0, 515], 8),
}


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(FEW))
def test_few_rows(name, D, kv):
    lens, hkv = FEW[name]
    _run(lens, 4 * hkv, hkv, D, 32, kv)
    _run(lens, 4 * hkv, hkv, D, 32, kv, window=200)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 1000])
def test_window(window, kv):
    _run(LENS + [1500], 8, 2, 64, 16, kv, window=window)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("softcap,scale,window", [(30.0, 0.0, 0), (2.0, 0.5, 0), (50.0, 0.0, 33), (0.0, -0.3, 0), (0.0, 1e-3, 0)])
def test_softcap_and_scale(softcap, scale, window, hq):
    _run(LENS, hq, 2, 64, 16, softcap=softcap, scale=scale, window=window)


def test_large_scores_and_scales_far_apart():
    # scores in the hundreds: one key takes nearly all the weight, late maxima rescale what came before
    _run(LENS + [3000], 8, 2, 128, 16, qscale=60.0)
    # cached rows between 2^-40 and 2^25 in one sequence
    _run(LENS + [3000], 8, 2, 64, 16, "e4m3", spread=5.0, qscale=1e-3)


def test_shared_pages_and_no_lse():
    _run([100, 90, 70, 33], 8, 2, 64, 16, share=[(0, 1, 5), (0, 2, 4), (1, 3, 2)], lse=False)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_what_lies_behind_the_last_key_is_never_used(kv):
    """Every row that no key of a sequence has is NaN (codes and scales too):
    the rest of the last pages, the pages of nobody, keys outside the window."""
    lens, page, window = [1, 17, 40, 64, 0], 16, 20

    def poison(p, tab):
        keep = np.zeros((p.k.shape[0], page), bool)
        for b, n in enumerate(lens):
            for j in range(max(0, n - window), n):
                keep[tab[b, j // page], j % page] = True
        bad = np.where(keep[:, None, :, None], 0, 1).astype(bool) & np.ones(p.k.shape, bool)
        for a, nan in ((p.k, np.int16(0x7FC0) if kv == "bf16" else 0x7F), (p.v, np.int16(-1) if kv == "bf16" else 0xFF)):
            a[bad] = nan
        if kv == "e4m3":
            for a in (p.ks, p.vs):
                a[bad[..., 0]] = 255
    out, lse = _run(lens, 8, 2, 64, page, kv, window=window, edit=poison)
    assert np.isfinite(out).all()


def test_infinite_and_nan_values_stay_where_they_enter():
    """An infinite v in one key leaves its element of the output not finite, and
    touches no other; a NaN in k makes its sequence's head NaN and no other's."""
    lens, page = [40, 40, 40], 16

    def edit(p, tab):
        p.v[tab[0, 1], 0, 3, 5] = np.int16(0x7F80)                   # +inf, key 19 of sequence 0
        p.k[tab[1, 2], 1, 0, 7] = np.int16(0x7FC0)                   # NaN, key 32 of sequence 1, head 1
    out, lse = _run(lens, 4, 2, 64, page, edit=edit, check=False)
    assert not np.isfinite(out[0, :2, 5]).any() and np.isfinite(np.delete(out[0], 5, 1)).all()
    assert np.isfinite(out[0, 2:]).all()
    assert np.isnan(out[1, 2:]).all() and np.isfinite(out[1, :2]).all() and np.isfinite(out[2]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bad_pages_and_lengths_are_left_out_and_reported(kv):
    def holes(p, tab):
        tab[0, 1], tab[1, 0], tab[2, :] = -7, 10 ** 6, -1            # a hole, a first page, a whole sequence
    _run([50, 20, 64, 33], 8, 2, 64, 16, kv, edit=holes, status=moe.MOE_ERR_BAD_INDEX)
    # a negative length counts as none, one above the row's capacity as the capacity
    _run([-5, 70, 10], 8, 2, 64, 16, kv, row=4, extra=5, status=moe.MOE_ERR_BAD_INDEX)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 elements, the sequence's pages at its two ends."""
    hkv, page, D = 16, 1024, 128
    pages = 2 ** 32 // (hkv * page * D) + 3
    rng = np.random.default_rng(3)
    n, ids = 2500, [0, pages - 1, pages - 2]
    small = Pool(3, hkv, page, D, "bf16", rng)
    big = {m: torch.zeros((pages, hkv, page, D), dtype=torch.int16, device="cuda") for m in "kv"}
    for i, at in enumerate(ids):
        for m in "kv":
            big[m][at] = small.dev[m][i]
    tab = np.array([ids], np.int32)
    qb = bf16_of(rng.standard_normal((1, hkv, D)))
    o = torch.empty((1, hkv, D), dtype=torch.float32, device="cuda")
    with handle(hkv, hkv, D, page, pages, 1, 3) as h:
        # the appended token is the sequence's last key
        pos = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
        kv = torch.from_numpy(bf16_of(rng.standard_normal((2, 1, hkv, D)))).cuda()
        pool = moe.kv_pool(big["k"], big["v"])
        td = torch.from_numpy(tab).cuda()
        moe.moe_kv_append(h, pool, kv[0], kv[1], pos, td, 1)
        moe.moe_kv_copy_pages(h, [pool], torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda"), 1)
        moe.moe_attn_decode(h, pool, torch.from_numpy(qb).cuda(), pos + 1, td, 1, o)
        torch.cuda.synchronize()
        assert moe.moe_kv_status(h) == moe.MOE_OK
    for i, m in enumerate("kv"):
        getattr(small, m)[2, :, (n - 1) % page] = kv[i, 0].cpu().numpy()
        assert torch.equal(big[m][pages - 3], big[m][pages - 1])
    check_attention(small, okv.bf16(qb), [n], np.array([[0, 1, 2]], np.int32), page, f64(o), None, D ** -0.5)


def test_refusals():
    B, hq, hkv, D, page = 2, 4, 2, 64, 16
    q = torch.zeros((B, hq, D), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros((B, hq, D), dtype=torch.float32, device="cuda")
    lens, tab = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, 1)))
    p = torch.zeros(1, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    good = moe.kv_pool(p, p)
    with handle(hq, hkv, D, page, 1, B, 1) as h:
        def refused(pool=good, q=q, lens=lens, tab=tab, B=B, o=o, **kw):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_attn_decode(h, pool, q, lens, tab, B, o, **kw)
            assert e.value.code == moe.MOE_ERR_INVALID_ARG, kw
        refused(B=3), refused(B=-1), refused(q=None), refused(lens=None), refused(tab=None), refused(o=None)
        refused(pool=moe.kv_pool(p, None)), refused(pool=moe.kv_pool(p, p, p, p))
        refused(q=q.data_ptr() + 8), refused(o=o.data_ptr() + 4), refused(o=q)
        refused(window=-1), refused(softcap=-1.0), refused(softcap=float("inf")), refused(scale=float("nan"))
        moe.moe_attn_decode(h, good, None, None, None, 0, None)
        assert moe.moe_kv_status(h) == moe.MOE_OK


def test_refuses_overlaps_and_extreme_factors():
    B, hq, hkv, D, page = 2, 4, 2, 64, 16
    lens, tab = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, 1)))
    p = torch.zeros(1, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    n = B * hq * D * 2                              # bytes of q; out takes twice that, lse 32
    at = torch.zeros(8 * n, dtype=torch.uint8, device="cuda").data_ptr() + 2 * n
    with handle(hq, hkv, D, page, 1, B, 1) as h:
        def run(q, o, lse=None, **kw):
            moe.moe_attn_decode(h, moe.kv_pool(p, p), at + q, lens, tab, B, at + o, None if lse is None else at + lse, **kw)

        def refused(*a, **kw):
            with pytest.raises(moe.MoeError) as e:
                run(*a, **kw)
            assert e.value.code == moe.MOE_ERR_INVALID_ARG, (a, kw)
        refused(0, n - 16), refused(2 * n - 16, 0), refused(0, -2 * n + 16)
        refused(0, n, lse=n - 16), refused(0, n, lse=3 * n - 16), refused(0, n, lse=-16)
        for kw in dict(scale=2.0 ** 33), dict(scale=-2.0 ** 33), dict(softcap=2.0 ** -33), dict(softcap=2.0 ** 33), dict(scale=1e300):
            refused(0, n, **kw)
        run(0, n, lse=3 * n), run(2 * n, 0, lse=3 * n), run(0, n, lse=-32)
        run(0, n, scale=2.0 ** 32, softcap=2.0 ** -32), run(0, n, scale=-2.0 ** 32, softcap=2.0 ** 32)
        assert moe.moe_kv_status(h) == moe.MOE_OK


def test_keys_whose_score_is_minus_infinity_weigh_nothing():
    """q of ones against keys with one element of -inf: those keys alone drop
    out; a sequence of none other ends like one without keys."""
    hq, hkv, D, page = 4, 2, 64, 16
    rng = np.random.default_rng(5)
    lens = np.array([40, 5], np.int32)
    p = Pool(4, hkv, page, D, "bf16", rng)
    tab = np.array([[0, 1, 2], [3, -1, -1]], np.int32)
    keep = np.ones((4, page), bool)
    for page_id, off in (0, 0), (0, 7), (1, 15), (2, 3):
        keep[page_id, off] = False
    keep[3, :5] = False
    i, off = np.nonzero(~keep)
    p.k[i, :, off, 9] = np.int16(-128)                               # 0xFF80, -inf
    p.upload()
    q = torch.ones(2, hq, D, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty(2, hq, D, device="cuda"), torch.empty(2, hq, device="cuda")
    with handle(hq, hkv, D, page, 4, 2, 3) as h:
        moe.moe_attn_decode(h, p.struct, q, torch.from_numpy(lens).cuda(), torch.from_numpy(tab).cuda(), 2, o, lse=lse)
        assert moe.moe_kv_status(h) == moe.MOE_OK
    assert not o[1].any() and torch.isneginf(lse[1]).all()
    # the same sequence with those keys taken out
    rows = [(int(tab[0, j // page]), j % page) for j in range(40)]
    rows = [r for r in rows if keep[r]]
    c = Pool(4, hkv, page, D, "bf16", rng)
    for j, (i, off) in enumerate(rows):
        c.k[j // page, :, j % page], c.v[j // page, :, j % page] = p.k[i, :, off], p.v[i, :, off]
    check_attention(c, np.ones((1, hq, D)), [len(rows)], np.array([[0, 1, 2]], np.int32), page, f64(o[:1]), f64(lse[:1]), D ** -0.5)


def test_allocation_failure_and_next_call():
    moe.moe_ffn_test_fail_allocs(1)
    try:
        with pytest.raises(moe.MoeError) as e:
            moe.moe_kv_create(moe.kv_config(4, 2, 64, 16, 4, 2, 2), 0)
        assert e.value.code == moe.MOE_ERR_OOM
    finally:
        moe.moe_ffn_test_fail_allocs(0)
    _run([17], 4, 2, 64, 16)
