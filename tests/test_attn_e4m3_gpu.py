"""Attention over E4M3 caches where the scores are large or the values' scales
lie far apart, against fp64."""
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


def _attend(p, q_bits, lens, tab, page, out="f32", **kw):
    B, hq, D = q_bits.shape
    hkv, pages = p.k.shape[1], p.k.shape[0]
    o = torch.empty((B, hq, D), dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    lse = torch.empty((B, hq), dtype=torch.float32, device="cuda")
    p.upload()
    with handle(hq, hkv, D, page, pages, B, tab.shape[1], "e4m3", out) as h:
        moe.moe_attn_decode(h, p.struct, torch.from_numpy(q_bits).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                            torch.from_numpy(tab).cuda(), B, o, lse=lse, **kw)
        assert moe.moe_kv_status(h) == moe.MOE_OK
    return f64(o), f64(lse)


HEADS = [(4, 2, 32), (4, 2, 64), (12, 1, 64), (4, 2, 96), (12, 1, 96), (8, 2, 128), (12, 1, 128)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,D", HEADS)
def test_one_key_gives_its_value_whatever_its_score(hq, hkv, D, out):
    """Scores up to 1e5.  The weight is 2^0 for the sum and 2^(a whole number)
    for the value: two exponentials of whole numbers (each within 2^-22), and the
    quotient, the factor and the store, half a step of 2^-23 each: 2^-21 + 3 2^-24.
    A value has 4 significant bits, so a bf16 output is the value itself."""
    rng = np.random.default_rng(D + hq)
    B, page = 64, 16
    p = Pool(B, hkv, page, D, "e4m3", rng, spread=5.0)
    p.ks[:] = 119
    tab = rng.permutation(B).astype(np.int32).reshape(B, 1)
    q = bf16_of(rng.standard_normal((B, hq, D)) * np.geomspace(0.1, 1e5, B)[:, None, None])
    got, _ = _attend(p, q, [1] * B, tab, page, out)
    for b in range(B):
        for h in range(hkv):
            v = okv.rows(p.v, p.vs, [int(tab[b, 0])], h, 1)[0]
            for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                tol = 0.0 if out == "bf16" else (2.0 ** -21 + 3 * 2.0 ** -24) * np.abs(v)
                assert np.all(np.abs(got[b, g] - v) <= tol), (b, g, float(np.max(np.abs(got[b, g] - v) / np.abs(v + (v == 0)))))


@pytest.mark.parametrize("score", [0.0, 30.37, -77.7, 333.3, 4001.7, 1e6])
@pytest.mark.parametrize("hq,hkv,D", HEADS)
def test_keys_of_one_score_give_the_mean_of_their_values(hq, hkv, D, score):
    """Equal keys have equal weights, and their error in common: what is left is
    two exponentials (2^-21 together), the weights' two terms (2^-21), n additions
    taken as 4 sqrt(n) 2^-24, all of the mean of |v|, and 2^-31 of the largest
    weight times scale for a code."""
    rng = np.random.default_rng(D + hq)
    page, lens = 16, [2, 16, 33, 300, 3000, 20000]
    row = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens)
    p = Pool(pages, hkv, page, D, "e4m3", rng, spread=2.0)
    p.k[:], p.ks[:] = 0x38, 127                                      # ones
    tab = table(lens, page, pages, row, rng)
    got, lse = _attend(p, bf16_of(np.ones((len(lens), hq, D))), lens, tab, page, scale=score / D if score else 1e-30)
    for b, n in enumerate(lens):
        ids = [int(i) for i in tab[b, :-(-n // page)]]
        for h in range(hkv):
            v = okv.rows(p.v, p.vs, ids, h, n)
            f = np.concatenate([okv.scale_of(p.vs[i, h]) for i in ids])[:n]
            tol = (2.0 ** -20 + 4 * np.sqrt(n) * 2.0 ** -24) * np.abs(v).mean(0) + 2.0 ** -31 * f.max() / n * np.abs(v / f[:, None]).sum(0)
            for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                err = np.abs(got[b, g] - v.mean(0))
                assert np.all(err <= tol), (b, g, float((err / tol).max()))
                want = score + np.log(n)
                assert abs(lse[b, g] - want) <= 2.0 ** -20 * max(1.0, abs(want))


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("rise", [3.0, -3.0, 40.0])
def test_scores_and_value_scales_that_move_apart(rise, hq, hkv, D):
    """Scores that rise (or fall) from key to key, so that the softmax's reference
    moves again and again, while the values' scales fall (or rise) over 2^-60 ..
    2^60: the output's reference goes its own way."""
    rng = np.random.default_rng(D + hq)
    page, lens = 16, [5, 40, 200, 700, 5000]
    row = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens)
    p = Pool(pages, hkv, page, D, "e4m3", rng)
    tab = table(lens, page, pages, row, rng)
    for b, n in enumerate(lens):
        for j in range(n):
            i, off = tab[b, j // page], j % page
            t = j / n * 40 if rise < 40 else j % 40                  # key 0's element is its score
            p.k[i, :, off] = 0
            p.k[i, :, off, 0] = 0x38 + int(8 * (t % 1.0)) if t >= 1 else 0x30
            p.ks[i, :, off] = 127 + int(np.log2(max(t, 1.0)))
            p.vs[i, :, off] = 127 + int(np.clip(60 - 3.1 * t + rng.integers(-3, 4), -60, 60))
    q = np.zeros((len(lens), hq, D))
    q[:, :, 0] = np.sign(rise) * np.linspace(1.0, 3.0, hq)
    q = bf16_of(q)
    got, lse = _attend(p, q, lens, tab, page, scale=3.0)
    check_attention(p, okv.bf16(q), lens, tab, page, got, lse, 3.0)


@pytest.mark.parametrize("hq,hkv,D", HEADS)
def test_value_scales_over_the_whole_range(hq, hkv, D):
    rng = np.random.default_rng(D + hq)
    page, lens = 16, [0, 1, 2, 15, 17, 33, 100, 257, 3000]
    row = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens)
    p = Pool(pages, hkv, page, D, "e4m3", rng)
    p.vs[:] = np.clip(np.rint(119 + 40 * rng.standard_normal(p.vs.shape)), 1, 220)
    tab = table(lens, page, pages, row, rng)
    for qscale in (1.5, 60.0):
        q = bf16_of(qscale * rng.standard_normal((len(lens), hq, D)))
        got, lse = _attend(p, q, lens, tab, page)
        check_attention(p, okv.bf16(q), lens, tab, page, got, lse, D ** -0.5)


@pytest.mark.parametrize("hq,hkv,D", HEADS)
def test_a_scale_byte_of_255_is_nan(hq, hkv, D):
    """With codes that are numbers: a key's makes its scores NaN, a value's the
    output; outside the keys that count it is never used."""
    rng = np.random.default_rng(D)
    page, lens = 16, [40, 40, 40, 3000, 3000, 40, 33]
    row = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens)
    p = Pool(pages, hkv, page, D, "e4m3", rng)
    tab = table(lens, page, pages, row, rng)
    at = lambda b, j: (tab[b, j // page], slice(None), j % page)     # noqa: E731
    q = np.ones((len(lens), hq, D))
    p.k[at(0, 19)] = 0xB8                                            # ones, negative: a score of -inf were the byte infinity
    p.ks[at(0, 19)] = 255
    p.vs[at(1, 7)] = p.vs[at(3, 2999)] = 255
    p.ks[at(4, 0)] = 255
    p.vs[at(5, 3)] = p.ks[at(5, 4)] = 255                            # before the window of 30
    p.vs[at(6, 40)] = p.ks[at(6, 47)] = 255                          # behind the last key
    got, lse = _attend(p, bf16_of(q), lens, tab, page)
    assert np.isnan(got[[0, 1, 3, 4]]).all() and np.isnan(lse[[0, 4]]).all()
    assert np.isfinite(got[[2, 6]]).all() and np.isfinite(lse[[1, 2, 3, 6]]).all()
    keep = [2, 6]
    check_attention(p, q[keep], [lens[b] for b in keep], tab[keep], page, got[keep], lse[keep], D ** -0.5)
    got, lse = _attend(p, bf16_of(q), [40] * 7, tab, page, window=30)
    assert np.isfinite(got[[2, 5]]).all() and np.isfinite(lse[[2, 5]]).all()
    check_attention(p, q[[5]], [40], tab[[5]], page, got[[5]], lse[[5]], D ** -0.5, window=30)


@pytest.mark.parametrize("hq,hkv,D", HEADS)
def test_scale_byte_zero_is_the_smallest_scale(hq, hkv, D):
    """2^-127, not zero: seen with queries of 2^120."""
    rng = np.random.default_rng(D)
    page, lens = 16, [1, 33, 700]
    row = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens)
    p = Pool(pages, hkv, page, D, "e4m3", rng)
    p.ks[:] = 0
    p.ks[rng.random(p.ks.shape) < 0.3] = 1
    tab = table(lens, page, pages, row, rng)
    q = bf16_of(2.0 ** 120 * rng.standard_normal((len(lens), hq, D)))
    got, lse = _attend(p, q, lens, tab, page, scale=0.25)
    check_attention(p, okv.bf16(q), lens, tab, page, got, lse, 0.25)
    assert np.abs(lse[0]).max() > 2.0 ** -6                          # the scores are there


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,D", HEADS + [(12, 1, 32), (24, 1, 128)])
@pytest.mark.parametrize("softcap,scale,window", [(30.0, 0.0, 0), (2.0, 0.5, 0), (50.0, 0.0, 33), (5.0, -0.4, 100), (0.0, -0.3, 0),
                                                  (0.0, 1e-3, 17)])
def test_softcap_and_scale(softcap, scale, window, hq, hkv, D, out):
    """Every kernel of E4M3 rows with capped and negative scores: the cap comes
    before the values' scales, the keys' scales before the cap."""
    rng = np.random.default_rng(D + hq + window)
    page, lens = 16, [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 3000]
    row = -(-max(lens) // page)
    pages = sum(-(-n // page) for n in lens)
    p = Pool(pages, hkv, page, D, "e4m3", rng, spread=1.5)
    tab = table(lens, page, pages, row, rng)
    q = bf16_of(1.5 * rng.standard_normal((len(lens), hq, D)))
    got, lse = _attend(p, q, lens, tab, page, out, scale=scale, softcap=softcap, window=window)
    check_attention(p, okv.bf16(q), lens, tab, page, got, lse, scale or D ** -0.5, softcap, window, out == "bf16")
