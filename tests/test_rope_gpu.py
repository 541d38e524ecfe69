"""Rotary positions and the cache append against fp64 formulas, and against
each other: the append writes the bytes that moe_rope and moe_ffn_act_quant
give."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from kv_setup import Pool, bf16_of, f64, handle, table
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


LAYOUT = {"half": moe.MOE_ROPE_HALF, "interleaved": moe.MOE_ROPE_INTERLEAVED}


def _desc(rot, layout, kind="none", base=10000.0):
    k = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}[kind]
    turns, scale = moe.moe_rope_table(rot, base, k, 8.0, 4096)
    dev = torch.from_numpy(turns.view(np.int64)).cuda()
    f, m = okv.rope_frequencies(rot, base, kind, 8.0, 4096)
    return moe.rope(dev, rot, LAYOUT[layout], scale), dev, f, m


def _check_rope(got, x, pos, f, m, layout):
    """|error| <= half a bf16 step of the value, and before that rounding 1e-6 of
    m (|a| + |b|): cos and sin are within 2.5e-7 (an angle within pi / 4 of its
    quarter turn held to 2^-24 of itself, sums of 32-bit terms), the products
    and the sum add 3 * 2^-24, the scaling 2^-24."""
    live = np.asarray(pos) >= 0
    x, got, pos = x[live], got[live], np.asarray(pos)[live]
    ref = okv.rope(x, pos, f, m, layout)
    r = 2 * len(f)
    size = np.abs(x)
    if layout == "half":
        both = size[..., :r // 2] + size[..., r // 2:r]
        both = np.concatenate([both, both], -1)
    else:
        both = np.repeat(size[..., 0:r:2] + size[..., 1:r:2], 2, -1)
    tol = 2.0 ** -8 * np.abs(ref[..., :r]) + 1.01e-6 * m * both + 1e-38
    assert np.all(np.abs(got[..., :r] - ref[..., :r]) <= tol), float((np.abs(got[..., :r] - ref[..., :r]) / tol).max())
    assert np.array_equal(got[..., r:], x[..., r:])                  # the rest of the head as it was


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hkv,D,rot,kind", [
    (1, 1, 1, 16, 16, "none"), (3, 4, 2, 64, 64, "linear"), (7, 6, 3, 80, 80, "ntk"), (5, 8, 1, 96, 48, "yarn"),
    (33, 32, 8, 128, 128, "none"), (130, 5, 5, 112, 16, "none"), (2, 40, 8, 128, 64, "yarn"), (600, 3, 1, 32, 32, "none"),
    (400, 32, 8, 128, 128, "none"),
])
def test_rope_against_fp64(T, hq, hkv, D, rot, kind, layout):
    rng = np.random.default_rng(T + D)
    desc, keep, f, m = _desc(rot, layout, kind)
    pos = rng.integers(0, 5000, T).astype(np.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[T - 1] = 2 ** 31 - 1, 1048575                    # the largest position; a far one
    if T > 4:
        pos[3] = -1                                                  # padding
    qkv = torch.from_numpy(bf16_of(rng.standard_normal((T, hq + 2 * hkv, D)))).cuda().view(torch.bfloat16)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    pd = torch.from_numpy(pos).cuda()
    with handle(hq, hkv, D) as h:
        # parts of one projection's rows, to new tensors with rows behind the last
        qo, ko = (torch.full((T + 2, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (hq, hkv))
        moe.moe_rope(h, desc, pd, T, q=q, q_out=qo, k=k, k_out=ko, ldq=q.stride(0), ldk=k.stride(0))
        torch.cuda.synchronize()
        assert torch.all(qo[T:] == 7.0) and torch.all(ko[T:] == 7.0)
        for t in np.nonzero(pos < 0)[0]:
            assert torch.all(qo[t] == 7.0) and torch.all(ko[t] == 7.0)
        _check_rope(f64(qo[:T]), f64(q), pos, f, m, layout)
        _check_rope(f64(ko[:T]), f64(k), pos, f, m, layout)
        # contiguous, one alone, and in place with the stride: the same bytes; the values and padding stay
        one = torch.zeros((T, hkv, D), dtype=torch.bfloat16, device="cuda")
        moe.moe_rope(h, desc, pd, T, k=k.contiguous(), k_out=one)
        own = qkv.clone()
        moe.moe_rope(h, desc, pd, T, q=own[:, :hq], q_out=own[:, :hq], k=own[:, hq:], k_out=own[:, hq:],
                     ldq=own.stride(0), ldk=own.stride(0))
        torch.cuda.synchronize()
        live = torch.from_numpy(pos >= 0).cuda()
        assert torch.equal(one[live].view(torch.int16), ko[:T][live].view(torch.int16))
        assert torch.equal(own[live][:, :hq].view(torch.int16), qo[:T][live].view(torch.int16))
        assert torch.equal(own[live][:, hq:hq + hkv].view(torch.int16), ko[:T][live].view(torch.int16))
        assert torch.equal(own[:, hq + hkv:], qkv[:, hq + hkv:]) and torch.equal(own[~live], qkv[~live])
        assert moe.moe_kv_status(h) == moe.MOE_OK


def test_rope_turns_by_exact_fractions():
    """A frequency of 1/8 turn a position: every eighth position returns the
    input, position 2 swaps the pair, position 4 negates it."""
    D = 16
    turns = torch.full((D // 2,), 2 ** 61, dtype=torch.int64, device="cuda")
    x = torch.arange(1, D + 1, dtype=torch.float32, device="cuda").to(torch.bfloat16).view(1, 1, D).repeat(6, 1, 1)
    pos = torch.tensor([0, 8, 2, 4, 2 ** 31 - 8, 2 ** 31 - 6], dtype=torch.int32, device="cuda")
    with handle(1, 1, D) as h:
        y = torch.empty_like(x)
        moe.moe_rope(h, moe.rope(turns, D, moe.MOE_ROPE_INTERLEAVED), pos, 6, q=x, q_out=y)
        a, b = f64(x)[0, 0, 0::2], f64(x)[0, 0, 1::2]
        got = f64(y)[:, 0]
        for i, (wa, wb) in enumerate([(a, b), (a, b), (-b, a), (-a, -b), (a, b), (-b, a)]):
            assert np.array_equal(got[i, 0::2], wa) and np.array_equal(got[i, 1::2], wb), i


def test_rope_refusals():
    D, T = 64, 4
    desc, keep, _, _ = _desc(64, "half")
    x = torch.zeros((T + 1, 4, D), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    with handle(4, 2, D) as h:
        def refused(code=moe.MOE_ERR_INVALID_ARG, rope=desc, T=T, pos=pos, **kw):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_rope(h, rope, pos, T, **kw)
            assert e.value.code == code, kw
        refused(q=x)
        refused(q_out=y)
        refused(q=x, q_out=y, T=-1)
        refused(q=x, q_out=y, pos=None)
        refused(q=x, q_out=y, ldq=4 * D - 8)                         # heads overlap
        refused(q=x, q_out=y, ldq=4 * D + 4)                         # rows off 16 bytes
        refused(q=x.data_ptr() + 2, q_out=y)
        refused(q=x, q_out=x.data_ptr() + 16)                        # overlaps without being the same
        refused(q=x, q_out=y, k=y, k_out=y)                          # q's output over k
        refused(q=x, q_out=y, T=(1 << 24) + 1, code=moe.MOE_ERR_UNSUPPORTED)
        for bad in [moe.rope(None, 64, 0), moe.rope(keep, 72, 0), moe.rope(keep, 24, 0), moe.rope(keep, 0, 0),
                    moe.rope(keep, 64, 2), moe.rope(keep, 64, 0, float("nan"))]:
            refused(rope=bad, q=x, q_out=y)
        moe.moe_rope(h, desc, None, 0, q=x, q_out=y)                 # no tokens: nothing to do
        moe.moe_rope(h, desc, pos, T)
        assert moe.moe_kv_status(h) == moe.MOE_OK and torch.count_nonzero(y) == 0


CASES = [  # T tokens of seqs sequences from `start`; heads, page
    (1, 1, 0, 4, 1, 16, 16, "bf16"), (9, 9, 40, 8, 2, 64, 16, "bf16"), (37, 3, 5, 6, 3, 80, 32, "bf16"),
    (70, 2, 1, 32, 8, 128, 64, "bf16"), (1, 1, 0, 4, 1, 32, 16, "e4m3"), (9, 9, 40, 8, 2, 64, 16, "e4m3"),
    (37, 3, 5, 6, 3, 96, 48, "e4m3"), (70, 2, 1, 32, 8, 128, 64, "e4m3"), (700, 4, 3, 16, 4, 128, 16, "e4m3"),
]


@pytest.mark.parametrize("T,seqs,start,hq,hkv,D,page,kv", CASES)
@pytest.mark.parametrize("layout,part", [("half", 1), ("interleaved", 2), ("half", 2), (None, 1)])
def test_append_writes_what_rope_and_act_quant_give(T, seqs, start, hq, hkv, D, page, kv, layout, part):
    rng = np.random.default_rng(T * 31 + D)
    rot = max(16, D // part // 16 * 16)
    seq = (np.arange(T) * seqs // T).astype(np.int32)
    pos = np.array([start + int((seq[:t] == seq[t]).sum()) for t in range(T)], np.int32)
    if T > 5:
        pos[4] = -1
    lens = [int(max([p + 1 for p, s in zip(pos, seq) if s == i] or [1])) for i in range(seqs)]
    row = max(-(-n // page) for n in lens)
    pages = seqs * row + 2
    tab = table(lens, page, pages, row, rng)
    p = Pool(pages, hkv, page, D, kv, rng)
    before = {n: a.copy() for n, a in p.bytes().items()}
    x = rng.standard_normal((T, hq + 2 * hkv, D)) * 2.0 ** rng.integers(-20, 20, (T, 1, 1))
    x[T // 2, hq:] = 0.0                                             # a row of zeros in the cache
    qkv = torch.from_numpy(bf16_of(x)).cuda().view(torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pd, sd, td = (torch.from_numpy(a).cuda() for a in (pos, seq, tab))
    with handle(hq, hkv, D, page, pages, seqs, row, kv) as h:
        ld = qkv.stride(0)
        qo = torch.full((T, hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
        if layout:
            desc, keep, f, m = _desc(rot, layout, "yarn")
            moe.moe_kv_append(h, p.struct, k, v, pd, td, T, seq=sd, rope=desc, q=q, q_out=qo, ldq=ld, ldk=ld, ldv=ld)
            kr = torch.zeros((T, hkv, D), dtype=torch.bfloat16, device="cuda")
            qr = torch.full_like(qo, 3.0)
            moe.moe_rope(h, desc, pd, T, q=q, q_out=qr, k=k, k_out=kr, ldq=ld, ldk=ld)
        else:
            moe.moe_kv_append(h, p.struct, k, v, pd, td, T, seq=sd, ldk=ld, ldv=ld)
            kr, qr = k.contiguous(), qo.clone()
        got = p.bytes()
        assert torch.equal(qo.view(torch.int16), qr.view(torch.int16))
        assert moe.moe_kv_status(h) == moe.MOE_OK
    want = before
    live = [t for t in range(T) if pos[t] >= 0]
    for name, rows in (("k", kr), ("v", v.contiguous())):
        if kv == "bf16":
            codes, sc = rows.view(torch.int16).cpu().numpy(), None
        else:
            hf = moe.moe_ffn_create(moe.config(8, 256, 128, 2, 1), 0)
            c = torch.zeros((T * hkv, D), dtype=torch.uint8, device="cuda")
            s = torch.zeros((T * hkv, 1), dtype=torch.uint8, device="cuda")
            moe.moe_ffn_act_quant(hf, rows, T * hkv, D, c, s)
            torch.cuda.synchronize()
            moe.moe_ffn_destroy(hf)
            codes, sc = c.view(T, hkv, D).cpu().numpy(), s.view(T, hkv).cpu().numpy()
        for t in live:
            at = tab[seq[t], pos[t] // page], slice(None), pos[t] % page
            want[name][at] = codes[t]
            if sc is not None:
                want[name + "s"][at] = sc[t]
    for name in want:
        assert np.array_equal(got[name], want[name]), name           # every other byte of the pool as it was


def test_append_without_seq_and_in_place_q():
    """seq NULL: token t is of sequence t; q rotated in place inside its rows."""
    T, hq, hkv, D, page = 5, 4, 2, 64, 16
    rng = np.random.default_rng(0)
    desc, keep, f, m = _desc(64, "half")
    tab = rng.permutation(10).astype(np.int32).reshape(5, 2)
    pos = np.array([0, 31, 16, 15, 7], np.int32)
    qkv = torch.from_numpy(bf16_of(rng.standard_normal((T, hq + 2 * hkv, D)))).cuda().view(torch.bfloat16)
    orig = qkv.clone()
    p = Pool(10, hkv, page, D, "bf16", rng)
    with handle(hq, hkv, D, page, 10, 5, 2) as h:
        ld = qkv.stride(0)
        moe.moe_kv_append(h, p.struct, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], torch.from_numpy(pos).cuda(),
                          torch.from_numpy(tab).cuda(), T, rope=desc, q=qkv, q_out=qkv, ldq=ld, ldk=ld, ldv=ld)
        got = p.bytes()
        assert moe.moe_kv_status(h) == moe.MOE_OK
    _check_rope(f64(qkv[:, :hq]), f64(orig[:, :hq]), pos, f, m, "half")
    assert torch.equal(qkv[:, hq:], orig[:, hq:])
    for t in range(T):
        at = tab[t, pos[t] // page], slice(None), pos[t] % page
        _check_rope(okv.bf16(got["k"][at])[None], f64(orig[t:t + 1, hq:hq + hkv]), pos[t:t + 1], f, m, "half")
        assert np.array_equal(got["v"][at], orig[t, hq + hkv:].view(torch.int16).cpu().numpy())


def test_append_bad_places_are_left_out_and_reported():
    T, hq, hkv, D, page = 6, 2, 1, 32, 16
    rng = np.random.default_rng(1)
    tab = np.array([[0, 1], [2, -1], [99, 3]], np.int32)
    seq = np.array([0, 1, 2, 3, -1, 0], np.int32)                    # 3 and -1 are no sequences
    pos = np.array([32, 16, 3, 0, 0, 1], np.int32)                   # 32 is beyond the row; pages -1 and 99
    desc, keep, f, m = _desc(32, "half")
    for kv in ("bf16", "e4m3"):
        p = Pool(4, hkv, page, D, kv, rng)
        before = {n: a.copy() for n, a in p.bytes().items()}
        x = torch.from_numpy(bf16_of(rng.standard_normal((3, T, hq, D)))).cuda().view(torch.bfloat16)
        k, v = x[1, :, :1].contiguous(), x[2, :, :1].contiguous()
        qo = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
        with handle(hq, hkv, D, page, 4, 3, 2, kv) as h:
            moe.moe_kv_append(h, p.struct, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(tab).cuda(), T,
                              seq=torch.from_numpy(seq).cuda(), rope=desc, q=x[0], q_out=qo)
            assert moe.moe_kv_status(h) == moe.MOE_ERR_BAD_INDEX
            assert moe.moe_kv_status(h) == moe.MOE_OK                # cleared
        got = p.bytes()
        for n in got:
            same = got[n] == before[n]
            same[0, :, 1] = True                                     # the one token that has a place
            assert same.all(), n
        assert not np.array_equal(got["v"][0, :, 1], before["v"][0, :, 1])
        _check_rope(f64(qo), f64(x[0]), pos, f, m, "half")


def test_in_place_beside_other_parts_of_the_rows():
    """q in place: k and v may lie between its rows, with its stride, and nowhere on them."""
    T, hq, hkv, D, page = 3, 4, 2, 64, 16
    desc, keep, _, _ = _desc(64, "half")
    ld = (hq + 2 * hkv) * D
    x = torch.zeros(2 * T * ld, dtype=torch.bfloat16, device="cuda")
    at = lambda e: x.data_ptr() + 2 * e                               # noqa: E731
    other = torch.zeros(T, hkv, D, dtype=torch.bfloat16, device="cuda")
    pos, seq = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    pos += torch.arange(T, device="cuda", dtype=torch.int32)
    tab = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    p = torch.zeros(2, 1, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    good = moe.kv_pool(p[0], p[1])
    with handle(hq, hkv, D, page, 1, 2, 1) as h:
        def rope(k, ldk, T=T, q=0):
            moe.moe_rope(h, desc, pos, T, q=at(q), q_out=at(q), ldq=ld, k=k, k_out=k, ldk=ldk)

        def append(k, v, ldk, ldv):
            moe.moe_kv_append(h, good, k, v, pos, tab, T, seq=seq, rope=desc, q=at(0), q_out=at(0), ldq=ld, ldk=ldk, ldv=ldv)

        def refused(f, *a, **kw):
            with pytest.raises(moe.MoeError) as e:
                f(*a, **kw)
            assert e.value.code == moe.MOE_ERR_INVALID_ARG, a
        end = ld - hkv * D
        for k, ldk in (at(0), ld), (at(hq * D - 8), ld), (at(hq * D), ld - 8), (at(end + 8), ld), (at(ld), ld):
            refused(rope, k, ldk)
            refused(append, k, other, ldk, 0)
            refused(append, other, k, 0, ldk)
        refused(rope, at(hq * D - 8), ld, T=1)
        refused(rope, at(0), ld, q=hkv * D - 8)
        rope(at(hq * D), ld), rope(at(end), ld), rope(at(T * ld), hkv * D), rope(at(0), ld, q=hkv * D)
        rope(at(hq * D), hkv * D, T=1)
        append(at(hq * D), at(end), ld, ld), append(at(T * ld), at(T * ld), 0, 0)
        assert moe.moe_kv_status(h) == moe.MOE_OK


def test_append_refusals():
    T, hq, hkv, D, page = 3, 4, 2, 64, 16
    desc, keep, _, _ = _desc(64, "half")
    k, v, q, qo = (torch.zeros((T, n, D), dtype=torch.bfloat16, device="cuda") for n in (hkv, hkv, hq, hq))
    pos, tab = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    p = torch.zeros(1, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(64, dtype=torch.uint8, device="cuda")
    good = moe.kv_pool(p, p.clone())
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    with handle(hq, hkv, D, page, 1, 2, 1) as h:
        def refused(pool=good, k=k, v=v, pos=pos, tab=tab, T=T, code=moe.MOE_ERR_INVALID_ARG, **kw):
            with pytest.raises(moe.MoeError) as e:
                moe.moe_kv_append(h, pool, k, v, pos, tab, T, **{"seq": seq, **kw})
            assert e.value.code == code, kw
        for bad in [moe.kv_pool(None, p), moe.kv_pool(p, None), moe.kv_pool(p, p, s, s), moe.kv_pool(p, p, s, None),
                    moe.kv_pool(p.data_ptr() + 2, p)]:
            refused(pool=bad)
        refused(k=None), refused(v=None), refused(pos=None), refused(tab=None), refused(T=-1)
        refused(seq=None)                                            # three tokens, two sequences
        refused(q=q, q_out=qo)                                       # q without a rotation
        refused(q=q, rope=desc), refused(q_out=qo, rope=desc)
        refused(ldk=64), refused(ldv=132), refused(q=q, q_out=qo, rope=desc, ldq=8)
        refused(q=q, q_out=k, rope=desc)                             # over an input
        refused(T=(1 << 24) + 1, code=moe.MOE_ERR_UNSUPPORTED)
        refused(rope=moe.rope(keep, 80, 0))
        moe.moe_kv_append(h, good, None, None, None, None, 0)
        assert moe.moe_kv_status(h) == moe.MOE_OK
    assert moe.lib().moe_kv_append(None, ctypes.byref(good), None, 0, None, 0, None, None, None, 1, None, None, 0, None,
                                   None) == moe.MOE_ERR_INVALID_ARG
