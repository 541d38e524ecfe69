"""The pages' bookkeeping and the rotary table (host code in libmoe_ffn.so, no
GPU): the manager against a model with plain lists over random histories, hand
cases, what it refuses; the table against 64-bit frequencies."""
import ctypes
import math
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, localcontext

import numpy as np
import pytest

import fp4_block_scaled_gb300 as moe
from oracle import kv as okv


@pytest.fixture
def manager():
    made = []

    def make(*a):
        made.append(moe.moe_kv_pages_create(*a))
        return made[-1]

    yield make
    for m in made:
        moe.moe_kv_pages_destroy(m)


def _same(m, model):
    assert moe.moe_kv_pages_free_pages(m) == model.free_pages()
    for i, (length, ids) in model.seqs.items():
        assert moe.moe_kv_pages_length(m, i) == length
        assert moe.moe_kv_pages_row(m, i, model.row).tolist() == ids + [-1] * (model.row - len(ids))
    assert [moe.moe_kv_pages_refs(m, p) for p in range(len(model.refs))] == model.refs


def _code(f, *a):
    with pytest.raises(moe.MoeError) as e:
        f(*a)
    return e.value.code


@pytest.mark.parametrize("pages,ps,seqs,row", [(7, 16, 4, 5), (70, 1, 9, 40), (128, 16, 20, 12), (1, 32, 2, 1)])
def test_manager_follows_the_model_over_random_histories(manager, pages, ps, seqs, row):
    for seed in range(4):
        rng = np.random.default_rng(seed)
        m, model = manager(pages, ps, seqs, row), okv.Pages(pages, ps, seqs, row)
        for _ in range(300):
            ids = list(model.seqs)
            what = rng.integers(0, 10)
            if what < 2 or not ids:
                want = model.open()
                if want is None:
                    assert _code(moe.moe_kv_pages_open, m) == moe.MOE_ERR_OOM
                else:
                    assert moe.moe_kv_pages_open(m) == want
            elif what < 6:
                i, n = int(rng.choice(ids)), int(rng.integers(0, 3 * ps + 1))
                try:
                    want = model.extend(i, n)
                except (ValueError, MemoryError) as e:
                    code = moe.MOE_ERR_OOM if isinstance(e, MemoryError) else moe.MOE_ERR_INVALID_ARG
                    assert _code(moe.moe_kv_pages_extend, m, i, n) == code
                else:
                    assert moe.moe_kv_pages_extend(m, i, n) == want
            elif what < 8:
                i = int(rng.choice(ids))
                want = model.fork(i)
                if want is None:
                    assert _code(moe.moe_kv_pages_fork, m, i) == moe.MOE_ERR_OOM
                else:
                    assert moe.moe_kv_pages_fork(m, i) == want
            elif what < 9:
                i = int(rng.choice(ids))
                model.free(i)
                moe.moe_kv_pages_free(m, i)
            else:
                most = int(rng.integers(0, pages + 1))
                assert moe.moe_kv_pages_compact(m, most).tolist() == [list(p) for p in model.compact(most)]
            _same(m, model)


def test_a_fork_gets_its_own_page_at_its_first_token_inside_a_shared_one(manager):
    m = manager(8, 16, 4, 4)
    a = moe.moe_kv_pages_open(m)
    assert moe.moe_kv_pages_extend(m, a, 20) is None
    b = moe.moe_kv_pages_fork(m, a)
    assert moe.moe_kv_pages_free_pages(m) == 6 and moe.moe_kv_pages_refs(m, 1) == 2
    assert moe.moe_kv_pages_extend(m, b, 1) == (1, 2)          # page 1 is shared and half full
    assert moe.moe_kv_pages_extend(m, a, 1) is None            # now page 1 is a's alone
    assert moe.moe_kv_pages_row(m, a, 4).tolist() == [0, 1, -1, -1]
    assert moe.moe_kv_pages_row(m, b, 4).tolist() == [0, 2, -1, -1]
    # on a page's border nothing is copied
    assert moe.moe_kv_pages_extend(m, a, 11) is None
    c = moe.moe_kv_pages_fork(m, a)
    assert moe.moe_kv_pages_extend(m, c, 1) is None and moe.moe_kv_pages_row(m, c, 4).tolist() == [0, 1, 3, -1]
    moe.moe_kv_pages_free(m, a)
    assert [moe.moe_kv_pages_refs(m, p) for p in range(4)] == [2, 1, 1, 1]
    moe.moe_kv_pages_free(m, b)
    assert moe.moe_kv_pages_compact(m, 8).tolist() == [[3, 2]]
    assert moe.moe_kv_pages_row(m, c, 4).tolist() == [0, 1, 2, -1]


def test_manager_refusals(manager):
    L = moe.lib()
    out = ctypes.c_void_p()
    for bad in [(0, 16, 1, 1), (1, 0, 1, 1), (1, 16, 0, 1), (1, 16, 1, 0), (-5, 16, 1, 1), (1, 1 << 20, 1, 1 << 20)]:
        assert L.moe_kv_pages_create(*bad, ctypes.byref(out)) == moe.MOE_ERR_INVALID_ARG and out.value is None
    m = manager(4, 16, 2, 2)
    assert _code(moe.moe_kv_pages_extend, m, 0, 1) == moe.MOE_ERR_INVALID_ARG        # not open
    a = moe.moe_kv_pages_open(m)
    for f, args in [(moe.moe_kv_pages_extend, (a, -1)), (moe.moe_kv_pages_extend, (a, 33)), (moe.moe_kv_pages_extend, (2, 1)),
                    (moe.moe_kv_pages_extend, (-1, 1)), (moe.moe_kv_pages_fork, (1,)), (moe.moe_kv_pages_free, (1,)),
                    (moe.moe_kv_pages_length, (7,)), (moe.moe_kv_pages_refs, (4,)), (moe.moe_kv_pages_refs, (-1,)),
                    (moe.moe_kv_pages_compact, (-1,))]:
        assert _code(f, m, *args) == moe.MOE_ERR_INVALID_ARG, (f, args)
    moe.moe_kv_pages_extend(m, a, 32)
    assert _code(moe.moe_kv_pages_row, m, a, 1) == moe.MOE_ERR_INVALID_ARG           # two pages do not fit one entry
    assert _code(moe.moe_kv_pages_extend, m, a, 2 ** 31 - 1) == moe.MOE_ERR_INVALID_ARG
    moe.moe_kv_pages_free(m, a)
    assert _code(moe.moe_kv_pages_free, m, a) == moe.MOE_ERR_INVALID_ARG             # twice
    one = (ctypes.c_int32 * 2)()
    n = ctypes.c_int()
    assert L.moe_kv_pages_extend(None, 0, 1, one) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_pages_extend(m, 0, 1, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_pages_compact(m, None, 1, ctypes.byref(n)) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_pages_free_pages(None) == moe.MOE_ERR_INVALID_ARG
    moe.moe_kv_pages_destroy(None)


@pytest.mark.parametrize("kind,name", [(0, "none"), (1, "linear"), (2, "ntk"), (3, "yarn")])
@pytest.mark.parametrize("rot,base,factor,trained", [(128, 10000.0, 4.0, 8192), (64, 500000.0, 32.0, 4096), (16, 10000.0, 1.0, 2048)])
def test_rope_table(kind, name, rot, base, factor, trained):
    turns, scale = moe.moe_rope_table(rot, base, kind, factor, trained)
    f, m = okv.rope_frequencies(rot, base, name, factor, trained)
    # a 64-bit fraction of a turn holds f to 2^-65 turns; the fp64 formulas of
    # the two sides agree to a few units of 2^-52
    err = np.abs(turns.astype(np.float64) / 2.0 ** 64 - f / (2 * math.pi))
    assert np.all(err <= 2.0 ** -64 + 16 * 2.0 ** -52 * f / (2 * math.pi))
    assert abs(scale - m) <= 2.0 ** -23


def test_rope_table_refusals():
    for bad in [(0, 1e4), (3, 1e4), (-2, 1e4), (1026, 1e4), (64, 1.0), (64, -3.0), (64, math.nan), (64, math.inf),
                (64, 1e4, 4), (64, 1e4, -1), (64, 1e4, 1, 0.5), (64, 1e4, 1, math.nan), (64, 1e4, 3, 4.0, 0),
                (2, 1e4, 2, 4.0)]:
        assert _code(moe.moe_rope_table, *bad) == moe.MOE_ERR_INVALID_ARG, bad


def test_cache_configs_and_null_handles_are_refused():
    ok = dict(num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=10, max_seqs=3, max_pages_per_seq=4)
    assert moe.moe_kv_pool_bytes(moe.kv_config(**ok)) == (10 * 2 * 16 * 64 * 2, 0)
    assert moe.moe_kv_pool_bytes(moe.kv_config(**ok, kv_dtype=moe.MOE_KV_E4M3_UE8M0)) == (10 * 2 * 16 * 64, 10 * 2 * 16)
    bad = [(k, v, moe.MOE_ERR_INVALID_ARG) for k in ok for v in (0, -1)]
    bad += [("num_q_heads", 7, moe.MOE_ERR_INVALID_ARG), ("kv_dtype", 2, moe.MOE_ERR_INVALID_ARG),
            ("out_dtype", 2, moe.MOE_ERR_INVALID_ARG)]
    bad += [(k, v, moe.MOE_ERR_UNSUPPORTED) for k, v in
            [("head_dim", 40), ("head_dim", 144), ("page_size", 24), ("page_size", 2048), ("max_seqs", 2049),
             ("num_q_heads", 514), ("max_pages_per_seq", 1 << 27)]]
    L = moe.lib()
    h = ctypes.c_void_p()
    for k, v, code in bad:
        cfg = moe.kv_config(**{**{n: x for n, x in ok.items()}, k: v})
        assert _code(moe.moe_kv_pool_bytes, cfg) == code, (k, v)
        assert L.moe_kv_create(ctypes.byref(h), ctypes.byref(cfg), 0) == code and h.value is None
    cfg = moe.kv_config(**{**ok, "head_dim": 48}, kv_dtype=moe.MOE_KV_E4M3_UE8M0)
    assert _code(moe.moe_kv_pool_bytes, cfg) == moe.MOE_ERR_UNSUPPORTED
    e = moe.MOE_ERR_INVALID_ARG
    assert L.moe_kv_create(None, ctypes.byref(cfg), 0) == e
    assert L.moe_rope(None, None, None, 1, None, 0, None, None, 0, None, None) == e
    assert L.moe_kv_append(None, None, None, 0, None, 0, None, None, None, 1, None, None, 0, None, None) == e
    assert L.moe_attn_decode(None, None, None, None, None, 1, 1.0, 0.0, 0, None, None, None) == e
    assert L.moe_kv_copy_pages(None, None, 0, None, 0, None) == e
    assert L.moe_kv_status(None, None) == e
    L.moe_kv_destroy(None)


def test_word_call_refusals():
    """moe_kv_call takes the calls' arguments as 64-bit words and refuses what they would."""
    L, e = moe.lib(), moe.MOE_ERR_INVALID_ARG
    for op in (-1, 4):
        assert L.moe_kv_call(op, bytes(8 * 16)) == e
    for op in range(4):
        assert L.moe_kv_call(op, None) == e
        assert L.moe_kv_call(op, bytes(8 * 16)) == e                 # no handle
    pool, rope = moe.kv_pool(0, 0), moe.rope(0, 16, 0)
    for f in (lambda: moe.moe_rope(None, rope, None, 1), lambda: moe.moe_kv_append(None, pool, None, None, None, None, 1),
              lambda: moe.moe_attn_decode(None, pool, None, None, None, 1, None),
              lambda: moe.moe_kv_copy_pages(None, [pool], None, 1), lambda: moe.moe_kv_copy_pages(None, [], None, 0)):
        assert _code(f) == e


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def _exact_turns(rot, base, kind, factor, trained):
    """f_i / (2 pi) 2^64 to 60 digits."""
    with localcontext() as c:
        c.prec = 70
        base, factor, rot = Decimal(base), Decimal(factor), Decimal(rot)
        ln = base.ln()
        if kind == moe.MOE_ROPE_SCALE_NTK:
            ln += factor.ln() * rot / (rot - 2)
        f = [(-2 * i * ln / rot).exp() for i in range(int(rot) // 2)]
        if kind == moe.MOE_ROPE_SCALE_LINEAR:
            f = [x / factor for x in f]
        if kind == moe.MOE_ROPE_SCALE_YARN:
            d = lambda t: rot * (trained / (2 * PI * t)).ln() / (2 * ln)     # noqa: E731
            lo = max(Decimal(0), d(32).to_integral_value(ROUND_FLOOR))
            hi = min(rot - 1, d(1).to_integral_value(ROUND_CEILING))
            r = [min(Decimal(1), max(Decimal(0), (i - lo) / max(Decimal("0.001"), hi - lo))) for i in range(len(f))]
            f = [x / factor * a + x * (1 - a) for x, a in zip(f, r)]
        return [x / (2 * PI) * 2 ** 64 for x in f]


@pytest.mark.parametrize("kind", range(4))
@pytest.mark.parametrize("rot,base,factor,trained", [
    (128, 10000.0, 4.0, 8192), (80, 10000.0, 8.0, 4096), (64, 500000.0, 32.0, 4096), (96, 1e6, 1.7, 32768), (16, 10000.0, 1.0, 2048),
    (1024, 10000.0, 3.0, 100), (6, 1.5, 1e6, 1 << 30), (32, 1.0000001, 2.5, 1), (48, 1e300, 1e10, 5000)])
def test_rope_table_is_rounded_from_the_frequencies(kind, rot, base, factor, trained):
    """A position's angle is off by p 2^-65 turns only if the table's entries are
    the 64-bit fractions next to f_i / (2 pi): half a unit, and 2^-84 of up to 2^62
    units for the arithmetic."""
    turns, _ = moe.moe_rope_table(rot, base, kind, factor, trained)
    want = _exact_turns(rot, base, kind, factor, trained)
    err = [abs(Decimal(int(t)) - w) for t, w in zip(turns, want)]
    assert max(err) <= Decimal(0.5 + 2.0 ** -20), (int(np.argmax([float(e) for e in err])), float(max(err)))
