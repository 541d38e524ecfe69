"""Shared pieces of the cache's GPU tests: handles, pools, tables, tolerances."""
import contextlib

import numpy as np
import torch

import fp4_block_scaled_gb300 as moe
from oracle import kv as okv


@contextlib.contextmanager
def handle(hq, hkv, D, page=16, pages=1, seqs=1, row=1, kv="bf16", out="f32"):
    h = moe.moe_kv_create(moe.kv_config(
        hq, hkv, D, page, pages, seqs, row, kv_dtype=moe.MOE_KV_E4M3_UE8M0 if kv == "e4m3" else moe.MOE_KV_BF16,
        out_dtype=moe.MOE_OUT_F32 if out == "f32" else moe.MOE_OUT_BF16), 0)
    try:
        yield h
    finally:
        torch.cuda.synchronize()
        moe.moe_kv_destroy(h)


def bf16_of(x):
    """fp array -> bf16 bits (host int16)."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy()


def f64(t):
    """bf16 / fp32 device tensor -> fp64 host array."""
    return t.float().cpu().numpy().astype(np.float64)


class Pool:
    """A pool of random rows on the host and the device; `poison` fills every
    row with NaN first, so that only rows written by put() are numbers."""

    def __init__(self, pages, hkv, page, D, kv, rng, poison=False, spread=0.0):
        shape = (pages, hkv, page, D)
        self.kv = kv
        if kv == "bf16":
            self.k, self.v = (bf16_of(np.full(shape, np.nan) if poison else rng.standard_normal(shape)) for _ in range(2))
            self.ks = self.vs = None
        else:
            code = lambda: np.where((c := rng.integers(0, 256, shape)) & 0x7F == 0x7F, 0x38, c)  # noqa: E731
            self.k, self.v = (np.full(shape, 0x7F, np.uint8) if poison else code().astype(np.uint8) for _ in range(2))
            # codes reach 448: scales around 2^-7 give values around 1
            byte = lambda: np.clip(np.rint(119 + spread * rng.standard_normal(shape[:3])), 1, 254)  # noqa: E731
            self.ks, self.vs = (np.full(shape[:3], 255, np.uint8) if poison else byte().astype(np.uint8) for _ in range(2))
        self.dev = {n: torch.from_numpy(getattr(self, n)).cuda() for n in ("k", "v", "ks", "vs") if getattr(self, n) is not None}
        self.struct = moe.kv_pool(*[self.dev[n] for n in ("k", "v", "ks", "vs") if n in self.dev])

    def upload(self):
        for n, t in self.dev.items():
            t.copy_(torch.from_numpy(getattr(self, n)))

    def bytes(self):
        torch.cuda.synchronize()
        return {n: t.cpu().numpy() for n, t in self.dev.items()}


def table(lens, page, pages, row, rng, share=()):
    """Random page table; (a, b, n) in share: b's first n pages are a's."""
    ids = iter(rng.permutation(pages).astype(np.int32))
    t = np.full((len(lens), row), -1, np.int32)
    for b, n in enumerate(lens):
        need = -(-min(int(n), row * page) // page) if n > 0 else 0
        t[b, :need] = [next(ids) for _ in range(need)]
    for a, b, n in share:
        t[b, :n] = t[a, :n]
    return t


def check_attention(pool, q, lens, tab, page, out, lse, scale, softcap=0.0, window=0, out_bf16=False, num_pages=None):
    """Every head of every sequence against the fp64 formulas.

    Bounds: a score is a sum of D exact products in fp32, its error taken as
    4 sqrt(D) 2^-24 of the sum of the products' sizes, times scale, and a
    relative 2^-21 for scaling, tanh cap and exponent (max(1, |s|) of them);
    the weights are off by the same relative amounts, twice (numerator and
    denominator); weights enter the product with 16 significant bits for a bf16
    output (2^-17), 22 at least for an fp32 one (2^-21), and n fp32 additions are
    taken as 4 sqrt(n) 2^-24.  All of it applies to
    sum_j p_j |v_j|.  A bf16 output is off by half a step more.

    An E4M3 row's weight is w_j = p_j s_j (s_j its scale) times codes c_j, held
    as two f16 terms relative to a reference that keeps the largest weight so
    far at 2^7 or above: f16's smallest steps are 2^-24, so each term is off by at
    most 2^-25 beside its relative error, together 2^-24 = 2^-31 2^7.  The
    output is therefore off by up to 2^-31 max_i w_i sum_j |c_jd| more (this
    matters only where the row that dominates has a code of zero)."""
    hkv, D = pool.k.shape[1], pool.k.shape[3]
    B, hq = q.shape[:2]
    G = hq // hkv
    num_pages = num_pages or pool.k.shape[0]
    for b in range(B):
        n = max(0, min(int(lens[b]), tab.shape[1] * page))
        ids = [int(p) if 0 <= p < num_pages else None for p in tab[b, :-(-n // page)]]
        seen = np.repeat(np.array([p is not None for p in ids], bool), page)[:n]
        j = np.arange(n)
        if window:
            seen = seen & (j >= n - window)
        for h in range(hkv):
            g = slice(h * G, (h + 1) * G)
            k = okv.rows(pool.k, pool.ks, ids, h, n)
            v = okv.rows(pool.v, pool.vs, ids, h, n)
            ref, rl, size, prod, big, p = okv.attention(q[b, g], k, v, seen, scale, softcap)
            ds = 4 * np.sqrt(D) * 2.0 ** -24 * prod + 2.0 ** -21 * max(1.0, big)
            sums = 4 * np.sqrt(max(1, n)) * 2.0 ** -24
            tol = (2 * ds + (2.0 ** -16 if out_bf16 else 2.0 ** -20) + sums)[:, None] * size + 1e-37
            if pool.ks is not None and p.size:
                f = np.concatenate([okv.scale_of(pool.vs[i, h]) if i is not None else np.zeros(page) for i in ids])[:n][seen]
                codes = np.abs(v[seen] / f[:, None]).sum(0)
                tol = tol + 2.0 ** -31 * (p * f).max(1)[:, None] * codes
            if out_bf16:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
            err = np.abs(out[b, g] - ref)
            assert np.all(err <= tol), (b, h, n, float((err / tol).max()))
            if lse is not None:
                none = np.isinf(rl)
                assert np.array_equal(np.isneginf(lse[b, g]), none), (b, h, n)
                el = np.abs(np.where(none, 0.0, lse[b, g] - np.where(none, 0.0, rl)))
                assert np.all(el <= ds + sums + 2.0 ** -22 * np.maximum(1, np.abs(np.where(none, 0, rl)))), (b, h, n, el)
