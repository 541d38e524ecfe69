"""The cache's calls on streams and in graphs: a handle's first calls captured,
two handles at work at once, the largest batch, calls back to back."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
from busy_stream import busy_default_stream
from kv_setup import Pool, bf16_of, check_attention, f64, handle, table
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


class Step:
    """One layer's step for sequences of the given lengths: append the last
    token of each, attend."""

    def __init__(self, lens, hq, hkv, D, page, kv, seed):
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.D, self.hq = lens, page, D, hq
        B, row = len(lens), max(-(-n // page) for n in lens)
        self.B, self.row, self.pages = B, row, sum(-(-n // page) for n in lens) + 1
        self.tab = table(lens, page, self.pages, row, rng)
        self.pool = Pool(self.pages, hkv, page, D, kv, rng)
        self.qkv = torch.from_numpy(bf16_of(rng.standard_normal((B, hq + 2 * hkv, D)))).cuda().view(torch.bfloat16)
        self.q, self.k, self.v = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:]
        self.pos = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
        self.ld, self.td = self.pos + 1, torch.from_numpy(self.tab).cuda()
        turns, scale = moe.moe_rope_table(D, 10000.0)
        self.freqs = torch.from_numpy(turns.view(np.int64)).cuda()
        self.rope = moe.rope(self.freqs, D, moe.MOE_ROPE_HALF, scale)
        self.qr = torch.zeros((B, hq, D), dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros((B, hq, D), dtype=torch.float32, device="cuda")
        self.lse = torch.zeros((B, hq), dtype=torch.float32, device="cuda")

    def run(self, h, s=None):
        ld = self.qkv.stride(0)
        moe.moe_kv_append(h, self.pool.struct, self.k, self.v, self.pos, self.td, self.B, rope=self.rope, q=self.q,
                          q_out=self.qr, ldq=ld, ldk=ld, ldv=ld, stream=s)
        moe.moe_attn_decode(h, self.pool.struct, self.qr, self.ld, self.td, self.B, self.out, lse=self.lse, stream=s)

    def check(self, some=None):
        for n, a in self.pool.bytes().items():
            setattr(self.pool, n, a)
        at = np.arange(self.B) if some is None else np.array(some)
        check_attention(self.pool, f64(self.qr)[at], [self.lens[i] for i in at], self.tab[at], self.page, f64(self.out)[at],
                        f64(self.lse)[at], self.D ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_handles_first_calls_may_be_captured(kv):
    st = Step([300, 17, 1, 2000], 8, 2, 64, 16, kv, 1)
    s = torch.cuda.Stream()
    with handle(8, 2, 64, 16, st.pages, st.B, st.row, kv) as h:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        other = torch.zeros_like(st.qr)
        with torch.cuda.graph(g, stream=s):
            moe.moe_rope(h, st.rope, st.pos, st.B, q=st.q, q_out=other, ldq=st.qkv.stride(0), stream=s)
            st.run(h, s)
        assert not st.out.any()                                      # nothing ran yet
        for _ in range(3):
            st.out.fill_(float("nan"))
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                g.replay()
            s.synchronize()
            st.check()
            assert torch.equal(other.view(torch.int16), st.qr.view(torch.int16))
        assert moe.moe_kv_status(h, s) == moe.MOE_OK


def test_two_handles_at_work_at_once():
    """Each handle has a workspace of its own: steps of two models on two
    streams, many in flight, give what they give alone, bit for bit."""
    a, b = Step([5000, 300, 44], 16, 4, 128, 32, "bf16", 2), Step([700] * 9, 8, 8, 64, 16, "e4m3", 3)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with handle(16, 4, 128, 32, a.pages, a.B, a.row, "bf16") as ha, handle(8, 8, 64, 16, b.pages, b.B, b.row, "e4m3") as hb:
        a.run(ha), b.run(hb)
        torch.cuda.synchronize()
        wa, wb = a.out.clone(), b.out.clone()
        a.check(), b.check()
        for _ in range(20):
            a.out.zero_(), b.out.zero_()
            torch.cuda.synchronize()
            for _ in range(10):
                a.run(ha, s1), b.run(hb, s2)
            torch.cuda.synchronize()
            assert torch.equal(a.out, wa) and torch.equal(b.out, wb)
        assert moe.moe_kv_status(ha) == moe.MOE_OK and moe.moe_kv_status(hb) == moe.MOE_OK


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_the_largest_batch(kv):
    lens = [1 + (i * 53) % 90 for i in range(2048)]
    lens[700] = 4000
    st = Step(lens, 4, 2, 64, 16, kv, 4)
    with handle(4, 2, 64, 16, st.pages, st.B, st.row, kv) as h:
        st.run(h)
        torch.cuda.synchronize()
        assert moe.moe_kv_status(h) == moe.MOE_OK
    st.check(list(range(0, 2048, 29)) + [699, 700, 701, 2047])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_new_handle_works_at_once_on_a_stream_beside_a_busy_default_one(kv):
    """The tickets of rows split among CTAs are zero when the handle is there,
    whatever the memory held before and whatever the default stream has to do
    (torch's other streams do not wait for it)."""
    st = Step([5000, 300, 44], 8, 2, 64, 16, kv, 5)
    s = torch.cuda.Stream()
    cfg = moe.kv_config(8, 2, 64, 16, st.pages, st.B, st.row, kv_dtype=moe.MOE_KV_E4M3_UE8M0 if kv == "e4m3" else moe.MOE_KV_BF16,
                        out_dtype=moe.MOE_OUT_F32)
    with handle(8, 2, 64, 16, st.pages, st.B, st.row, kv) as h:     # kernels loaded
        st.run(h, s)
        torch.cuda.synchronize()
    for _ in range(3):
        st.out.fill_(float("nan"))
        with busy_default_stream():
            h = moe.moe_kv_create(cfg, 0)
            for _ in range(4):
                st.run(h, s)
            s.synchronize()
        assert moe.moe_kv_status(h, s) == moe.MOE_OK
        moe.moe_kv_destroy(h)
        st.check()
