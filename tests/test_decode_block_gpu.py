"""A whole decode layer from the library's calls, captured in one graph and
replayed token by token: norm -> q/k/v projection -> rotate and append ->
attention -> output projection -> norm with the residual -> router -> experts ->
the next norm's residual.  Every stage against the fp64 formulas on the GPU's own
inputs of that stage."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
import oracle
import synth
from kv_setup import Pool, check_attention
from kv_setup import handle as kv_handle
from lin_setup import MODE, TYPE, Weights, code_buffers, f64, handle, rand
from moe_setup import fill_layer
from oracle import lin as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


def near(y, x, w, fmt, bf16=True):
    """y is the product of bf16 rows x, quantised, with the weights."""
    ref, total = ol.linear(ol.values(*ol.quantise(f64(x), fmt), fmt), w.values())
    tol = ol.linear_tolerance(w.K, total)
    tol = tol + (np.abs(ref) + tol) * 2.0 ** -8 if bf16 else tol
    assert np.all(np.abs(f64(y) - ref) <= tol)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("B", [1, 5, 20])
def test_layer_steps_in_a_replayed_graph(fmt, B):
    hq, hkv, D, page, row = 4, 2, 64, 16, 4
    H, E, I, k, eps = hq * D, 8, 128, 2, 1e-5
    rng = np.random.default_rng(B)
    s, m = torch.cuda.Stream(), MODE[fmt]
    pool = Pool(B * row, hkv, page, D, "bf16", rng)
    tab_np = rng.permutation(B * row).reshape(B, row).astype(np.int32)
    cfg = moe.config(E, H, I, k, B, out_dtype=moe.MOE_OUT_F32)
    ffn = moe.moe_ffn_create(cfg, 0)
    try:
        es = fill_layer(ffn, cfg)
        ex = [synth.expert_canonical(H, I, e) for e in range(E)]
        router = torch.from_numpy(synth.router_weights_bf16(E, H).view(np.int16)).cuda()
        turns, scale = moe.moe_rope_table(D, 10000.0)
        freqs = torch.from_numpy(turns.view(np.int64)).cuda()
        rope = moe.rope(freqs, D, moe.MOE_ROPE_HALF, scale)
        f32, bf16 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        res, mid, fin = (torch.zeros((B, H), **f32) for _ in range(3))
        tab = torch.from_numpy(tab_np).cuda()
        pos, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        u1, u2, u3, o = (torch.zeros((B, H), **bf16) for _ in range(4))
        qkv = torch.zeros((B, hq + 2 * hkv, D), **bf16)
        qr, att = torch.zeros((B, hq, D), **bf16), torch.zeros((B, hq, D), **bf16)
        logits, topk_w = torch.zeros((B, E), **f32), torch.zeros((B, k), **f32)
        idx = torch.zeros((B, k), dtype=torch.int32, device="cuda")
        y = torch.zeros((B, H), **f32)
        q1, s1 = code_buffers(B, H, fmt)
        g1, g2, g3 = ((1 + 0.1 * rand(rng, (H,))).to(torch.bfloat16) for _ in range(3))
        with handle(B, H) as h, kv_handle(hq, hkv, D, page, B * row, B, row, "bf16", "bf16") as kv:
            wq, wo = Weights(h, (hq + 2 * hkv) * D, H, rng, 118, 121), Weights(h, H, H, rng, 118, 121)
            n1, n2, n3 = (moe.norm(g, H, eps, t, TYPE["f32"]) for g, t in ((g1, TYPE["f32"]), (g2, TYPE["bf16"]), (g3, TYPE["f32"])))
            ld = (hq + 2 * hkv) * D
            torch.cuda.synchronize()

            def step():
                moe.moe_rms_norm(h, n1, res, B, out=u1, act_mode=m, codes=q1, scales=s1, stream=s)
                moe.moe_linear(h, wq.desc, m, q1, B, qkv, TYPE["bf16"], x_scales=s1, stream=s)
                moe.moe_kv_append(kv, pool.struct, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, tab, B, rope=rope, q=qkv, q_out=qr,
                                  ldq=ld, ldk=ld, ldv=ld, stream=s)
                moe.moe_attn_decode(kv, pool.struct, qr, lens, tab, B, att, stream=s)
                moe.moe_linear(h, wo.desc, m, att, B, o, TYPE["bf16"], stream=s)
                moe.moe_rms_norm(h, n2, o, B, residual=res, residual_out=mid, out=u2, stream=s)
                moe.moe_router_topk(ffn, u2, router, B, idx, topk_w, logits=logits, stream=s)
                moe.moe_ffn_forward(ffn, u2, idx, topk_w, es.table, y, B, s)
                moe.moe_rms_norm(h, n3, y, B, residual=mid, residual_out=fin, out=u3, stream=s)

            lens.fill_(1)
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                step()                                               # first-use set-up of the experts outside the capture
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
            for t in range(20):
                res.copy_(rand(rng, (B, H), 2.0))
                pos.fill_(t), lens.fill_(t + 1)
                torch.cuda.synchronize()
                with torch.cuda.stream(s):
                    graph.replay()
                assert moe.moe_lin_status(h, s) == moe.MOE_OK and moe.moe_kv_status(kv, s) == moe.MOE_OK
                assert moe.moe_ffn_status(ffn, s) == moe.MOE_OK
                if t not in (0, 7, 19):
                    continue
                for u, r, g in ((u1, res, g1), (u2, mid, g2), (u3, fin, g3)):
                    want = ol.norm(f64(r), f64(g), eps)
                    assert np.all(np.abs(f64(u) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -19))
                assert torch.equal(mid, o.float() + res) and torch.equal(fin, y + mid)
                near(qkv.view(B, -1), u1, wq, fmt)
                near(o, att.view(B, H), wo, fmt)
                for name, a in pool.bytes().items():
                    setattr(pool, name, a)
                check_attention(pool, f64(qr), [t + 1] * B, tab_np, page, f64(att), None, D ** -0.5, out_bf16=True)
                ri, rw = oracle.topk_softmax(f64(logits), k)
                assert np.array_equal(idx.cpu().numpy(), ri)
                ref = oracle.moe_ffn([c for c, _ in ex], [q for _, q in ex], H, I, u2.view(torch.int16).cpu().numpy().view(np.uint16), ri,
                                     topk_w.cpu().numpy())
                assert np.abs(f64(y) - ref).max() <= 2e-3 * np.sqrt(np.mean(ref ** 2))
    finally:
        torch.cuda.synchronize()
        moe.moe_ffn_destroy(ffn)
