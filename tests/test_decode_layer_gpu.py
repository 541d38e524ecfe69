"""A decode step's operators as they are used together: append (rotate, write),
attention and the expert FFN captured in one CUDA graph that is replayed as the
sequences grow, fork, end and move; every step against the fp64 formulas."""
import numpy as np
import pytest
import torch

import fp4_block_scaled_gb300 as moe
import oracle
import synth
from kv_setup import Pool, bf16_of, check_attention, f64, handle
from moe_setup import fill_layer
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.lib()
    yield


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_steps_in_a_replayed_graph(kv):
    hq, hkv, D, page, pages, B, row = 4, 2, 64, 16, 40, 6, 8
    H, E, I, k = hq * D, 8, 128, 2
    rng = np.random.default_rng(7)
    m = moe.moe_kv_pages_create(pages, page, B, row)
    cfg = moe.config(E, H, I, k, B, out_dtype=moe.MOE_OUT_F32)
    ffn = moe.moe_ffn_create(cfg, 0)
    s = torch.cuda.Stream()
    layers = [Pool(pages, hkv, page, D, kv, rng, poison=True) for _ in range(2)]
    try:
        es = fill_layer(ffn, cfg)
        ex = [synth.expert_canonical(H, I, e) for e in range(E)]
        turns, scale = moe.moe_rope_table(D, 10000.0)
        table_d = torch.from_numpy(turns.view(np.int64)).cuda()
        desc = moe.rope(table_d, D, moe.MOE_ROPE_HALF, scale)
        dev = dict(device="cuda")
        qkv = torch.zeros((2, B, hq + 2 * hkv, D), dtype=torch.bfloat16, **dev)
        qr = torch.zeros((2, B, hq, D), dtype=torch.bfloat16, **dev)
        att = torch.zeros((2, B, hq, D), dtype=torch.bfloat16, **dev)
        y = torch.zeros((2, B, H), dtype=torch.float32, **dev)
        pos, lens = torch.full((B,), -1, dtype=torch.int32, **dev), torch.zeros(B, dtype=torch.int32, **dev)
        tab = torch.full((B, row), -1, dtype=torch.int32, **dev)
        idx_np = synth.routing_uniform(B, E, k, seed=1)
        w_np = synth.routing_weights(B, k, seed=1)
        idx, w = torch.from_numpy(idx_np).cuda(), torch.from_numpy(w_np).cuda()
        with handle(hq, hkv, D, page, pages, B, row, kv, "bf16") as h:
            def step():
                for l in range(2):
                    x, ld = qkv[l], qkv[l].stride(0)
                    moe.moe_kv_append(h, layers[l].struct, x[:, hq:hq + hkv], x[:, hq + hkv:], pos, tab, B, rope=desc, q=x,
                                      q_out=qr[l], ldq=ld, ldk=ld, ldv=ld, stream=s)
                    moe.moe_attn_decode(h, layers[l].struct, qr[l], lens, tab, B, att[l], stream=s)
                    moe.moe_ffn_forward(ffn, att[l], idx, w, es.table, y[l], B, s)

            with torch.cuda.stream(s):
                step()                                               # first-use set-up outside the capture
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()

            seqs = [moe.moe_kv_pages_open(m) for _ in range(3)]
            for n, i in zip((30, 0, 15), seqs):                      # prompts, written in one call a layer
                moe.moe_kv_pages_extend(m, i, n)
            tab_np = np.full((B, row), -1, np.int32)

            def upload():
                for i in range(B):
                    tab_np[i] = moe.moe_kv_pages_row(m, i, row) if i in seqs else -1
                tab.copy_(torch.from_numpy(tab_np))
            upload()
            pk = torch.from_numpy(bf16_of(rng.standard_normal((2, 2, 45, hkv, D)))).cuda()
            pp = torch.tensor(list(range(30)) + list(range(15)), dtype=torch.int32, device="cuda")
            ps = torch.tensor([seqs[0]] * 30 + [seqs[2]] * 15, dtype=torch.int32, device="cuda")
            torch.cuda.synchronize()
            for l in range(2):
                moe.moe_kv_append(h, layers[l].struct, pk[l, 0], pk[l, 1], pp, tab, 45, seq=ps, rope=desc, stream=s)
            for t in range(24):
                if t == 5:
                    seqs.append(moe.moe_kv_pages_fork(m, seqs[0]))   # inside a page
                if t == 9:
                    seqs += [moe.moe_kv_pages_fork(m, seqs[0]), moe.moe_kv_pages_fork(m, seqs[2])]
                if t == 15:
                    for i in (seqs[0], seqs[3]):
                        moe.moe_kv_pages_free(m, i)
                        seqs.remove(i)
                copies = [c for c in (moe.moe_kv_pages_extend(m, i, 1) for i in seqs) if c]
                if t in (5, 9):
                    assert copies
                if t == 16:                                          # the freed pages leave holes below
                    moved = moe.moe_kv_pages_compact(m, pages)
                    assert len(moved)
                    copies += [tuple(c) for c in moved.tolist()]
                s.synchronize()
                upload()
                x = torch.from_numpy(bf16_of(rng.standard_normal((2, B, hq + 2 * hkv, D)))).cuda().view(torch.bfloat16)
                qkv.copy_(x)
                n = [moe.moe_kv_pages_length(m, i) if i in seqs else 0 for i in range(B)]
                lens.copy_(torch.tensor(n, dtype=torch.int32))
                pos.copy_(torch.tensor([v - 1 for v in n], dtype=torch.int32))      # -1: padding
                pairs = torch.tensor(copies, dtype=torch.int32, device="cuda").reshape(-1, 2)
                torch.cuda.synchronize()
                if copies:
                    moe.moe_kv_copy_pages(h, [p.struct for p in layers], pairs, len(copies), stream=s)
                with torch.cuda.stream(s):
                    graph.replay()
                assert moe.moe_kv_status(h, s) == moe.MOE_OK and moe.moe_ffn_status(ffn, s) == moe.MOE_OK
                for l in range(2):
                    for name, a in layers[l].bytes().items():
                        setattr(layers[l], name, a)
                    # the cache's newest rows: v as it was given (or its values to half an E4M3 step of the row's largest)
                    for i in seqs:
                        at = [int(p) for p in tab_np[i, :-(-n[i] // page)]]
                        for g in range(hkv):
                            v = okv.rows(layers[l].v, layers[l].vs, at, g, n[i])[-1]
                            want = f64(qkv[l, i, hq + hkv + g])
                            tol = 0.0 if kv == "bf16" else 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * 2 * np.abs(want).max() / 448
                            assert np.all(np.abs(v - want) <= tol)
                    check_attention(layers[l], f64(qr[l]), n, tab_np, page, f64(att[l]), None, D ** -0.5, out_bf16=True)
                    ref = oracle.moe_ffn([c for c, _ in ex], [q for _, q in ex], H, I,
                                         att[l].view(torch.int16).cpu().numpy().view(np.uint16).reshape(B, H), idx_np, w_np)
                    got = f64(y[l])
                    assert np.abs(got - ref).max() <= 2e-3 * np.sqrt(np.mean(ref ** 2)), t
            assert np.array_equal(f64(att[:, [i for i in range(B) if i not in seqs]]), 0 * f64(att[:, [i for i in range(B) if i not in seqs]]))
    finally:
        torch.cuda.synchronize()
        moe.moe_ffn_destroy(ffn)
        moe.moe_kv_pages_destroy(m)
