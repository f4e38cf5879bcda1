"""GPU: the 8-bit cache operators together, as a verify step uses them.

VerifyStep with cache_bits = 8: the prefix quantised, attention over the codes, acceptance, the
accepted path committed into the codes, and the next step's attention over the grown cache; and
the path before it: projection rows -> norms and rotation -> cache write / tree attention.
"""
import math

import numpy as np
import pytest
import torch

import kvq_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B
from eagle_speculative_decoding_tree_gb300 import synth
from eagle_speculative_decoding_tree_gb300.step import VerifyStep

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def see_of(anc_mask, R):
    m = anc_mask.cpu().numpy().view(np.uint64)
    return np.stack([(m[:, :, j // 64] >> np.uint64(j % 64)) & np.uint64(1) for j in range(R)], -1).astype(bool)


def close(out, lse, ref):
    """bf16 output: half a step of the output, and P's terms and fp32 against sum p |v| (the
    derivation stands in the attention tests; precise, few hundred keys: under 2^-14)."""
    o, r, mass = out.double().cpu().numpy(), ref[0], ref[2]
    assert (np.abs(o - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -14 * mass + 1e-6).all()
    if lse is not None:
        assert np.abs(lse.double().cpu().numpy() - ref[1]).max() <= 1e-4


@pytest.mark.parametrize("name,prefix,layers,batch", [("llama8b", 333, 2, 1), ("concurrency", 200, 2, 3),
                                                      ("vicuna7b", 130, 1, 1), ("long128k", 510, 2, 1)])
def test_verify_steps_over_an_8_bit_cache(name, prefix, layers, batch):
    w = synth.WORKLOADS[name].with_(prefix=prefix, prefix_min=min(prefix, 65), vocab=2048)
    st = VerifyStep(w, batch=batch, layers=layers, cache_bits=8, keep_host=True)
    ref_step = VerifyStep(w, batch=batch, layers=layers)  # 16-bit: the same acceptance
    val = lambda bits: torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).double().numpy()
    G, D, P = w.group, w.head_dim, w.max_seq
    codes, scales, host = [], [], []
    for q, kc, vc, tk, tv in st.host:
        host.append([val(x) for x in (q, tk, tv)])
        for x in (kc, vc):
            c, s = np.zeros(x.shape, np.uint8), np.zeros((batch, w.n_kv_heads, -(-P // 64)), np.float32)
            for b in range(batch):
                for h in range(w.n_kv_heads):
                    H.append(c[b, h], s[b, h], val(x[b, h])[:st.seq_len0[b]], 0)
            codes.append(c)
            scales.append(s)
    see = see_of(st.anc_mask, st.R)
    seq = st.seq_len0.copy()
    for step in range(2):  # the second step reads what the first committed
        for l in range(layers):
            st.attn_layer(l, lse=True)
            q, tk, tv = host[l]
            kv = [H.values(codes[2 * l + i], scales[2 * l + i]) for i in (0, 1)]
            ref = H.attention(q, kv[0], kv[1], tk, tv, seq, np.full(batch, st.R), see, 1 / math.sqrt(D))
            close(st.out[l], st.lse, ref)
        st.accept()
        st.commit()
        torch.cuda.synchronize()
        n_acc, path = st.acc.n_acc.cpu().numpy(), st.acc.path.cpu().numpy()
        if step == 0:
            ref_step.run(reset=False)
            assert torch.equal(st.acc.n_acc, ref_step.acc.n_acc) and torch.equal(st.acc.out_tok, ref_step.acc.out_tok)
            assert torch.equal(st.commit_pos, ref_step.commit_pos)
        for l in range(layers):
            for i in (0, 1):
                for b in range(batch):
                    rows = host[l][1 + i][b][:, path[b, :n_acc[b] + 1]]
                    for h in range(w.n_kv_heads):
                        H.append(codes[2 * l + i][b, h], scales[2 * l + i][b, h], rows[h], int(seq[b]))
        seq = seq + n_acc + 1
        assert np.array_equal(st.seq_len.cpu().numpy(), seq) and int(st.acc.status) == 0
        for l in range(layers):
            for got, gs, i in ((st.k8[l], st.ks[l], 0), (st.v8[l], st.vs[l], 1)):
                want = H.decode(codes[2 * l + i])
                live = np.arange(P)[None, :] < seq[:, None]
                g = H.decode(got.cpu().numpy())
                assert np.array_equal(np.moveaxis(g, 2, 1)[live], np.moveaxis(want, 2, 1)[live])
                assert np.array_equal(gs.cpu().numpy(), scales[2 * l + i])


def test_cache_bits_are_checked():
    with pytest.raises(ValueError, match="cache_bits"):
        VerifyStep(synth.WORKLOADS["tiny"], cache_bits=8)
    with pytest.raises(ValueError, match="cache_bits"):
        VerifyStep(synth.WORKLOADS["llama8b"], cache_bits=4)


def test_from_projection_to_attention_in_one_graph():
    """Prompt projection -> rotation -> cache; tree projection -> rotation -> attention -> commit,
    captured once and replayed on other data."""
    Bn, N, R, Hq, Hk, D, P, maxd = 2, 150, 9, 8, 2, 128, 256, 3
    width = (Hq + 2 * Hk) * D
    bf = torch.bfloat16
    new = lambda *s: torch.empty(*s, dtype=bf, device="cuda")
    x0, x1 = new(Bn, N, width), new(Bn, R, width)
    wq, wk = [(1 + 0.1 * torch.randn(D, device="cuda")).to(bf) for _ in range(2)]
    inv = (10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)).float()
    pos0 = torch.arange(N, device="cuda", dtype=torch.int32).repeat(Bn, 1).contiguous()
    par = np.array([-1, 0, 0, 1, 1, 2, 3, 3, 5])
    dep, see = np.zeros(R, int), np.eye(R, dtype=bool)
    for i in range(1, R):
        dep[i] = dep[par[i]] + 1
        see[i] |= see[par[i]]
    mask = torch.from_numpy(np.array([int(sum(1 << j for j in range(R) if see[i, j])) for i in range(R)], np.int64))
    mask = mask.cuda().repeat(Bn, 1)[..., None].contiguous()
    seq0 = np.array([N, 97])
    seq = i32(seq0)
    q0, k0, v0 = new(Bn, N, Hq, D), new(Bn, Hk, N, D), new(Bn, Hk, N, D)
    q1, k1, v1 = new(Bn, R, Hq, D), new(Bn, Hk, R, D), new(Bn, Hk, R, D)
    kc, vc = [torch.zeros(Bn, Hk, P, D, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    ks, vs = [torch.zeros(Bn, Hk, P // 64, device="cuda") for _ in range(2)]
    pos1 = i32(seq0[:, None] + dep[None])
    out, out2 = new(Bn, R, Hq, D), new(Bn, R, Hq, D)
    d0 = B.QkNormRopeDesc(Bn, N, Hq, Hk, D, D, 0, 0, 1e-6, B.EAGLE_BF16)
    d1 = B.QkNormRopeDesc(Bn, R, Hq, Hk, D, D, 0, 0, 1e-6, B.EAGLE_BF16)
    dw = B.KvqDesc(Bn, Hk, D, P, N, B.EAGLE_BF16)
    da = B.AttnDesc(Bn, R, Hq, Hk, D, P, 1 / math.sqrt(D), B.EAGLE_BF16, 0, B.EAGLE_BF16, B.EAGLE_ATTN_PRECISE)
    dc = B.CommitDesc(1, Bn, Hk, D, R, P, maxd, B.EAGLE_BF16, 0, B.EAGLE_BF16)
    ws = torch.zeros(B.workspace_size(B.EAGLE_WS_TREE_ATTN_KVQ, da), dtype=torch.uint8, device="cuda")
    lay = B.KvqLayerPointers([kc], [ks], [vc], [vs], [k1], [v1])
    n_acc, path = i32([2, 3]), i32([[0, 1, 3, -1], [0, 2, 5, 8]])
    zero, start, cpos = i32([0, 0]), i32(seq0), i32(np.zeros((Bn, maxd + 1)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        seq.copy_(start)
        B.eagle_qk_norm_rope(d0, x0, wq, wk, inv, pos0, q0, k0, v0)
        B.eagle_kvq_write(dw, k0, v0, zero, start, kc, ks, vc, vs, status)
        B.eagle_qk_norm_rope(d1, x1, wq, wk, inv, pos1, q1, k1, v1)
        B.eagle_tree_attn_kvq(da, q1, kc, ks, vc, vs, k1, v1, seq, mask, out, None, ws)
        B.eagle_kvq_commit(dc, lay, n_acc, path, seq, cpos, status=status)
        B.eagle_tree_attn_kvq(da, q1, kc, ks, vc, vs, k1, v1, seq, mask, out2, None, ws)

    fill = lambda seed: [x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed + i)))
                         for i, x in enumerate((x0, x1))]
    fill(1)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 5):
        fill(seed)
        g.replay()
        torch.cuda.synchronize()
        assert int(status) == 0 and int(ws[:4].view(torch.int32)) == 0
        assert seq.cpu().tolist() == [N + 3, 97 + 4]
        # each stage against 64 bits on the stage's own inputs
        f = lambda t: t.double().cpu().numpy()
        qr, qb = H.rope(f(x1).reshape(Bn, R, Hq + 2 * Hk, D)[:, :, :Hq], f(wq), 1e-6, pos1.cpu().numpy(),
                        inv.cpu().numpy(), D, False)
        assert (np.abs(f(q1) - qr) <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -16 * qb).all()
        for res, n in ((out, seq0), (out2, seq0 + np.array([3, 4]))):
            cs = []
            for t, rows in ((k0, k1), (v0, v1)):
                c, s = np.zeros((Bn, Hk, P, D), np.uint8), np.zeros((Bn, Hk, P // 64), np.float32)
                for b in range(Bn):
                    for h in range(Hk):
                        H.append(c[b, h], s[b, h], f(t)[b, h, :seq0[b]], 0)
                        if n[b] > seq0[b]:
                            H.append(c[b, h], s[b, h], f(rows)[b, h][path.cpu().numpy()[b, :n[b] - seq0[b]]], int(seq0[b]))
                cs.append(H.values(c, s))
            ref = H.attention(f(q1), cs[0], cs[1], f(k1), f(v1), n, [R] * Bn, np.stack([see] * Bn), 1 / math.sqrt(D))
            close(res, None, ref)
