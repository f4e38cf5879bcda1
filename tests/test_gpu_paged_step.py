"""GPU: the paged cache operators together, as a verify step uses them.

VerifyStep with pages: the prefix written, attention over the pages, acceptance, the accepted path committed, and the
next step's attention over the grown cache; with eviction: weights collected and the cache cut down after each step.
Tolerances: paged_helpers.
"""
import math

import numpy as np
import pytest
import torch

import paged_helpers as H
from eagle_speculative_decoding_tree_gb300 import binding as B
from eagle_speculative_decoding_tree_gb300 import synth
from eagle_speculative_decoding_tree_gb300.step import VerifyStep

pytestmark = pytest.mark.gpu


def see_of(st):
    m = st.anc_mask.cpu().numpy().view(np.uint64)
    return np.stack([(m[:, :, j // 64] >> np.uint64(j % 64)) & np.uint64(1) for j in range(st.R)], -1).astype(bool)


def check_layer(st, l, see, seq, table, lse):
    """The layer's outputs against attention in 64 bits over the pages as they are."""
    w, bf = st.w, st.w.dtype == "bf16"
    q, tk, tv, kp, vp = (H.f64(x[l]) for x in (st.q, st.tk, st.tv, st.kp, st.vp))
    out, z = H.f64(st.out[l]), H.f64(lse)
    for b in range(st.B):
        k, v = H.rows_of(kp, table[b], seq[b]), H.rows_of(vp, table[b], seq[b])
        adds, rel = (144, 2.0 ** -16) if bf else H.fp32_kinds(st.R * w.group)
        ref = H.attention(q[b], k, v, tk[b], tv[b], see[b], seq[b], st.R, 1 / math.sqrt(w.head_dim), adds=adds)
        mass = H.attention(q[b], k, np.abs(v), tk[b], np.abs(tv[b]), see[b], seq[b], st.R, 1 / math.sqrt(w.head_dim))[0]
        H.check_attention(out[b], z[b], ref, bf, rel * mass)


@pytest.mark.parametrize("name,prefix,layers,batch,page", [("llama8b", 333, 2, 1, 64), ("concurrency", 200, 2, 3, 16),
                                                           ("vicuna7b", 130, 1, 1, 128), ("long128k", 510, 2, 1, 32),
                                                           ("tiny", 100, 2, 2, 16)])
def test_verify_steps_over_pages(name, prefix, layers, batch, page):
    w = synth.WORKLOADS[name].with_(prefix=prefix, prefix_min=min(prefix, 65), vocab=2048)
    st = VerifyStep(w, batch=batch, layers=layers, page_size=page)
    flat = VerifyStep(w, batch=batch, layers=layers)  # contiguous: the same tree, acceptance and rows
    see, table, seq = see_of(st), st.table.cpu().numpy(), st.seq_len0.copy()
    for step in range(2):  # the second step reads what the first committed
        for l in range(layers):
            st.attn_layer(l, lse=True)
            check_layer(st, l, see, seq, table, st.lse)
        st.accept()
        st.commit()
        flat.run(reset=False)
        torch.cuda.synchronize()
        assert torch.equal(st.acc.n_acc, flat.acc.n_acc) and torch.equal(st.acc.out_tok, flat.acc.out_tok)
        assert torch.equal(st.commit_pos, flat.commit_pos) and torch.equal(st.seq_len, flat.seq_len)
        assert int(st.acc.status) == 0 and int(st.attn_ws[:4].view(torch.int32)) == 0
        seq = st.seq_len.cpu().numpy()
        for l in range(layers):
            for pages, cache in ((st.kp[l], flat.kc[l]), (st.vp[l], flat.vc[l])):
                for b in range(batch):
                    assert np.array_equal(H.rows_of(H.f64(pages), table[b], seq[b]), H.f64(cache)[b, :, :seq[b]])


@pytest.mark.parametrize("name", ["llama8b", "concurrency"])
def test_verify_steps_with_eviction(name):
    """Two steps, each of which cuts the cache down: the rows and weights that stay, and attention over them."""
    w = synth.WORKLOADS[name].with_(prefix=300, prefix_min=60, vocab=2048)
    layers, batch, (limit, budget, sink, recent) = 2, 1 if name == "llama8b" else 4, (150, 120, 4, 32)
    st = VerifyStep(w, batch=batch, layers=layers, page_size=16, evict=(limit, budget, sink, recent))
    see = see_of(st)
    table, seq = st.table.cpu().numpy(), st.seq_len0.copy()
    scale = 1 / math.sqrt(w.head_dim)
    # what every head of every layer holds: K, V, weights
    held = [[[H.rows_of(H.f64(x[l]), table[b], seq[b]) for x in (st.kp, st.vp)] + [np.zeros((w.n_kv_heads, seq[b]))]
             for b in range(batch)] for l in range(layers)]
    for step in range(2):
        for l in range(layers):
            st.attn_layer(l)
            check_layer(st, l, see, seq, table, st.lse_layers[l])
        st.accept()
        st.commit()
        for l in range(layers):
            st.add_weights(l)
        torch.cuda.synchronize()
        n_acc, path = st.acc.n_acc.cpu().numpy(), st.acc.path.cpu().numpy()
        got = [H.f64(x) for x in st.weights]
        for l in range(layers):
            q, z = H.f64(st.q[l]), H.f64(st.lse_layers[l])
            for b in range(batch):
                nodes = path[b, : n_acc[b] + 1]
                old = held[l][b]
                for i, t in enumerate((st.tk, st.tv)):
                    old[i] = np.concatenate((old[i], H.f64(t[l])[b][:, nodes]), 1)
                L = old[0].shape[1]
                add, err = H.weights(q[b, nodes], z[b, nodes], old[0], L, scale)
                want = add + np.concatenate((old[2], np.zeros((w.n_kv_heads, len(nodes)))), 1)
                have = H.rows_of(got[l], table[b], L)
                assert (np.abs(have - want) <= err + 2 * H.U32 * want).all()
                old[2] = have  # (which of two close weights is larger is the library's to say)
        st.evict_long()
        torch.cuda.synchronize()
        assert int(st.acc.status) == 0
        kept, table, new = st.kept.cpu().numpy(), st.table.cpu().numpy(), st.seq_len.cpu().numpy()
        for b in range(batch):
            L = held[0][b][0].shape[1]
            assert new[b] == (budget if L > limit else L)
            for l in range(layers):
                for h in range(w.n_kv_heads):
                    if L > limit:
                        rows = H.kept_rows(held[l][b][2][h].astype(np.float32), L, budget, sink, recent)
                        assert np.array_equal(kept[l, b, h], rows)
                held[l][b] = [np.stack([x[h][kept[l, b, h]] for h in range(w.n_kv_heads)]) if L > limit else x
                              for x in held[l][b]]
                for x, want in zip((st.kp, st.vp, st.weights), held[l][b]):
                    assert np.array_equal(H.rows_of(H.f64(x[l]), table[b], new[b]), want)
        seq = new.copy()


def test_a_captured_step_with_eviction_repeats():
    """The whole step in one graph: reset, attention, acceptance, commit, weights, eviction; the same bits each time."""
    w = synth.WORKLOADS["concurrency"].with_(prefix=400, prefix_min=90, vocab=2048)
    st = VerifyStep(w, batch=3, layers=2, page_size=32, evict=(200, 160, 4, 32))
    st.run()
    torch.cuda.synchronize()
    state = lambda: [t.clone() for t in (*st.out, st.table, st.spare, st.seq_len, st.kept, *st.weights, *st.kp, st.acc.path)]
    first = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            st.run()
        for _ in range(3):
            graph.replay()
    side.synchronize()
    for x, y in zip(first, state()):
        assert torch.equal(x, y)
    assert int(st.acc.status) == 0


def test_page_sizes_are_checked():
    w = synth.WORKLOADS["llama8b"]
    for kw in (dict(page_size=48), dict(page_size=64, cache_bits=8), dict(evict=(10, 5, 1, 1))):
        with pytest.raises(ValueError):
            VerifyStep(w, layers=1, **kw)
