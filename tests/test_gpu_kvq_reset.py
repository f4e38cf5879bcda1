"""GPU: a verify step over an 8-bit cache repeats itself after reset()."""
import pytest
import torch

from eagle_speculative_decoding_tree_gb300 import synth
from eagle_speculative_decoding_tree_gb300.step import VerifyStep

pytestmark = pytest.mark.gpu


def result(st):
    """Outputs, acceptance and the cache's rows, after a run."""
    torch.cuda.synchronize()
    n = st.seq_len.tolist()
    rows = [t[b, :, : n[b]].clone() for t in st.k8 + st.v8 for b in range(st.B)]
    scales = [t[b, :, : -(-n[b] // 64)].clone() for t in st.ks + st.vs for b in range(st.B)]
    return [t.clone() for t in st.out] + [st.acc.n_acc.clone(), st.acc.out_tok.clone(), st.seq_len.clone()] + rows + scales


def step(name, prefix, batch, layers):
    w = synth.WORKLOADS[name].with_(prefix=prefix, prefix_min=min(prefix, 65), vocab=2048)
    st = VerifyStep(w, batch=batch, layers=layers, cache_bits=8)
    for t in st.tk + st.tv:  # the accepted rows need a larger scale than the prefix's last block has
        t.mul_(64)
    return st


@pytest.mark.parametrize("name,prefix,batch", [("llama8b", 333, 1), ("llama8b", 320, 1), ("concurrency", 200, 3),
                                               ("long128k", 510, 2)])
def test_run_after_run_is_the_same(name, prefix, batch):
    st = step(name, prefix, batch, 2)
    st.run()
    first = result(st)
    for _ in range(2):
        st.run()
        assert all(torch.equal(a, b) for a, b in zip(first, result(st)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run()
    for _ in range(2):
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, result(st)))


def test_variants_do_not_depend_on_those_before():
    want = []
    for k in range(3):
        st = step("llama8b", 333, 1, 1)
        st.add_variants(2)
        st.use_variant(k)
        st.run()
        want.append(result(st))
    for k in (2, 0, 1, 0, 2):  # all in one step
        st.use_variant(k)
        st.run()
        assert all(torch.equal(a, b) for a, b in zip(want[k], result(st)))


def test_construction_holds_one_layer_in_16_bits_at_a_time():
    """Peak memory of building the step: the codes and about one layer's bf16 cache beside what stays."""
    w = synth.WORKLOADS["llama8b"].with_(prefix=8192, vocab=2048)
    layers = 8
    VerifyStep(w, batch=1, layers=1, cache_bits=8)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    st = VerifyStep(w, batch=1, layers=layers, cache_bits=8)
    torch.cuda.synchronize()
    layer = 2 * w.n_kv_heads * w.max_seq * w.head_dim * 2  # one layer's K and V in bf16
    over = torch.cuda.max_memory_allocated() - torch.cuda.memory_allocated()
    assert st.L == layers and over <= 3 * layer  # (this layer's, the one before's, copies on their way)
