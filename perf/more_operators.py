"""The operators around the paged KV cache, as measured cases.

A paged cache is a pool of pages a layer, [n_pages][Hkv][T][D] for K and V each (T tokens a page),
and a table [B][max_pages] that names each request's pages in order.  Five operators, each with a
plain form in elementary torch operations (32 bits, rounded once) and the call of the library:

  write    K/V rows of prompts or of single new tokens into their pages
  commit   the accepted path's K/V rows into the pages of every layer
  attn     attention of a request's new tokens (one, a chain, a whole draft tree) over its pages and
           the new tokens' own K/V; scores may be capped by a tanh, biased by the distance, and cut
           off behind a window
  weights  the attention weight that each cached token got from the accepted rows, added up
  evict    every head's cache cut down to its first, its last and its heaviest tokens

Shapes: the verify step's workloads (llama8b: 32 query / 8 KV heads x 128, 61 tree rows, 8K prefix;
long128k: 128K tokens; concurrency: 32 ragged requests of 1K to 16K tokens; vicuna7b: 32 / 32 heads;
the tiny workload's 4 heads of 64).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one request over a short cache, distance bias (latency)
        dict(name="attn_token1k", op="attn", batch=1, rows=1, hq=32, hkv=8, dim=128, page=16, low=1000, high=1000,
             ragged=False, cap=0.0, window=0, slopes=True, dtype="bf16"),
        # one new token over 128K tokens: the cache's bytes
        dict(name="attn_token128k", op="attn", batch=1, rows=1, hq=32, hkv=8, dim=128, page=64, low=131072, high=131072,
             ragged=False, cap=0.0, window=0, slopes=False, dtype="bf16"),
        # the next tokens of 32 requests of 1K to 16K tokens, capped scores
        dict(name="attn_ragged32", op="attn", batch=32, rows=1, hq=32, hkv=8, dim=128, page=64, low=1024, high=16384,
             ragged=False, cap=30.0, window=0, slopes=False, dtype="bf16"),
        # the llama8b verify pass: 61 tree nodes over 8K tokens
        dict(name="attn_tree61", op="attn", batch=1, rows=61, hq=32, hkv=8, dim=128, page=64, low=8192, high=8192,
             ragged=False, cap=0.0, window=0, slopes=False, dtype="bf16"),
        # one layer's prompt into its pages: bandwidth
        dict(name="write_prompt8k", op="write", batch=1, hkv=8, dim=128, page=64, cap_rows=8256, rows=8192,
             ragged=False, dtype="bf16"),
        # the new tokens of 64 requests (latency)
        dict(name="write_tokens64", op="write", batch=64, hkv=8, dim=128, page=16, cap_rows=500, rows=1, ragged=True,
             dtype="bf16"),
        # the accepted path of one request, every layer (latency)
        dict(name="commit_llama8b", op="commit", layers=32, batch=1, hkv=8, dim=128, page=64, cap_rows=2112, rows=61,
             depth=7, dtype="bf16"),
        # 32 requests at once
        dict(name="commit_batch32", op="commit", layers=32, batch=32, hkv=8, dim=128, page=32, cap_rows=576, rows=61,
             depth=6, dtype="bf16"),
        # the weights of one new token over 8K
        dict(name="weights_token8k", op="weights", batch=1, rows=1, depth=0, hq=32, hkv=8, dim=128, page=64, low=8192,
             high=8192, cap=0.0, window=0, slopes=False, dtype="bf16"),
        # the weights of an accepted path of up to 8 of 61 tree rows over 128K tokens
        dict(name="weights_path128k", op="weights", batch=1, rows=61, depth=7, hq=32, hkv=8, dim=128, page=64,
             low=131072, high=131072, cap=0.0, window=0, slopes=False, dtype="bf16"),
        # all layers of one request from 8K tokens to 2K
        dict(name="evict_llama8b", op="evict", layers=32, batch=1, hkv=8, dim=128, page=64, low=8192, high=8192,
             limit=4096, budget=2048, sink=4, recent=256, dtype="bf16"),
        # 16 ragged requests, some of which are short enough as they are
        dict(name="evict_ragged16", op="evict", layers=8, batch=16, hkv=8, dim=128, page=16, low=500, high=6000,
             limit=2000, budget=1000, sink=4, recent=100, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["write", "commit", "attn", "attn", "attn", "weights", "evict"])
    hq, hkv, dim = rng.choice([(32, 8, 128), (32, 32, 128), (4, 4, 64), (8, 2, 64), (28, 4, 128), (16, 1, 128)])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "write":
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, 32000 // batch * 8 // max(8, hkv))
        return dict(op=op, batch=batch, hkv=hkv, dim=dim, page=page, cap_rows=rows + rng.randint(64, 1500), rows=rows,
                    ragged=rng.random() < 0.7, dtype=dtype)
    if op == "commit":
        batch, depth = _log(rng, 1, 24), rng.randint(1, 11)
        return dict(op=op, layers=rng.randint(1, 32), batch=batch, hkv=min(hkv, 8), dim=dim, page=page,
                    cap_rows=rng.randint(100, 600), rows=rng.randint(depth + 1, 128), depth=depth, dtype=dtype)
    if op == "evict":
        batch, layers = _log(rng, 1, 16), rng.randint(1, 16)
        high = _log(rng, 64, min(60000, 120000 // (batch * layers)) * 8 // max(8, hkv))
        limit = rng.randint(high // 3, high - 1)
        budget = rng.randint(1, max(1, min(limit, 12000)))
        sink = rng.randint(0, min(4, budget))
        return dict(op=op, layers=layers, batch=batch, hkv=hkv, dim=dim, page=page, low=rng.randint(high // 2, high),
                    high=high, limit=limit, budget=budget, sink=sink, recent=rng.randint(0, (budget - sink) // 2),
                    dtype=dtype)
    batch = _log(rng, 1, 32)
    if op == "weights":
        depth = rng.randint(0, 8)
        rows = depth + 1 if depth == 0 else rng.randint(depth + 1, 100)
        work = depth + 1
    else:
        rows = 1 if rng.random() < 0.5 else _log(rng, 1, 128)
        depth, work = 0, rows
    half = 2 if dtype == "f32" else 1
    high = _log(rng, 16, max(16, min(131072, 250000 // half, 1500000 // half // work) // batch * 8 // max(8, hkv)))
    case = dict(op=op, batch=batch, rows=rows, hq=hq, hkv=hkv, dim=dim, page=page, low=rng.randint(high // 2, high),
                high=high, cap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, _log(rng, 8, 2 * high)]),
                slopes=rng.random() < 0.25, dtype=dtype)
    if op == "weights":
        case["depth"] = depth
        case["low"], case["high"] = case["low"] + depth + 1, case["high"] + depth + 1
    else:
        case["ragged"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------- work
def _element(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    op, B, D, e = case["op"], case["batch"], case["dim"], _element(case)
    if op == "write":
        n = B * case["rows"] * (0.75 if case["ragged"] else 1.0) * case["hkv"] * 2
        return {"bytes": n * D * e * 2, "flops": 0}
    if op == "commit":
        n = case["layers"] * B * (1 + case["depth"] / 2) * case["hkv"] * 2
        return {"bytes": n * D * e * 2, "flops": 0}
    mean = (case["low"] + case["high"]) / 2
    if op == "evict":
        span = max(1, case["high"] - case["low"] + 1)
        over = min(1.0, max(0.0, (case["high"] - max(case["limit"], case["low"] - 1)) / span))
        long = (max(case["limit"], case["low"]) + case["high"]) / 2
        heads = case["layers"] * B * case["hkv"] * over
        return {"bytes": heads * (long * 4 + case["budget"] * (4 * D * e + 8)), "flops": 0}
    seen = min(mean, case["window"]) if case["window"] else mean
    if op == "weights":
        R = 1 + case["depth"] / 2
        return {"bytes": B * (case["hkv"] * (min(mean, seen + R) * D * e + 8 * mean) + R * case["hq"] * (D * e + 4)),
                "flops": 2 * B * R * case["hq"] * D * seen}
    R = case["rows"] * (0.75 if case["ragged"] else 1.0)
    kv = 2 * case["hkv"] * B * (seen + R) * D * e
    io = B * R * case["hq"] * (2 * D * e + 4)
    return {"bytes": kv + io, "flops": 4 * B * R * case["hq"] * D * (seen + R / 2)}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rng(seed, k):
    return np.random.RandomState((seed * 7919 + k) % (1 << 31))


def _rows(g, dt, *shape):
    """K- or V-like rows: normal, a few channels larger."""
    x = torch.randn(*shape, device="cuda", generator=g)
    x[..., :: shape[-1] // 4] *= 2.0
    return x.to(dt)


def _lengths(case, seed):
    """Tokens and tree nodes of each request."""
    r = _rng(seed, 13)
    B = case["batch"]
    seq = r.randint(case["low"], case["high"] + 1, B).astype(np.int32)
    ragged = case.get("ragged", False)
    nodes = r.randint(max(1, case["rows"] // 2), case["rows"] + 1, B) if ragged else np.full(B, case.get("rows", 1))
    return seq, nodes.astype(np.int32)


def _tables(case, seed, rows, spare=0):
    """Pages of each request for `rows` tokens and `spare` more rows, scattered over the pool."""
    T, B = case["page"], case["batch"]
    mp, sp = -(-rows // T), -(-spare // T)
    order = _rng(seed, 17).permutation(B * (mp + sp) + 3)[: B * (mp + sp)].astype(np.int32)
    return order[: B * mp].reshape(B, mp), order[B * mp:].reshape(B, sp), B * (mp + sp) + 3


def _trees(case, seed):
    """Random draft trees: parents before children; ancestor masks as 64-bit words."""
    r = _rng(seed, 7)
    B, R = case["batch"], case["rows"]
    mask = np.zeros((B, R, (R + 63) // 64), np.uint64)
    for i in range(R):
        if i:
            back = r.randint(1, min(i, 9) + 1, B)
            mask[:, i] = mask[np.arange(B), i - back]
        mask[:, i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return torch.from_numpy(mask.view(np.int64)).cuda()


def _slopes(case):
    """A slope a head, in a geometric series down to 2^-8."""
    h = case["hq"]
    return torch.exp2(-8.0 * torch.arange(1, h + 1, device="cuda").double() / h).float() if case["slopes"] else None


def _path(case, seed):
    """Accepted path of each request: node rows in increasing order, -1 behind them."""
    r = _rng(seed, 5)
    B, R, dep = case["batch"], case["rows"], case["depth"]
    n_acc = r.randint(0, dep + 1, B)
    path = np.sort(np.stack([np.concatenate([[0], 1 + r.permutation(R - 1)[:dep]]) for _ in range(B)]), 1)
    path[np.arange(dep + 1)[None] > n_acc[:, None]] = -1
    return n_acc.astype(np.int32), path.astype(np.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, B, D, H, T, dt = case["op"], case["batch"], case["dim"], case["hkv"], case["page"], DTYPES[case["dtype"]]
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    st = dict(case=case, status=torch.zeros(1, device="cuda", dtype=torch.int32))
    if op == "write":
        table, _, n = _tables(case, seed, case["cap_rows"])
        r, N = _rng(seed, 3), case["rows"]
        count = r.randint((N + 1) // 2, N + 1, B) if case["ragged"] else np.full(B, N)
        start = r.randint(0, case["cap_rows"] - count + 1) if case["ragged"] else np.zeros(B)
        st["start"], st["count"], st["table"] = i32(start), i32(count), i32(table)
        st["k"], st["v"] = (_rows(g, dt, B, H, N, D) for _ in range(2))
        st["kp"], st["vp"] = (_rows(g, dt, n, H, T, D) for _ in range(2))
    elif op == "commit":
        table, _, n = _tables(case, seed, case["cap_rows"])
        L, R, dep = case["layers"], case["rows"], case["depth"]
        n_acc, path = _path(case, seed)
        st["table"], st["n_acc"], st["path"] = i32(table), i32(n_acc), i32(path)
        st["seq0"] = i32(_rng(seed, 3).randint(0, case["cap_rows"] - dep, B))
        st["seq"] = st["seq0"].clone()
        st["pos"] = torch.zeros(B, dep + 1, device="cuda", dtype=torch.int32)
        st["tk"], st["tv"] = (_rows(g, dt, L, B, H, R, D) for _ in range(2))
        st["kp"], st["vp"] = (_rows(g, dt, L, n, H, T, D) for _ in range(2))
    elif op == "evict":
        seq, _ = _lengths(case, seed)
        L, N = case["layers"], case["budget"]
        table, spare, n = _tables(case, seed, case["high"] + 1, N)
        # one buffer for what an eviction changes besides the pages, so that one copy repeats the step
        flat = np.concatenate([table.ravel(), spare.ravel(), seq])
        st["index0"] = i32(flat)
        st["index"] = st["index0"].clone()
        t, s, q = st["index"].split([table.size, spare.size, B])
        st["table"], st["spare"], st["seq"] = t.view(table.shape), s.view(spare.shape), q
        st["kp"], st["vp"] = (_rows(g, dt, L, n, H, T, D) for _ in range(2))
        # heavy-tailed, as accumulated weights are
        st["w"] = torch.exp(2.5 * torch.randn(L, n, H, T, device="cuda", generator=g) - 4)
        st["kept"] = torch.zeros(L, B, H, N, device="cuda", dtype=torch.int32)
    else:
        seq, nodes = _lengths(case, seed)
        R, hq = case["rows"], case["hq"]
        table, _, n = _tables(case, seed, case["high"])
        st["seq"], st["table"], st["slopes"] = i32(seq), i32(table), _slopes(case)
        st["kp"] = _rows(g, dt, n, H, T, D)
        st["q"] = _rows(g, dt, B, R, hq, D)
        if op == "attn":
            st["vp"] = _rows(g, dt, n, H, T, D)
            st["tk"], st["tv"] = (_rows(g, dt, B, H, R, D) for _ in range(2))
            st["nodes"], st["mask"] = i32(nodes) if case["ragged"] else None, _trees(case, seed)
            st["out"] = torch.zeros(B, R, hq, D, device="cuda", dtype=dt)
            st["lse"] = torch.zeros(B, R, hq, device="cuda")
        else:
            n_acc, path = _path(case, seed)
            st["n_acc"], st["path"] = i32(n_acc), i32(path)
            st["w0"] = torch.exp(2.5 * torch.randn(n, H, T, device="cuda", generator=g) - 4)
            st["w"] = torch.zeros(n, H, T, device="cuda")
            # what attention left: the log sums of the accepted rows (those of the others count for nothing)
            z = torch.logsumexp(_path_scores(st)[0], -1).permute(0, 2, 1, 3).reshape(B, -1, hq)
            to = torch.where(st["path"] < 0, R, st["path"]).long()[..., None].expand_as(z)
            st["lse"] = torch.full((B, R + 1, hq), 20.0, device="cuda").scatter(1, to, z)[:, :R].contiguous()
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a user's program of the library keeps: descriptors, layer pointers, workspace."""
    from eagle_speculative_decoding_tree_gb300 import binding as E
    c = st["case"]
    dt = E.EAGLE_F32 if c["dtype"] == "f32" else E.EAGLE_BF16
    n, mp, H, D, T = st["kp"].shape[-4], st["table"].shape[1], c["hkv"], c["dim"], c["page"]
    scale = 1.0 / math.sqrt(D)
    if c["op"] == "write":
        st["desc"] = E.PagedDesc(c["batch"], H, D, T, n, mp, c["rows"], dt)
    elif c["op"] == "commit":
        st["desc"] = E.PagedCommitDesc(c["layers"], c["batch"], H, D, T, n, mp, c["rows"], c["depth"], dt, 0, dt)
        st["layers"] = E.LayerPointers(*[list(st[x].unbind(0)) for x in ("kp", "vp", "tk", "tv")])
        st["ws"] = torch.zeros(E.workspace_size(E.EAGLE_WS_PAGED_COMMIT, st["desc"]), device="cuda", dtype=torch.uint8)
    elif c["op"] == "evict":
        st["desc"] = E.PagedEvictDesc(c["layers"], c["batch"], H, D, T, n, mp, c["limit"], c["budget"], c["sink"],
                                      c["recent"], dt)
        st["layers"] = E.PagedLayerPointers(*[list(st[x].unbind(0)) for x in ("kp", "vp", "w")])
        st["ws"] = torch.zeros(E.workspace_size(E.EAGLE_WS_PAGED_EVICT, st["desc"]), device="cuda", dtype=torch.uint8)
    elif c["op"] == "weights":
        st["desc"] = E.PagedWeightsDesc(c["batch"], c["rows"], c["hq"], H, D, T, n, mp, c["depth"], scale, c["cap"],
                                        c["window"], dt)
    else:
        st["desc"] = E.PagedAttnDesc(c["batch"], c["rows"], c["hq"], H, D, T, n, mp, scale, c["cap"], c["window"], dt,
                                     dt, E.EAGLE_ATTN_PRECISE, E.EAGLE_ENGINE_AUTO)
        st["ws"] = torch.zeros(E.workspace_size(E.EAGLE_WS_PAGED_ATTN, st["desc"]), device="cuda", dtype=torch.uint8)


# ------------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        from eagle_speculative_decoding_tree_gb300 import binding as E
        if op == "write":
            E.eagle_paged_write(st["desc"], st["k"], st["v"], st["table"], st["start"], st["count"], st["kp"],
                                st["vp"], st["status"])
            return st["kp"], st["vp"], st["status"]
        if op == "commit":
            st["seq"].copy_(st["seq0"])  # the same step again
            E.eagle_paged_commit(st["desc"], st["layers"], st["table"], st["n_acc"], st["path"], st["seq"], st["pos"],
                                 st["ws"], status=st["status"])
            return st["kp"], st["vp"], st["seq"], st["pos"], st["status"]
        if op == "weights":
            E.eagle_paged_weights(st["desc"], st["q"], st["lse"], st["kp"], st["table"], st["seq"], st["n_acc"],
                                  st["path"], st["w0"], st["w"], slopes=st["slopes"], status=st["status"])
            return st["w"], st["status"]
        if op == "evict":
            st["index"].copy_(st["index0"])  # the same step again
            E.eagle_paged_evict(st["desc"], st["layers"], st["table"], st["spare"], st["seq"], st["kept"], st["ws"],
                                status=st["status"])
            return st["kp"], st["vp"], st["w"], st["kept"], st["index"], st["status"]
        E.eagle_paged_attn(st["desc"], st["q"], st["kp"], st["vp"], st["table"], st["tk"], st["tv"], st["seq"],
                           st["mask"], st["out"], st["lse"], st["ws"], n_nodes=st["nodes"], slopes=st["slopes"],
                           status=st["status"])
        return st["out"], st["lse"], st["status"]
    return {"write": _write, "commit": _commit, "attn": _attn, "weights": _weights, "evict": _evict}[op](st)


# ------------------------------------------------------------------------------- plain forms
def _whole(pages, table, lead=0):
    """The rows of each request in order, [.., B, Hkv, max_pages * T, ..] fp32, from pages [.., n, Hkv, T, ..]
    with `lead` dimensions before n."""
    x = pages.index_select(lead, table.long().flatten()).float().unflatten(lead, tuple(table.shape))
    return x.transpose(lead + 1, lead + 2).flatten(lead + 2, lead + 3)


def _at(table, rows, T):
    """Page and row in it of cache rows [B, n]; rows past the table end are clamped (and masked by the caller)."""
    page = table.long().gather(1, (rows // T).clamp(max=table.shape[1] - 1))
    return page, rows % T


def _write(st):
    c = st["case"]
    j = torch.arange(c["rows"], device="cuda")
    start, count = st["start"].long()[:, None], st["count"].long()[:, None]
    page, at = _at(st["table"], start + j, c["page"])
    b, i = torch.nonzero(j < count, as_tuple=True)
    for pages, rows in ((st["kp"], st["k"]), (st["vp"], st["v"])):
        pages[page[b, i], :, at[b, i]] = rows[b, :, i]
    return st["kp"], st["vp"], st["status"]


def _commit(st):
    c = st["case"]
    m = torch.arange(c["depth"] + 1, device="cuda")
    seq0, n = st["seq0"].long()[:, None], st["n_acc"].long()[:, None] + 1
    page, at = _at(st["table"], seq0 + m, c["page"])
    b, i = torch.nonzero(m < n, as_tuple=True)
    node = st["path"].long()[b, i]
    for pages, tree in ((st["kp"], st["tk"]), (st["vp"], st["tv"])):
        pages.transpose(0, 1).transpose(1, 3)[page[b, i], at[b, i]] = tree.permute(1, 3, 2, 0, 4)[b, node]
    return st["kp"], st["vp"], (seq0 + n)[:, 0].int(), torch.where(m < n, seq0 + m, -1).int(), st["status"]


def _shape(s, dist, c, slopes, G):
    """Cap, distance bias and window of scores [B, Hkv, n, G, keys]; dist [B, n, keys]."""
    d = dist[:, None, :, None].float()
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    if slopes is not None:
        s = s - slopes.view(1, -1, 1, G, 1) * d
    if c["window"]:
        s = s.masked_fill(d >= c["window"], -math.inf)
    return s


def _attn(st):
    c = st["case"]
    B, R, H, D = c["batch"], c["rows"], c["hkv"], c["dim"]
    G = c["hq"] // H
    q = st["q"].float().view(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    k = torch.cat((_whole(st["kp"], st["table"]), st["tk"].float()), 2)
    s = (q @ k.transpose(-1, -2) * (1.0 / math.sqrt(D))).view(B, H, R, G, -1)
    P = k.shape[2] - R
    bits = ((st["mask"][..., None] >> torch.arange(64, device="cuda")) & 1).flatten(-2)[..., :R].bool()  # [B, R, R]
    r, j = torch.arange(R, device="cuda"), torch.arange(P, device="cuda")
    nodes = st["nodes"].long() if st["nodes"] is not None else torch.full((B,), R, device="cuda")
    live = r < nodes[:, None]
    seq = st["seq"].long()[:, None, None]
    bits = bits & live[:, None]
    depth = bits.sum(-1) - 1
    dist = torch.cat((seq + depth[..., None] - j, depth[..., None] - depth[:, None]), -1)
    s = _shape(s, dist, c, st["slopes"], G)
    seen = torch.cat(((j < seq).expand(B, R, P), bits), -1)
    s = s.masked_fill(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    v = torch.cat((_whole(st["vp"], st["table"]), st["tv"].float()), 2)
    o = (p.flatten(2, 3) @ v).view(B, H, R, G, D) / l
    lay = lambda x: x.permute(0, 2, 1, 3, 4).reshape(B, R, H * G, -1)
    here = live[:, :, None, None]
    out = torch.where(here, lay(o), st["out"].float()).to(st["out"].dtype)
    return out, torch.where(here, lay(top + torch.log(l)), st["lse"][..., None])[..., 0], st["status"]


def _path_scores(st):
    """Scores [B, Hkv, path, G, keys] of the accepted rows (-inf: not attended to), and the rows' nodes."""
    c = st["case"]
    B, H, D = c["batch"], c["hkv"], c["dim"]
    G, M = c["hq"] // H, c["depth"] + 1
    node = st["path"].long().clamp(min=0)
    q = st["q"].float().gather(1, node[..., None, None].expand(-1, -1, H * G, D))
    q = q.view(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    k = _whole(st["kp"], st["table"])
    s = (q @ k.transpose(-1, -2) * (1.0 / math.sqrt(D))).view(B, H, M, G, -1)
    m, j = torch.arange(M, device="cuda"), torch.arange(k.shape[2], device="cuda")
    n = st["n_acc"].long()[:, None] + 1
    dist = ((st["seq"].long()[:, None] - n + m)[..., None] - j)
    s = _shape(s, dist, c, st["slopes"], G)
    seen = (dist >= 0) & (m < n)[..., None]
    return s.masked_fill(~seen[:, None, :, None], -math.inf), node


def _weights(st):
    c = st["case"]
    B, H, T = c["batch"], c["hkv"], c["page"]
    s, node = _path_scores(st)
    G, M = s.shape[3], s.shape[2]
    lse = st["lse"].gather(1, node[..., None].expand(-1, -1, H * G)).view(B, M, H, G).transpose(1, 2)
    got = torch.exp(s - lse[..., None]).sum((2, 3))  # [B, H, keys]
    n = st["n_acc"].long()[:, None] + 1
    j = torch.arange(got.shape[-1], device="cuda")
    seq = st["seq"].long()[:, None]
    old = _whole(st["w0"], st["table"])
    new = torch.where((j < seq - n)[:, None], old, 0.0) + got
    new = torch.where((j < seq)[:, None], new, _whole(st["w"], st["table"]))
    st["w"][st["table"].long()] = new.unflatten(-1, (-1, T)).transpose(1, 2)
    return st["w"], st["status"]


def _evict(st):
    c = st["case"]
    L, B, H, T, N = c["layers"], c["batch"], c["hkv"], c["page"], c["budget"]
    st["index"].copy_(st["index0"])
    table, spare, seq = st["table"].long(), st["spare"].long(), st["seq"].long()
    w = _whole(st["w"], st["table"], 1)  # [L, B, H, P]
    j = torch.arange(w.shape[-1], device="cuda")
    len_ = seq[:, None, None]
    rank = torch.where((j < c["sink"]) | (j >= len_ - c["recent"]), math.inf, w)
    rank = torch.where(j < len_, rank, -math.inf)
    keep = rank.sort(dim=-1, descending=True, stable=True).indices[..., :N].sort(-1).values  # [L, B, H, N]
    over = seq > c["limit"]
    n = torch.arange(N, device="cuda")
    dst, at = _at(st["spare"], n.expand(B, N), T)
    lay = torch.arange(L, device="cuda").view(L, 1, 1, 1)
    head = torch.arange(H, device="cuda").view(1, 1, H, 1)
    dst, at = dst.view(1, B, 1, N), at.view(1, B, 1, N)
    src = table.view(1, B, 1, -1).expand(L, B, H, -1).gather(-1, keep // T)
    move = over.view(1, B, 1, 1)
    for pages in (st["kp"], st["vp"], st["w"]):
        m = move if pages.dim() == 4 else move[..., None]
        pages[lay, dst, head, at] = torch.where(m, pages[lay, src, head, keep % T], pages[lay, dst, head, at])
    kept = torch.where(move, keep.int(), st["kept"])
    bp, o = spare.shape[1], over[:, None]
    first = table[:, :bp].clone()
    new_table = torch.cat((torch.where(o, spare, first), table[:, bp:]), 1)
    new_spare = torch.where(o, first, spare)
    new_seq = torch.where(over, N, seq)
    index = torch.cat((new_table.flatten(), new_spare.flatten(), new_seq)).int()
    return st["kp"], st["vp"], st["w"], kept, index, st["status"]


# ------------------------------------------------------------------------------- 64 bits
def _cached(pages, row, n):
    """The first n rows of the request with page list `row`, [H, n, ...] fp64."""
    x = torch.cat([pages[p] for p in row], 1)
    return x[:, :n].double()


def _prob(s, dist, c, slopes):
    """exact's scores [n, hq, keys] from raw ones; dist [n, keys]."""
    if c["cap"]:
        s = torch.tanh(s / c["cap"]) * c["cap"]
    if slopes is not None:
        s = s - torch.einsum("h,nk->nhk", slopes.double(), dist.double())
    if c["window"]:
        s = torch.where((dist < c["window"])[:, None], s, -math.inf)
    return s


def exact(case, seed):
    op, H, D = case["op"], case["hkv"], case["dim"]
    if op not in ("attn", "weights"):
        return None  # rows moved as they are
    st = prepare(case, seed)
    G = case["hq"] // H
    seq, nodes = _lengths(case, seed)
    table = st["table"].tolist()
    T = case["page"]
    if op == "attn":
        bits = st["mask"].cpu().numpy().view(np.uint64)
        out, lse = st["out"].double(), st["lse"].double()
        for b in range(case["batch"]):
            L, n = int(seq[b]), int(nodes[b])
            see = np.zeros((n, n), bool)
            for i in range(n):
                for a in range(i + 1):
                    see[i, a] = (int(bits[b, i, a // 64]) >> (a % 64)) & 1
            place = torch.from_numpy(L - 1 + see.sum(1)).cuda()  # where a node stands
            pages = table[b][: -(-L // T)]
            k, v = (torch.cat((_cached(st[x + "p"], pages, L), st["t" + x][b, :, :n].double()), 1) for x in "kv")
            s = torch.einsum("nhgd,hkd->nhgk", st["q"][b, :n].double().view(n, H, G, D), k).flatten(1, 2) / math.sqrt(D)
            s = _prob(s, place[:, None] - torch.cat((torch.arange(L, device="cuda"), place)), case, st["slopes"])
            s[..., L:] = torch.where(torch.from_numpy(see).cuda()[:, None], s[..., L:], -math.inf)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[..., None]).view(n, H, G, -1)
            out[b, :n], lse[b, :n] = torch.einsum("nhgk,hkd->nhgd", p, v).flatten(1, 2), z
        return out, lse, None
    w = st["w"].double()
    n_acc, path = _path(case, seed)
    for b in range(case["batch"]):
        L, n = int(seq[b]), int(n_acc[b]) + 1
        pages = table[b][: -(-L // T)]
        node = torch.from_numpy(path[b, :n]).long().cuda()
        s = torch.einsum("nhgd,hkd->nhgk", st["q"][b, node].double().view(n, H, G, D), _cached(st["kp"], pages, L))
        place = torch.arange(L - n, L, device="cuda")
        dist = place[:, None] - torch.arange(L, device="cuda")
        s = _prob(s.flatten(1, 2) / math.sqrt(D), dist, case, st["slopes"])
        s = torch.where((dist >= 0)[:, None], s, -math.inf)
        p = torch.exp(s - st["lse"][b, node].double()[..., None]).view(n, H, G, L).sum((0, 2))
        p[:, : L - n] += torch.cat([st["w0"][x] for x in pages], 1)[:, : L - n].double()
        for i, x in enumerate(pages):
            w[x, :, : min(T, L - i * T)] = p[:, i * T: min((i + 1) * T, L)]
    return w, None
