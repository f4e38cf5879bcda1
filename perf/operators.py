"""The operators around the 8-bit KV cache, as measured cases.

Five operators of the verify step's data path, each with a plain form in elementary torch
operations (fp32, fp64 where 32 bits lose what matters) and the call of the library:

  rope    q / k norms per head, rotation at each tree node's position, and the layout that
          tree attention reads, from the QKV projection's rows
  write   K/V rows quantised into an 8-bit cache (e4m3, one power-of-two scale for each
          block of 64 tokens and head)
  read    rows of that cache read back
  commit  the accepted path's K/V rows appended to the 8-bit caches of every layer
  attn    tree attention over the 8-bit cache and the tree's own bf16 K/V

Shapes: the verify step's workloads (llama8b: 32 query / 8 KV heads x 128, 61 tree rows, 8K
prefix; long128k: a chain of 8 over 128K tokens; concurrency: 32 ragged requests of 1K to 16K
tokens; vicuna7b: 32 / 32 heads; the tiny workload's 4 heads of 64).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64        # tokens of a cache block that share a scale
E4M3_MAX = 448.0  # largest finite e4m3 value
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the rows of one llama8b verify pass on their way into tree attention (latency)
        dict(name="rope_tree61", op="rope", batch=1, rows=61, hq=32, hkv=8, dim=128, rot=128, pad=0,
             interleaved=False, norm=True, dtype="bf16", far=8192),
        # the projection of a whole 8K prompt: bandwidth
        dict(name="rope_prompt8k", op="rope", batch=1, rows=8192, hq=32, hkv=8, dim=128, rot=128, pad=0,
             interleaved=False, norm=True, dtype="bf16", far=8192),
        # one layer's prompt K/V into the 8-bit cache
        dict(name="write_prompt8k", op="write", batch=1, hkv=8, dim=128, cap=8256, rows=8192, ragged=False,
             dtype="bf16"),
        # chunks of ragged requests that begin and end inside blocks
        dict(name="write_ragged32", op="write", batch=32, hkv=8, dim=128, cap=4160, rows=1021, ragged=True,
             dtype="bf16"),
        # a whole prefix read back, and ragged spans of it in fp32
        dict(name="read_prefix8k", op="read", batch=1, hkv=8, dim=128, cap=8256, rows=8192, ragged=False,
             dtype="bf16"),
        dict(name="read_ragged_f32", op="read", batch=7, hkv=8, dim=128, cap=4160, rows=999, ragged=True,
             dtype="f32"),
        # the accepted path of one request, every layer (latency)
        dict(name="commit_llama8b", op="commit", layers=32, batch=1, hkv=8, dim=128, cap=2112, rows=61, depth=7,
             dtype="bf16"),
        # 32 requests at once
        dict(name="commit_batch32", op="commit", layers=32, batch=32, hkv=8, dim=128, cap=576, rows=61, depth=6,
             dtype="bf16"),
        # a single token of one request over a short prefix (latency)
        dict(name="attn_single", op="attn", batch=1, rows=1, hq=32, hkv=8, dim=128, low=777, high=777, ragged=False,
             out="bf16"),
        # the llama8b verify pass: 61 tree nodes over 8K tokens
        dict(name="attn_llama8b", op="attn", batch=1, rows=61, hq=32, hkv=8, dim=128, low=8192, high=8192,
             ragged=False, out="bf16"),
        # a chain of 8 over 128K tokens: the cache's bytes; outputs in fp32
        dict(name="attn_long128k", op="attn", batch=1, rows=8, hq=32, hkv=8, dim=128, low=131072, high=131072,
             ragged=False, out="f32"),
        # 32 requests of 1K to 16K tokens, trees of different sizes
        dict(name="attn_ragged32", op="attn", batch=32, rows=61, hq=32, hkv=8, dim=128, low=1024, high=16384,
             ragged=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "commit", "attn", "attn"])
    hq, hkv, dim = rng.choice([(32, 8, 128), (32, 32, 128), (4, 4, 64), (8, 2, 64), (28, 4, 128), (16, 1, 128)])
    if op == "rope":
        batch = rng.randint(1, 8)
        rows = _log(rng, 1, max(2, 12000 // batch) * 8 // max(8, hkv))
        return dict(op=op, batch=batch, rows=rows, hq=hq, hkv=hkv, dim=dim, rot=rng.choice([dim, dim // 2]),
                    pad=rng.choice([0, 0, 64]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), far=_log(rng, 64, 131072))
    if op in ("write", "read"):
        batch = _log(rng, 1, 32)
        rows = _log(rng, 1, 32000 // batch * 8 // max(8, hkv))
        return dict(op=op, batch=batch, hkv=hkv, dim=dim, cap=rows + rng.randint(64, 1500), rows=rows,
                    ragged=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "commit":
        batch, depth = _log(rng, 1, 24), rng.randint(1, 11)
        return dict(op=op, layers=rng.randint(1, 32), batch=batch, hkv=min(hkv, 8), dim=dim,
                    cap=rng.randint(100, 600), rows=rng.randint(depth + 1, 128), depth=depth,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    batch = _log(rng, 1, 16)
    rows = _log(rng, 1, 128)
    high = _log(rng, 1, 130000 // batch * 8 // max(8, hkv))
    return dict(op=op, batch=batch, rows=rows, hq=hq, hkv=hkv, dim=dim, low=rng.randint(0, high), high=high,
                ragged=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------------------- work
def _spans(case, seed):
    """write / read: first cache row and row count of each request; attn: prefix lengths."""
    r = np.random.RandomState((seed * 7919 + 13) % (1 << 31))
    B = case["batch"]
    if case["op"] == "attn":
        seq = r.randint(case["low"], case["high"] + 1, B)
        nodes = r.randint(max(1, case["rows"] // 2), case["rows"] + 1, B) if case["ragged"] else np.full(B, case["rows"])
        return seq.astype(np.int32), nodes.astype(np.int32)
    if not case["ragged"]:
        return np.zeros(B, np.int32), np.full(B, case["rows"], np.int32)
    count = r.randint((case["rows"] + 1) // 2, case["rows"] + 1, B)
    return r.randint(0, case["cap"] - count + 1).astype(np.int32), count.astype(np.int32)


def work(case):
    op, B, D = case["op"], case["batch"], case["dim"]
    if op == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        width = (case["hq"] + 2 * case["hkv"]) * D
        return {"bytes": B * case["rows"] * (2 * width * e + 4),
                "flops": B * case["rows"] * (case["hq"] + case["hkv"]) * D * 7}
    if op in ("write", "read"):
        e = 2 if case["dtype"] == "bf16" else 4
        n = B * case["rows"] * (0.75 if case["ragged"] else 1.0) * case["hkv"] * 2
        return {"bytes": n * (D * (e + 1) + 4 / BLOCK), "flops": n * D * 2}
    if op == "commit":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["layers"] * B * (1 + (case["depth"] + 1) / 2) * case["hkv"] * 2
        return {"bytes": n * D * (e + 1), "flops": n * D * 2}
    seq, R = B * (case["low"] + case["high"]) / 2, case["rows"] * (0.75 if case["ragged"] else 1.0)
    kv = 2 * case["hkv"] * (seq * (D + 4 / BLOCK) + B * R * D * 2)
    io = B * R * case["hq"] * (D * (2 + (2 if case["out"] == "bf16" else 4)) + 4)
    return {"bytes": kv + io, "flops": 4 * R * case["hq"] * D * (seq + B * R / 2)}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, *shape):
    """K- or V-like rows: normal, a few channels larger, block-to-block changes of size."""
    x = torch.randn(*shape, device="cuda", generator=g)
    chan = torch.ones(shape[-1], device="cuda")
    chan[:: shape[-1] // 4] = 3.0
    size = torch.exp2(torch.randint(-2, 2, shape[:-2] + (1, 1), device="cuda", generator=g).float() * 0.5)
    return x * chan * size


def _block_scale(amax):
    """Smallest power of two s with amax <= 448 s (0 for a block of zeros)."""
    m, e = torch.frexp(amax.float())  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    s = torch.ldexp(torch.ones_like(m), torch.clamp(e - 9 + (m > 0.875).int(), min=-126))
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _filled(x):
    """A whole cache quantised from x [..., P, D], P a multiple of 64: codes and scales."""
    xb = x.unflatten(-2, (-1, BLOCK))
    s = _block_scale(xb.abs().amax((-1, -2)))
    codes = (xb / torch.where(s > 0, s, torch.ones_like(s))[..., None, None]).to(torch.float8_e4m3fn)
    return codes.flatten(-3, -2), s


def _trees(case, seed):
    """Random draft trees: parents before children; ancestor masks as 64-bit words."""
    r = np.random.RandomState((seed * 104729 + 7) % (1 << 31))
    B, R = case["batch"], case["rows"]
    W = (R + 63) // 64
    mask = np.zeros((B, R, W), np.uint64)
    for i in range(R):
        if i:
            back = r.randint(1, min(i, 9) + 1, B)
            mask[:, i] = mask[np.arange(B), i - back]
        mask[:, i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return torch.from_numpy(mask.view(np.int64)).cuda()


def prepare(case, seed):
    g = _gen(seed)
    op, B, D = case["op"], case["batch"], case["dim"]
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    st = dict(case=case)
    if op == "rope":
        dt, R, hq, hkv = DTYPES[case["dtype"]], case["rows"], case["hq"], case["hkv"]
        width = (hq + 2 * hkv) * D
        st["qkv"] = torch.randn(B, R, width + case["pad"], device="cuda", generator=g).to(dt)
        st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt) if case["norm"] else None
                              for _ in range(2))
        st["inv_freq"] = (500000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda").double() / case["rot"])).float()
        base = torch.randint(0, case["far"], (B, 1), device="cuda", generator=g)
        st["pos"] = (base + torch.randint(0, max(8, R), (B, R), device="cuda", generator=g)).int()
        st["q"] = torch.zeros(B, R, hq, D, device="cuda", dtype=dt)
        st["k"], st["v"] = (torch.zeros(B, hkv, R, D, device="cuda", dtype=dt) for _ in range(2))
    elif op in ("write", "read"):
        dt, P, N, H = DTYPES[case["dtype"]], case["cap"], case["rows"], case["hkv"]
        start, count = _spans(case, seed)
        st["start"], st["count"] = i32(start), i32(count)
        nb = -(-P // BLOCK)
        for n in ("k", "v"):
            codes, s = _filled(_rows(g, B, H, nb * BLOCK, D))
            st[n + "8"], st[n + "s"] = codes[:, :, :P].contiguous(), s
            st[n] = _rows(g, B, H, N, D).to(dt) if op == "write" else torch.zeros(B, H, N, D, device="cuda", dtype=dt)
        st["status"] = torch.zeros(1, device="cuda", dtype=torch.int32)
    elif op == "commit":
        dt, P, R, H, L, dep = DTYPES[case["dtype"]], case["cap"], case["rows"], case["hkv"], case["layers"], case["depth"]
        nb = -(-P // BLOCK)
        for n in ("k", "v"):
            codes, s = _filled(_rows(g, L, B, H, nb * BLOCK, D))
            st[n + "8"], st[n + "s"] = codes[..., :P, :].contiguous(), s
            st["t" + n] = _rows(g, L, B, H, R, D).to(dt)
        r = np.random.RandomState((seed * 31 + 5) % (1 << 31))
        n_acc = r.randint(0, dep + 1, B)
        path = np.sort(np.stack([np.concatenate([[0], 1 + r.permutation(R - 1)[:dep]]) for _ in range(B)]), 1)
        path[np.arange(dep + 1)[None] > n_acc[:, None]] = -1
        st["n_acc"], st["path"] = i32(n_acc), i32(path)
        st["seq0"] = i32(r.randint(0, P - dep, B))
        st["seq"] = st["seq0"].clone()
        st["pos"] = torch.zeros(B, dep + 1, device="cuda", dtype=torch.int32)
        st["status"] = torch.zeros(1, device="cuda", dtype=torch.int32)
    else:
        R, hq, hkv = case["rows"], case["hq"], case["hkv"]
        seq, nodes = _spans(case, seed)
        P = (case["high"] + 16 + BLOCK - 1) // BLOCK * BLOCK
        st["seq"], st["nodes"] = i32(seq), i32(nodes) if case["ragged"] else None
        for n in ("k", "v"):
            st[n + "8"], st[n + "s"] = _filled(_rows(g, B, hkv, P, D))
            st["t" + n] = _rows(g, B, hkv, R, D).bfloat16()
        st["qq"] = torch.randn(B, R, hq, D, device="cuda", generator=g).bfloat16()
        st["mask"] = _trees(case, seed)
        st["out"] = torch.zeros(B, R, hq, D, device="cuda", dtype=DTYPES[case["out"]])
        st["lse"] = torch.zeros(B, R, hq, device="cuda")
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a user's program of the library keeps: descriptors, layer pointers, workspace."""
    from eagle_speculative_decoding_tree_gb300 import binding as E
    c = st["case"]
    dt = E.EAGLE_F32 if c.get("dtype", "bf16") == "f32" else E.EAGLE_BF16
    if c["op"] == "rope":
        st["desc"] = E.QkNormRopeDesc(c["batch"], c["rows"], c["hq"], c["hkv"], c["dim"], c["rot"],
                                      (c["hq"] + 2 * c["hkv"]) * c["dim"] + c["pad"], int(c["interleaved"]), 1e-6, dt)
    elif c["op"] in ("write", "read"):
        st["desc"] = E.KvqDesc(c["batch"], c["hkv"], c["dim"], c["cap"], c["rows"], dt)
    elif c["op"] == "commit":
        st["desc"] = E.CommitDesc(c["layers"], c["batch"], c["hkv"], c["dim"], c["rows"], c["cap"], c["depth"], dt, 0,
                                  dt)
        st["layers"] = E.KvqLayerPointers(*[list(st[n].unbind(0)) for n in ("k8", "ks", "v8", "vs", "tk", "tv")])
    else:
        f32 = c["out"] == "f32"
        st["desc"] = E.AttnDesc(c["batch"], c["rows"], c["hq"], c["hkv"], c["dim"], st["k8"].shape[2],
                                1.0 / math.sqrt(c["dim"]), E.EAGLE_BF16, 0, E.EAGLE_F32 if f32 else E.EAGLE_BF16,
                                E.EAGLE_ATTN_PRECISE if f32 else E.EAGLE_ATTN_FAST)
        st["ws"] = torch.zeros(E.workspace_size(E.EAGLE_WS_TREE_ATTN_KVQ, st["desc"]), device="cuda", dtype=torch.uint8)


# ------------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        from eagle_speculative_decoding_tree_gb300 import binding as E
        if op == "rope":
            E.eagle_qk_norm_rope(st["desc"], st["qkv"], st["wq"], st["wk"], st["inv_freq"], st["pos"], st["q"],
                                 st["k"], st["v"])
            return st["q"], st["k"], st["v"]
        if op == "write":
            E.eagle_kvq_write(st["desc"], st["k"], st["v"], st["start"], st["count"], st["k8"], st["ks"], st["v8"],
                              st["vs"], st["status"])
            return st["k8"], st["ks"], st["v8"], st["vs"], st["status"]
        if op == "read":
            E.eagle_kvq_read(st["desc"], st["k8"], st["ks"], st["v8"], st["vs"], st["start"], st["count"], st["k"],
                             st["v"], st["status"])
            return st["k"], st["v"], st["status"]
        if op == "commit":
            st["seq"].copy_(st["seq0"])  # the same step again
            E.eagle_kvq_commit(st["desc"], st["layers"], st["n_acc"], st["path"], st["seq"], st["pos"],
                               status=st["status"])
            return st["k8"], st["ks"], st["v8"], st["vs"], st["seq"], st["pos"], st["status"]
        E.eagle_tree_attn_kvq(st["desc"], st["qq"], st["k8"], st["ks"], st["v8"], st["vs"], st["tk"], st["tv"],
                              st["seq"], st["mask"], st["out"], st["lse"], st["ws"], n_nodes=st["nodes"])
        return st["out"], st["lse"]
    return {"rope": _rope, "write": _write, "read": _read, "commit": _commit, "attn": _attn}[op](st)


# ------------------------------------------------------------------------------- plain forms
def _rope(st):
    c = st["case"]
    hq, hkv, D, rot = c["hq"], c["hkv"], c["dim"], c["rot"]
    dt = DTYPES[c["dtype"]]
    x = st["qkv"][..., : (hq + 2 * hkv) * D].float().unflatten(-1, (-1, D))
    q, k, v = x[:, :, :hq], x[:, :, hq: hq + hkv], x[:, :, hq + hkv:]
    ang = st["pos"].double()[..., None, None] * st["inv_freq"].double()
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()

    def turn(y, w):
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        r = y[..., :rot]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., : rot // 2], r[..., rot // 2:])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((r, y[..., rot:]), -1).to(dt)

    return turn(q, st["wq"]), turn(k, st["wk"]).transpose(1, 2).contiguous(), v.to(dt).transpose(1, 2).contiguous()


def _append(codes, scales, rows, first, count):
    """rows[..., :count, :] quantised into cache rows first .. first + count - 1 (first and
    count broadcast over the leading dims), in place.  A block that begins before `first`
    keeps its rows: its scale only grows, and its codes are then rounded to the new one."""
    P, D = codes.shape[-2:]
    nb = scales.shape[-1]
    N = rows.shape[-2]
    W = (N + BLOCK - 1 + BLOCK - 1) // BLOCK  # blocks a span of N rows can touch
    b0 = first // BLOCK
    pos = b0[..., None] * BLOCK + torch.arange(W * BLOCK, device=codes.device)  # [..., W * 64]
    src = pos - first[..., None]
    new = (src >= 0) & (src < count[..., None])
    old = src < 0
    at = pos.clamp(max=P - 1)[..., None].expand(*codes.shape[:-2], W * BLOCK, D)
    cur = codes.view(torch.uint8).gather(-2, at)
    blk = (b0[..., None] + torch.arange(W, device=codes.device)).clamp(max=nb - 1).expand(*codes.shape[:-2], W)
    s_old = scales.gather(-1, blk)
    x = rows.float().gather(-2, src.clamp(0, N - 1)[..., None].expand(*codes.shape[:-2], W * BLOCK, D))
    amax = torch.where(new[..., None], x.abs(), 0.0).unflatten(-2, (W, BLOCK)).amax((-1, -2))
    touched = new.unflatten(-1, (W, BLOCK)).any(-1)
    holds = old.unflatten(-1, (W, BLOCK)).any(-1)
    s_new = torch.maximum(_block_scale(amax), torch.where(holds, s_old, 0.0))
    div = torch.where(s_new > 0, s_new, torch.ones_like(s_new))
    ratio = (torch.where(holds, s_old, 0.0) / div).repeat_interleave(BLOCK, -1)[..., None]
    put = (x / div.repeat_interleave(BLOCK, -1)[..., None]).to(torch.float8_e4m3fn)
    keep = (cur.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn)
    moved = (old & touched.repeat_interleave(BLOCK, -1))[..., None]
    res = torch.where(new[..., None], put.view(torch.uint8), torch.where(moved, keep.view(torch.uint8), cur))
    # rows past the cache's end and untouched rows are not written: send them to row pos = 0 of
    # a copy with one spare row
    wr = (new | (old & touched.repeat_interleave(BLOCK, -1))).expand(*codes.shape[:-2], W * BLOCK)
    flat = torch.arange(codes[..., 0, 0].numel(), device=codes.device).view(codes.shape[:-2])[..., None] * P + at[..., 0]
    codes.view(torch.uint8).view(-1, D)[flat[wr]] = res[wr]
    tb = touched.expand(*scales.shape[:-1], W)
    fb = torch.arange(scales[..., 0].numel(), device=codes.device).view(scales.shape[:-1])[..., None] * nb + blk
    scales.view(-1)[fb[tb]] = s_new[tb]


def _write(st):
    first, count = st["start"].long()[:, None], st["count"].long()[:, None]
    _append(st["k8"], st["ks"], st["k"], first, count)
    _append(st["v8"], st["vs"], st["v"], first, count)
    return st["k8"], st["ks"], st["v8"], st["vs"], st["status"]


def _read(st):
    N, P, D = st["case"]["rows"], st["case"]["cap"], st["case"]["dim"]
    j = torch.arange(N, device="cuda")
    at = (st["start"].long()[:, None] + j).clamp(max=P - 1)[:, None]  # [B, 1, N]
    live = (j < st["count"].long()[:, None])[:, None, :, None]
    H = st["case"]["hkv"]

    def back(codes, scales, out):
        x = codes.view(torch.uint8).gather(2, at[..., None].expand(-1, H, N, D)).view(torch.float8_e4m3fn).float()
        x = x * scales.gather(2, (at // BLOCK).expand(-1, H, N))[..., None]
        return torch.where(live, x, out.float()).to(out.dtype)

    return back(st["k8"], st["ks"], st["k"]), back(st["v8"], st["vs"], st["v"]), st["status"]


def _commit(st):
    L, R, D, dep = st["case"]["layers"], st["case"]["rows"], st["case"]["dim"], st["case"]["depth"]
    seq0, n = st["seq0"].long(), st["n_acc"].long() + 1
    node = st["path"].long().clamp(min=0)[None, :, None, :, None]
    for codes, scales, tree in ((st["k8"], st["ks"], st["tk"]), (st["v8"], st["vs"], st["tv"])):
        rows = tree.gather(3, node.expand(L, -1, tree.shape[2], -1, D))
        _append(codes, scales, rows, seq0[None, :, None], n[None, :, None])
    m = torch.arange(dep + 1, device="cuda")
    pos = torch.where(m < n[:, None], seq0[:, None] + m, -1).int()
    return st["k8"], st["ks"], st["v8"], st["vs"], (seq0 + n).int(), pos, st["status"]


def _attn(st):
    c = st["case"]
    hkv, D, R, B = c["hkv"], c["dim"], c["rows"], c["batch"]
    G, P = c["hq"] // hkv, st["k8"].shape[2]
    q = st["qq"].float().view(B, R, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, R * G, D)

    def whole(codes, scales, tree):
        x = codes.float().unflatten(2, (-1, BLOCK)) * scales[..., None, None]
        return torch.cat((x.flatten(2, 3), tree.float()), 2)

    s = q @ whole(st["k8"], st["ks"], st["tk"]).transpose(-1, -2) * (1.0 / math.sqrt(D))
    j = torch.arange(64, device="cuda")
    tree = ((st["mask"][..., None] >> j) & 1).flatten(-2)[..., :R].bool()  # [B, R, R]
    nodes = st["nodes"].long() if st["nodes"] is not None else torch.full((B,), R, device="cuda")
    r = torch.arange(R, device="cuda")
    live = r < nodes[:, None]
    seen = torch.arange(P, device="cuda") < st["seq"][:, None].long()
    seen = torch.cat((seen[:, None].expand(B, R, P), tree & live[:, None]), -1).repeat_interleave(G, 1)[:, None]
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    o = p @ whole(st["v8"], st["vs"], st["tv"]) / l
    lay = lambda x: x.view(B, hkv, R, G, -1).permute(0, 2, 1, 3, 4).reshape(B, R, hkv * G, -1)
    here = live[:, :, None, None]
    out = torch.where(here, lay(o), st["out"].float()).to(st["out"].dtype)
    return out, torch.where(here, lay(top + torch.log(l)), st["lse"][..., None])[..., 0]


# ------------------------------------------------------------------------------- 64 bits
def _round8(x):
    """x (fp64, |x| <= 448) to the nearest e4m3 value, ties to the even one."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    e = e + (x.abs() >= torch.exp2(e + 1)).double() - (x.abs() < torch.exp2(e)).double() * (e > -6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_append(codes, scales, rows, first, count):
    """One (request, head): codes [P, D] and scales [nb] in fp64, rows [n, D] at `first`."""
    done = 0
    while done < count:
        b = (first + done) // BLOCK
        lo, hi = b * BLOCK, min((b + 1) * BLOCK, first + count)
        at = first + done
        x = rows[..., done: done + hi - at, :]
        amax = x.abs().amax((-1, -2))
        need = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
        need = torch.where(amax > 448.0 * need, need * 2, torch.where(amax <= 224.0 * need, need / 2, need))
        old = scales[..., b].clone() if at > lo else torch.zeros_like(need)
        s = torch.maximum(torch.where(amax > 0, need, 0.0), old)
        d = torch.where(s > 0, s, 1.0)
        if at > lo:
            codes[..., lo:at, :] = _round8(codes[..., lo:at, :] * (old / d)[..., None, None])
        codes[..., at:hi, :] = _round8(x / d[..., None, None])
        scales[..., b] = s
        done += hi - at


def exact(case, seed):
    st = prepare(case, seed)
    op, B, D = case["op"], case["batch"], case["dim"]
    if op == "rope":
        hq, hkv, rot = case["hq"], case["hkv"], case["rot"]
        x = st["qkv"].double()[..., : (hq + 2 * hkv) * D].reshape(B, case["rows"], hq + 2 * hkv, D)
        ang = (st["pos"].double()[..., None] * st["inv_freq"].double())[:, :, None]
        z = torch.polar(torch.ones_like(ang), ang)

        def one(y, w):
            if w is not None:
                y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + 1e-6) * w.double()
            i = torch.arange(rot // 2, device="cuda")
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
            t = torch.complex(y[..., a], y[..., b]) * z
            y = y.clone()
            y[..., a], y[..., b] = t.real, t.imag
            return y

        return (one(x[:, :, :hq], st["wq"]), one(x[:, :, hq: hq + hkv], st["wk"]).permute(0, 2, 1, 3).contiguous(),
                x[:, :, hq + hkv:].permute(0, 2, 1, 3).contiguous())
    if op == "write":
        start, count = _spans(case, seed)
        res = []
        for n in ("k", "v"):
            codes, s, x = st[n + "8"].double(), st[n + "s"].double(), st[n].double()
            for b in range(B):
                _exact_append(codes[b], s[b], x[b], int(start[b]), int(count[b]))
            res += [codes, s]
        return (*res, None)
    if op == "read":
        start, count = _spans(case, seed)
        res = []
        for n in ("k", "v"):
            out = st[n].double()
            for b in range(B):
                f, c = int(start[b]), int(count[b])
                blk = torch.arange(f, f + c, device="cuda") // BLOCK
                out[b, :, :c] = st[n + "8"][b, :, f: f + c].double() * st[n + "s"][b].double()[:, blk, None]
            res.append(out)
        return (*res, None)
    if op == "commit":
        seq, acc, path = st["seq0"].tolist(), st["n_acc"].tolist(), st["path"].tolist()
        res = []
        for n in ("k", "v"):
            codes, s, tree = st[n + "8"].double(), st[n + "s"].double(), st["t" + n]
            for b in range(B):
                x = tree[:, b][:, :, path[b][: acc[b] + 1]].double()
                _exact_append(codes[:, b], s[:, b], x, seq[b], acc[b] + 1)
            res += [codes, s]
        return (*res, None, None, None)
    seq, nodes = _spans(case, seed)
    R, hq, hkv = case["rows"], case["hq"], case["hkv"]
    G = hq // hkv
    bits = st["mask"].cpu().numpy().view(np.uint64)
    out, lse = st["out"].double(), st["lse"].double()
    for b in range(B):
        L, n = int(seq[b]), int(nodes[b])
        see = np.zeros((n, n), bool)
        for i in range(n):
            for j in range(i + 1):
                see[i, j] = (int(bits[b, i, j // 64]) >> (j % 64)) & 1
        blk = torch.arange(L, device="cuda") // BLOCK
        kv = [torch.cat((st[m + "8"][b, :, :L].double() * st[m + "s"][b].double()[:, blk, None],
                         st["t" + m][b, :, :n].double()), 1) for m in ("k", "v")]
        s = torch.einsum("nhgd,hkd->hngk", st["qq"][b, :n].double().view(n, hkv, G, D), kv[0]) / math.sqrt(D)
        s[..., L:] = torch.where(torch.from_numpy(see).cuda()[None, :, None], s[..., L:], -math.inf)
        z = torch.logsumexp(s, -1)
        o = torch.einsum("hngk,hkd->nhgd", torch.exp(s - z[..., None]), kv[1])
        out[b, :n], lse[b, :n] = o.reshape(n, hq, D), z.permute(1, 0, 2).reshape(n, hq)
    return out, lse
