"""Cases of what a serving step does around its paged cache, and of the rotation that training shares with it.

Queries and keys are turned by their positions (rotate, and its backward pass). Keys and values may be
kept in 8 bits: they are quantised as they are written (write), read back where a program wants them in
16 bits again (read), and attended to as they lie (attend). A step that verifies trees of drafted tokens
first lays out who sees whom (tree), then attends from every node to the cache, its ancestors and itself
(attend, with `nodes`).

A row of d values of one token and head is held as E4M3 codes and one power of two, the smallest that
keeps the row's largest value within 448.

`own = False` computes these with elementary torch operations, `own = True` calls the library.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_LEAST, _MOST = -119, 119  # exponents of the scales


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # queries and keys of one decode step, far positions, frequencies of a context stretched fourfold
        {"name": "rotate decode step", "op": "rotate", "batch": 0, "rows": 64, "pad": 0, "hq": 32, "hk": 8, "d": 128, "turned": 128,
         "interleaved": False, "back": False, "far": 131072, "stretch": 4.0, "dtype": "bf16"},
        # gradients of queries and keys of a long training sequence, half of each head turned, pairs side by side
        {"name": "rotate training gradients", "op": "rotate", "batch": 1, "rows": 32768, "pad": 0, "hq": 16, "hk": 16, "d": 128,
         "turned": 64, "interleaved": True, "back": True, "far": 0, "stretch": 1.0, "dtype": "bf16"},
        # the keys and values of one decode step, kept in 8 bits
        {"name": "write decode step", "op": "write", "rows": 64, "pad": 0, "hkv": 8, "d": 128, "page": 64, "pages": 256,
         "dtype": "bf16"},
        # the keys and values of a step full of prompt chunks, its rows padded
        {"name": "write prompt chunks", "op": "write", "rows": 16301, "pad": 83, "hkv": 8, "d": 128, "page": 32, "pages": 1024,
         "dtype": "fp16"},
        # a short prefix taken out of the cache
        {"name": "read a prefix", "op": "read", "rows": 517, "pad": 3, "hkv": 4, "d": 64, "page": 16, "pages": 256, "dtype": "fp16"},
        # a batch of contexts handed on in 16 bits
        {"name": "read contexts", "op": "read", "rows": 65021, "pad": 0, "hkv": 8, "d": 128, "page": 64, "pages": 1200,
         "dtype": "bf16"},
        # a full decode batch of ragged contexts: the cache read is all there is
        {"name": "attend decode batch", "op": "attend", "bits": 8, "nodes": 0, "seqs": 64, "long": 0, "q": 1, "q_rest": 1, "kv": 8192,
         "spread": 0.5, "hkv": 8, "group": 4, "d": 128, "page": 64, "dtype": "bf16", "causal": True, "pad": 0},
        # a late chunk of a long prompt
        {"name": "attend prompt chunk", "op": "attend", "bits": 8, "nodes": 0, "seqs": 1, "long": 1, "q": 2048, "q_rest": 1,
         "kv": 16384, "spread": 0.0, "hkv": 8, "group": 4, "d": 128, "page": 128, "dtype": "bf16", "causal": True, "pad": 0},
        # one user's drafted tree
        {"name": "tree of one user", "op": "tree", "seqs": 1, "nodes": 32, "q": 26, "least": 26, "chunks": 0, "chunk": 0, "kv": 2001,
         "pad": 6},
        # the trees of a large batch, two prompt chunks among them, rows padded
        {"name": "trees of a batch", "op": "tree", "seqs": 300, "nodes": 64, "q": 64, "least": 17, "chunks": 2, "chunk": 1500,
         "kv": 8192, "pad": 41},
        # one user's tree verified over a 16-bit cache: the latency of a drafted step
        {"name": "attend one tree", "op": "attend", "bits": 16, "nodes": 32, "seqs": 1, "long": 1, "q": 26, "q_rest": 26, "kv": 2001,
         "spread": 0.0, "hkv": 8, "group": 4, "d": 128, "page": 16, "dtype": "bf16", "causal": False, "pad": 6},
        # a batch of trees verified over long contexts in 8 bits
        {"name": "attend trees", "op": "attend", "bits": 8, "nodes": 64, "seqs": 24, "long": 6, "q": 61, "q_rest": 22, "kv": 8192,
         "spread": 0.6, "hkv": 8, "group": 5, "d": 128, "page": 64, "dtype": "fp16", "causal": False, "pad": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "write", "read", "attend", "attend", "attend", "tree", "attend tree", "attend tree"])
    if op == "rotate":
        d, batch = rng.choice([64, 128, 256]), rng.choice([0, 0, 1, 2, 5])
        hq = rng.randint(1, 40)
        most = int(9.0e7 / (max(batch, 1) * hq * d))
        return {"op": op, "batch": batch, "rows": _log(rng, 1, min(16000, most)), "pad": rng.choice([0, 5]) if batch == 0 else 0,
                "hq": hq, "hk": rng.choice([1, 2, hq]), "d": d, "turned": rng.choice([d, d, d // 2, d // 4]),
                "interleaved": rng.choice([False, True]), "back": rng.choice([False, True]),
                "far": _log(rng, 1, 1000000) if batch == 0 else 0, "stretch": rng.choice([1.0, 1.0, 8.0]),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op in ("write", "read"):
        return {"op": op, "rows": _log(rng, 1, 16000), "pad": rng.choice([0, 0, 3, 50]), "hkv": rng.randint(1, 8),
                "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128, 256]), "pages": rng.randint(1001, 1100),
                "dtype": rng.choice(["bf16", "fp16"])}
    if op == "tree":
        nodes = rng.choice([32, 64, 96, 256])
        q = rng.randint(2, nodes)
        return {"op": op, "seqs": _log(rng, 1, 300), "nodes": nodes, "q": q, "least": rng.randint(1, q), "chunks": rng.randint(0, 1),
                "chunk": rng.randint(nodes + 1, 1000), "kv": _log(rng, 1100, 16000), "pad": rng.choice([0, 0, 5, 64])}
    c = {"op": "attend", "bits": 8, "nodes": 0, "hkv": rng.randint(1, 8), "group": rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16]),
         "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128, 256]), "dtype": rng.choice(["bf16", "fp16"]),
         "spread": round(rng.uniform(0.0, 0.9), 2), "pad": rng.choice([0, 0, 1, 7, 33])}
    heads = c["hkv"] * c["group"]
    if op == "attend tree":
        c.update(bits=rng.choice([8, 16]), nodes=rng.choice([32, 64, 128]), seqs=_log(rng, 1, 48), causal=False)
        c.update(q=rng.randint(2, c["nodes"]), long=rng.randint(0, c["seqs"]))
        c["q_rest"] = rng.randint(1, c["q"])
        room = min(1.0e9 / (c["seqs"] * c["hkv"] * c["d"] * 4), 1.2e9 / (c["seqs"] * c["q"] * heads))
        c["kv"] = _log(rng, c["q"], int(max(c["q"] + 1, min(20000, room))))
        return c
    kind = rng.choice(["decode", "decode", "drafted", "mixed", "chunk", "states"])
    if kind in ("decode", "drafted"):
        c.update(seqs=_log(rng, 1, 96), long=0, q=1, q_rest=1 if kind == "decode" else rng.randint(2, 9), causal=True)
        c["q"] = c["q_rest"]
        room = 1.2e9 / (c["seqs"] * c["hkv"] * c["d"] * 4)
        c["kv"] = _log(rng, c["q"], int(max(c["q"] + 1, min(40000, room))))
    elif kind == "mixed":
        c.update(seqs=rng.randint(2, 24), long=1, q=_log(rng, 8, 700), q_rest=1, causal=True)
        c["kv"] = _log(rng, c["q"], int(max(c["q"] + 1, min(6000, 1.2e9 / (c["seqs"] * c["q"] * heads)))))
    else:
        causal = kind == "chunk"
        c.update(seqs=rng.randint(1, 4), q_rest=1, q=_log(rng, 16, 2000), causal=causal)
        c["long"] = c["seqs"]
        lo = c["q"] if causal else 1
        c["kv"] = _log(rng, lo, int(max(lo + 1, min(16000, 1.0e9 / (c["seqs"] * c["q"] * heads)))))
    return c


def _lengths(c):
    """(new tokens, keys with them) of each sequence: the first `long` bring q tokens, the others q_rest."""
    n = [c["q"] if b < c["long"] else c["q_rest"] for b in range(c["seqs"])]
    kv = [int(c["kv"] - c["kv"] * c["spread"] * ((b * 379) % 1000) / 1000) for b in range(c["seqs"])]
    return n, [max(k, m, 1) if c["causal"] or c["nodes"] else max(k, 1) for k, m in zip(kv, n)]


def _tree_lengths(c):
    """New tokens of each sequence: the first `chunks` bring a prompt chunk, the others least .. q nodes."""
    return [c["chunk"] if b < c["chunks"] else c["least"] + (b * 379) % (c["q"] - c["least"] + 1) for b in range(c["seqs"])]


def _pages(tokens, page):
    return (tokens + page - 1) // page


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(n):
    at = [0]
    for m in n:
        at.append(at[-1] + m)
    return at


def _parents(n, most, g):
    """Each node's parent in its sequence: mostly one of the few nodes before it, at times the context (-1)."""
    total = sum(n)
    back = torch.randint(1, 9, (total,), generator=g, device="cuda").tolist()
    out = []
    for m in n:
        for i in range(m):
            up = i - back[len(out)]
            out.append(max(up, -1) if m <= most else i - 1)
    return out


def _masks(n, most, parents):
    """Rows of who sees whom, as 32-bit words, by following each node's parent."""
    words, at = [], 0
    for m in n:
        seen = []
        for i in range(m):
            up = parents[at + i]
            seen.append((seen[up] if up >= 0 else 0) | 1 << i if m <= most else 0)
        words += [[(x >> 32 * w & 0xFFFFFFFF) - (x >> 32 * w + 31 & 1) * (1 << 32) for w in range(most // 32)] for x in seen]
        at += m
    return words


def _quantised(rows, hkv, d, g, like):
    """Values of a cache in 8 bits: codes [rows, hkv, d] and exponents + 127 [rows, hkv]."""
    x = torch.randn(rows, hkv, d, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(rows, hkv, 1, generator=g, device="cuda"))
    return _codes(x.to(like))


def _codes(x):
    """E4M3 codes and exponents + 127 of rows of 16-bit values."""
    m, e = torch.frexp(x.float().abs().amax(-1))  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 * 2^9
    s = torch.where(m <= 0.875, e - 9, e - 8).clamp(_LEAST, _MOST)
    s = torch.where(m == 0, torch.full_like(s, _LEAST), s)
    codes = torch.ldexp(x.float(), -s[..., None]).to(torch.float8_e4m3fn)
    return codes, (s + 127).to(torch.uint8)


def _scales(e):
    return torch.ldexp(torch.ones((), device=e.device), e.to(torch.int32) - 127)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    dt = _TYPES[c.get("dtype", "bf16")]
    st = {"case": c}
    if c["op"] == "rotate":
        i = torch.arange(c["turned"] // 2, dtype=torch.float64, device="cuda")
        st["inv_freq"] = (10000.0 ** (-2.0 * i / c["turned"]) / c["stretch"]).float()
        rows = c["rows"] + c["pad"]
        if c["batch"] == 0:  # serving: rows of a ragged batch
            pos = torch.randint(0, c["far"], (c["rows"],), generator=g, device="cuda", dtype=torch.int32)
            st["positions"] = torch.cat([pos, torch.full((c["pad"],), -1, dtype=torch.int32, device="cuda")])
            shape = lambda h: (rows, h, c["d"])  # noqa: E731
        else:  # training: [batch, heads, tokens, d]
            st["positions"] = torch.arange(rows, dtype=torch.int32, device="cuda")
            shape = lambda h: (c["batch"], h, rows, c["d"])  # noqa: E731
        st["q"], st["k"] = (normal(*shape(h)).to(dt) for h in (c["hq"], c["hk"]))
        st["q_out"], st["k_out"] = torch.zeros_like(st["q"]), torch.zeros_like(st["k"])
    elif c["op"] in ("write", "read"):
        rows, d, hkv = c["rows"] + c["pad"], c["d"], c["hkv"]
        slots = torch.randperm(c["pages"] * c["page"], generator=g, device="cuda")[:c["rows"]].to(torch.int32)
        st["slots"] = torch.cat([slots, torch.full((c["pad"],), -1, dtype=torch.int32, device="cuda")])
        for name in ("k", "v"):
            if c["op"] == "write":
                st[name] = (normal(rows, hkv, d) * torch.exp(0.5 * normal(rows, hkv, 1))).to(dt)
                codes = torch.zeros(c["pages"], c["page"], hkv, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                scale = torch.full((c["pages"], hkv, c["page"]), 127, dtype=torch.uint8, device="cuda")
            else:
                st[name] = torch.zeros(rows, hkv, d, dtype=dt, device="cuda")
                codes, e = _quantised(c["pages"] * c["page"], hkv, d, g, dt)
                codes = codes.view(c["pages"], c["page"], hkv, d)
                scale = e.view(c["pages"], c["page"], hkv).transpose(1, 2).contiguous()
            # a page holds its tokens' heads side by side; the library sees (page, head, slot, d)
            st[name + "_cache"], st[name + "_scale"] = codes.transpose(1, 2), scale.view(torch.float8_e8m0fnu)
    elif c["op"] == "tree":
        n = _tree_lengths(c)
        st["cu_q"] = _i32(_starts(n))
        st["kv_len"] = _i32([max(m, int(c["kv"] - c["kv"] * 0.7 * ((b * 211) % 1000) / 1000)) for b, m in enumerate(n)])
        st["parents"] = _i32(_parents(n, c["nodes"], g) + [-1] * c["pad"])
    else:
        n, kv = _lengths(c)
        columns = _pages(max(kv), c["page"])
        total = sum(_pages(k, c["page"]) for k in kv)
        order = torch.randperm(total + 3, generator=g, device="cuda").tolist()
        table, at = [], 0
        for k in kv:
            m = _pages(k, c["page"])
            table.append(order[at:at + m] + [-1] * (columns - m))
            at += m
        st["table"], st["cu_q"], st["kv_len"] = _i32(table), _i32(_starts(n)), _i32(kv)
        rows, hq = sum(n) + c["pad"], c["hkv"] * c["group"]
        st["q"] = normal(rows, hq, c["d"]).to(dt)
        for name in ("k", "v"):
            if c["bits"] == 8:
                codes, e = _quantised((total + 3) * c["page"], c["hkv"], c["d"], g, dt)
                st[name + "_scale"] = e.view(total + 3, c["page"], c["hkv"]).transpose(1, 2).contiguous().view(torch.float8_e8m0fnu)
                st[name] = codes.view(total + 3, c["page"], c["hkv"], c["d"]).transpose(1, 2)
            else:
                st[name] = normal(total + 3, c["page"], c["hkv"], c["d"]).to(dt).transpose(1, 2)
        if c["nodes"]:
            masks = _masks(n, c["nodes"], _parents(n, c["nodes"], g))
            st["tree"] = _i32(masks + [[0] * (c["nodes"] // 32)] * c["pad"])
        st["out"] = torch.zeros(rows, hq, c["d"], dtype=dt, device="cuda")
        st["lse"] = torch.zeros(hq, rows, dtype=torch.float32, device="cuda")
        st["max_q"] = max(n)
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return _RUN[state["case"]["op"]](state)


def _rotate(st):
    c = st["case"]
    if own:
        from attn_fwd_03_gb300 import attn_rotary, attn_rotary_bwd
        turn = attn_rotary_bwd if c["back"] else attn_rotary
        q, k = turn(st["q"], st["k"], st["positions"], st["inv_freq"], interleaved=c["interleaved"], q_out=st["q_out"],
                    k_out=st["k_out"])
        return {"q": q, "k": k}
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if c["back"]:
        sin = -sin
    if c["batch"] == 0:  # one for all heads of a row
        cos, sin = cos[:, None], sin[:, None]
    m = c["turned"]
    res = {}
    for name in ("q", "k"):
        x = st[name].float()
        a, b = (x[..., 0:m:2], x[..., 1:m:2]) if c["interleaved"] else (x[..., :m // 2], x[..., m // 2:m])
        y0, y1 = a * cos - b * sin, b * cos + a * sin
        y = torch.stack([y0, y1], -1).flatten(-2) if c["interleaved"] else torch.cat([y0, y1], -1)
        y = torch.cat([y, x[..., m:]], -1).to(st[name].dtype)
        res[name] = torch.where((st["positions"] >= 0)[:, None, None], y, st[name + "_out"]) if c["batch"] == 0 else y
    return res


def _write(st):
    if own:
        from attn_fwd_03_gb300 import attn_pages_write_fp8
        attn_pages_write_fp8(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    else:
        rows, page = st["case"]["rows"], st["case"]["page"]
        slots = st["slots"][:rows].long()
        at = (slots // page, slots % page)
        for name in ("k", "v"):
            codes, e = _codes(st[name][:rows])
            st[name + "_cache"].view(torch.uint8).transpose(1, 2)[at] = codes.view(torch.uint8)
            st[name + "_scale"].view(torch.uint8).transpose(1, 2)[at] = e
    return {name: st[name] for name in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _read(st):
    if own:
        from attn_fwd_03_gb300 import attn_pages_read_fp8
        k, v = attn_pages_read_fp8(st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], k=st["k"], v=st["v"])
        return {"k": k, "v": v}
    rows, page = st["case"]["rows"], st["case"]["page"]
    slots = st["slots"][:rows].long()
    at = (slots // page, slots % page)
    res = {}
    for name in ("k", "v"):
        codes = st[name + "_cache"].view(torch.uint8).transpose(1, 2)[at].view(torch.float8_e4m3fn)
        scale = _scales(st[name + "_scale"].view(torch.uint8).transpose(1, 2)[at])
        res[name] = torch.cat([(codes.float() * scale[..., None]).to(st[name].dtype), st[name][rows:]])
    return res


def _tree(st):
    c = st["case"]
    if own:
        from attn_fwd_03_gb300 import attn_tree_plan
        mask, positions = attn_tree_plan(st["parents"], st["cu_q"], st["kv_len"], c["nodes"])
        return {"mask": mask, "positions": positions}
    cu, kv_len, parents, most = st["cu_q"].long(), st["kv_len"].long(), st["parents"].long(), c["nodes"]
    rows, dev = parents.numel(), parents.device
    n = cu[1:] - cu[:-1]
    t = torch.arange(rows, device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=n.numel() - 1)
    i, held = t - cu[seq], t < cu[-1]
    node = torch.arange(most, device=dev)
    up = parents[(cu[:-1, None] + node).clamp(max=rows - 1)]
    live = (node < n[:, None]) & (n <= most)[:, None]
    # who is an ancestor of whom: the parents' relation, squared until it has every distance
    seen = ((up[:, :, None] == node) | (node[:, None] == node)) & live[:, :, None] & live[:, None, :]
    far = 1
    while far < c["q"]:
        seen = torch.matmul(seen.float(), seen.float()) > 0
        far *= 2
    mine = seen[seq, i.clamp(0, most - 1)] & (held & (n[seq] <= most))[:, None]
    bits = (mine.view(rows, most // 32, 32).long() << torch.arange(32, device=dev)).sum(-1)
    depth = torch.where(n[seq] <= most, mine.sum(-1) - 1, i)
    pos = kv_len[seq] - n[seq] + depth
    return {"mask": bits.to(torch.int32), "positions": torch.where(held, pos, -1).int()}


def _attend(st):
    c = st["case"]
    tree = st.get("tree")
    if own:
        if c["bits"] == 8:
            from attn_fwd_03_gb300 import attn_paged_fp8
            out, lse = attn_paged_fp8(st["q"], st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"], st["cu_q"], st["kv_len"],
                                      causal=c["causal"], tree=tree, max_q=st["max_q"], out=st["out"], lse=st["lse"])
        else:
            from attn_fwd_03_gb300 import attn_paged_tree
            out, lse = attn_paged_tree(st["q"], st["k"], st["v"], st["table"], st["cu_q"], st["kv_len"], tree, max_q=st["max_q"],
                                       out=st["out"], lse=st["lse"])
        return {"out": out, "lse": lse}
    q, cu, kv_len, table = st["q"], st["cu_q"].long(), st["kv_len"].long(), st["table"].long().clamp(min=0)
    rows, hq, d = q.shape
    seqs, hkv, group, longest = table.shape[0], c["hkv"], c["group"], st["max_q"]
    keys = table.shape[1] * c["page"]

    def gathered(name):  # (seq, kv head, key, d)
        if c["bits"] == 16:
            return st[name][table].permute(0, 2, 1, 3, 4).reshape(seqs, hkv, keys, d).float()
        codes = st[name].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        codes *= _scales(st[name + "_scale"].view(torch.uint8)[table])[..., None]
        return codes.permute(0, 2, 1, 3, 4).reshape(seqs, hkv, keys, d)

    k, v = gathered("k"), gathered("v")
    at = torch.arange(longest, device=q.device)
    row = (cu[:-1, None] + at).clamp(max=rows - 1)
    qs = q[row].float().view(seqs, longest, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, group * longest, d)
    s = torch.matmul(qs, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(seqs, hkv, group, longest, keys)
    new = cu[1:] - cu[:-1]
    key = torch.arange(keys, device=q.device)
    if tree is not None:  # the context, and the nodes that the row's bits name
        rel = key - (kv_len - new)[:, None]
        words = tree[row]
        bit = torch.gather(words.view(seqs, longest, -1), 2, (rel // 32).clamp(0, words.shape[-1] - 1)[:, None].expand(-1, longest, -1))
        bit = (bit >> (rel % 32)[:, None].int() & 1) != 0
        sees = ((rel < 0) | (rel >= 0) & (rel < new[:, None]))[:, None] & ((rel < 0)[:, None] | bit)
    else:
        last = (kv_len - new)[:, None] + at if c["causal"] else (kv_len - 1)[:, None].expand(seqs, longest)
        sees = key <= torch.minimum(last, kv_len[:, None] - 1)[:, :, None]
    s.masked_fill_(~sees[:, None, None], float("-inf"))
    v = v.masked_fill((key >= kv_len[:, None])[:, None, :, None], 0.0)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hkv, group * longest, keys), v).view(seqs, hkv, group, longest, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(seqs, longest, hq, d)
    lse = (m0 + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(seqs, longest, hq)
    t = torch.arange(rows, device=q.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=seqs - 1)
    here = (t - cu[seq]).clamp(0, longest - 1)
    held = t < cu[-1]
    return {"out": torch.where(held[:, None, None], o[seq, here].to(q.dtype), st["out"]),
            "lse": torch.where(held[None], lse[seq, here].t(), st["lse"])}


_RUN = {"rotate": _rotate, "write": _write, "read": _read, "tree": _tree, "attend": _attend}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rotate":
        rows, heads, size = c["rows"] * max(c["batch"], 1), c["hq"] + c["hk"], _TYPES[c["dtype"]].itemsize
        return {"bytes": 2 * rows * heads * c["d"] * size + 4 * c["rows"] + 2 * c["turned"], "flops": 3 * rows * heads * c["turned"]}
    if c["op"] in ("write", "read"):  # 16-bit rows on one side, codes and a byte for the scale on the other
        return {"bytes": c["rows"] * (2 * c["hkv"] * (3 * c["d"] + 1) + 4), "flops": 0}
    if c["op"] == "tree":
        n = _tree_lengths(c)
        return {"bytes": 4 * (2 * len(n) + 1 + (2 + c["nodes"] // 32) * (sum(n) + c["pad"])), "flops": 0}
    n, kv = _lengths(c)
    hq, row = c["hkv"] * c["group"], c["d"] * 2
    held = c["d"] + 1 if c["bits"] == 8 else row
    if c["nodes"]:  # at least the context and the row itself
        pairs = sum(m * (k - m + 1) for m, k in zip(n, kv))
    else:
        pairs = sum(m * k - (m * (m - 1) // 2 if c["causal"] else 0) for m, k in zip(n, kv))
    tables = 4 * (2 * len(n) + 1 + sum(_pages(k, c["page"]) for k in kv)) + sum(n) * c["nodes"] // 8
    return {"bytes": 2 * sum(n) * hq * row + 4 * sum(n) * hq + 2 * sum(kv) * c["hkv"] * held + tables,
            "flops": 4 * c["d"] * hq * pairs}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "tree":
        return None
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "write": _exact_write, "read": _exact_read, "attend": _exact_attend}[c["op"]](c, st)


def _exact_rotate(c, st):
    """Each pair as a complex number times exp(i angle); a head at a time."""
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(st["positions"].double(), st["inv_freq"].double()) * (-1.0 if c["back"] else 1.0))
    m, res = c["turned"], {}
    for name in ("q", "k"):
        x, out = st[name], st[name + "_out"].double()
        for h in range(x.shape[1]):
            y = x[:, h].double()
            z = y[..., :m].unflatten(-1, (m // 2, 2) if c["interleaved"] else (2, m // 2))
            z = torch.complex(z[..., 0], z[..., 1]) if c["interleaved"] else torch.complex(z[..., 0, :], z[..., 1, :])
            z = z * turn
            y[..., :m] = torch.stack([z.real, z.imag], -1 if c["interleaved"] else -2).flatten(-2)
            out[:, h] = torch.where((st["positions"] >= 0)[:, None], y, out[:, h])
        res[name] = out
    return res


def _exact_write(c, st):
    """The values over their scales, not rounded, and the scales, by comparing with the powers of two one after another."""
    slots = st["slots"][:c["rows"]].long()
    res = {}
    for name in ("k", "v"):
        x = st[name][:c["rows"]].double()
        top, scale = x.abs().amax(-1), torch.full(x.shape[:2], 2.0 ** _LEAST, dtype=torch.float64, device="cuda")
        for e in range(_LEAST, _MOST):
            scale = torch.where(top > 448.0 * 2.0 ** e, 2.0 ** (e + 1), scale)
        codes = st[name + "_cache"].double().transpose(1, 2).reshape(-1, c["hkv"], c["d"])
        codes[slots] = x / scale[..., None]
        held = st[name + "_scale"].double().transpose(1, 2).reshape(-1, c["hkv"])
        held[slots] = scale
        res[name + "_cache"] = codes.view(c["pages"], c["page"], c["hkv"], c["d"]).transpose(1, 2)
        res[name + "_scale"] = held.view(c["pages"], c["page"], c["hkv"]).transpose(1, 2)
    return res


def _exact_read(c, st):
    res = {}
    for name in ("k", "v"):
        values = st[name + "_cache"].double() * st[name + "_scale"].double()[..., None]
        out = st[name].double()
        out[:c["rows"]] = values.transpose(1, 2).reshape(-1, c["hkv"], c["d"])[st["slots"][:c["rows"]].long()]
        res[name] = out
    return res


def _exact_attend(c, st):
    """Sequence by sequence and head by head in float64."""
    n, kv = _lengths(c)
    out, lse = st["out"].double(), st["lse"].double()
    start = 0
    for b in range(c["seqs"]):
        ctx = kv[b] - n[b]
        if c["nodes"]:
            words = st["tree"][start:start + n[b]].long() & 0xFFFFFFFF
            bits = torch.stack([words[:, j // 32] // 2 ** (j % 32) % 2 for j in range(n[b])], 1) != 0
        for h in range(c["hkv"]):
            ids = st["table"][b, :_pages(kv[b], c["page"])].long()
            k, v = (st[x].view(torch.uint8)[ids, h].view(st[x].dtype).reshape(-1, c["d"])[:kv[b]].double() for x in ("k", "v"))
            if c["bits"] == 8:
                k, v = (t * st[x].view(torch.uint8)[ids, h].view(torch.float8_e8m0fnu).reshape(-1, 1)[:kv[b]].double()
                        for t, x in ((k, "k_scale"), (v, "v_scale")))
            for g in range(c["group"]):
                hq = h * c["group"] + g
                for r0 in range(0, n[b], 2048):
                    r1 = min(n[b], r0 + 2048)
                    s = (st["q"][start + r0:start + r1, hq].double() @ k.t()) / math.sqrt(c["d"])
                    if c["nodes"]:
                        s[:, ctx:] = s[:, ctx:].masked_fill(~bits[r0:r1], -math.inf)
                    elif c["causal"]:
                        i = torch.arange(r0, r1, device=s.device)[:, None] + ctx
                        s = s.masked_fill(torch.arange(kv[b], device=s.device)[None] > i, -math.inf)
                    z = torch.logsumexp(s, 1)
                    out[start + r0:start + r1, hq] = torch.exp(s - z[:, None]) @ v
                    lse[hq, start + r0:start + r1] = z
        start += n[b]
    return {"out": out, "lse": lse}
