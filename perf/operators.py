"""Cases of the paged key/value cache: its page tables, its writes, and attention over it.

Serving keeps the keys and values of many sequences in pages of `page` tokens that a block table
names. Each engine step hands over, for every sequence, how many new tokens it brings; the step then
takes pages for them and says where each token goes (plan), stores their keys and values (write),
attends from the new tokens to everything cached (attend), and at the end of a sequence gives its
pages back (release).

`own = False` computes these with elementary torch operations, `own = True` calls the library.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence, one new token, a short context: the latency of a single-user step
        {"name": "attend one token", "op": "attend", "seqs": 1, "long": 0, "q": 1, "q_rest": 1, "kv": 517, "spread": 0.0,
         "hkv": 8, "group": 4, "d": 128, "page": 16, "dtype": "bf16", "causal": True, "pad": 0},
        # a full decode batch of ragged contexts: the cache read is all there is
        {"name": "attend decode batch", "op": "attend", "seqs": 64, "long": 0, "q": 1, "q_rest": 1, "kv": 8192, "spread": 0.5,
         "hkv": 8, "group": 4, "d": 128, "page": 64, "dtype": "bf16", "causal": True, "pad": 0},
        # several drafted tokens a sequence are verified at once; an odd number of heads to a group
        {"name": "attend drafted tokens", "op": "attend", "seqs": 16, "long": 0, "q": 5, "q_rest": 5, "kv": 4001, "spread": 0.6,
         "hkv": 4, "group": 7, "d": 64, "page": 32, "dtype": "fp16", "causal": True, "pad": 0},
        # decoding sequences share the step with a chunk of a new prompt; rows padded to a fixed count
        {"name": "attend mixed step", "op": "attend", "seqs": 17, "long": 1, "q": 512, "q_rest": 1, "kv": 4096, "spread": 0.5,
         "hkv": 8, "group": 4, "d": 128, "page": 64, "dtype": "bf16", "causal": True, "pad": 16},
        # a decoder's rows against an encoder's states of another length, every state visible
        {"name": "attend encoder states", "op": "attend", "seqs": 8, "long": 8, "q": 448, "q_rest": 1, "kv": 1500, "spread": 0.3,
         "hkv": 16, "group": 1, "d": 64, "page": 128, "dtype": "bf16", "causal": False, "pad": 0},
        # a late chunk of a long prompt: 4096 new tokens on top of 28672 cached ones
        {"name": "attend long prompt chunk", "op": "attend", "seqs": 1, "long": 1, "q": 4096, "q_rest": 1, "kv": 32768,
         "spread": 0.0, "hkv": 8, "group": 4, "d": 128, "page": 128, "dtype": "bf16", "causal": True, "pad": 0},
        # the keys and values of one decode step
        {"name": "write decode step", "op": "write", "rows": 64, "pad": 0, "hkv": 8, "d": 128, "page": 64, "pages": 1024,
         "dtype": "bf16"},
        # the keys and values of a step full of prompt chunks, its rows padded
        {"name": "write prompt chunks", "op": "write", "rows": 16301, "pad": 83, "hkv": 8, "d": 128, "page": 32,
         "pages": 2048, "dtype": "fp16"},
        # tables of a decode step: a few sequences cross into a new page
        {"name": "plan decode step", "op": "plan", "seqs": 64, "long": 0, "q": 1, "q_rest": 1, "kv": 4096, "spread": 0.9,
         "page": 16, "pad": 0},
        # tables of a large step: hundreds of sequences, long chunks among them, padded rows
        {"name": "plan prompt chunks", "op": "plan", "seqs": 500, "long": 31, "q": 2011, "q_rest": 7, "kv": 16384,
         "spread": 0.9, "page": 32, "pad": 41},
        # two of sixteen sequences have ended
        {"name": "release a few", "op": "release", "seqs": 16, "kv": 2048, "spread": 0.9, "page": 64, "every": 8},
        # half of a large batch is dropped at once
        {"name": "release half a batch", "op": "release", "seqs": 777, "kv": 16384, "spread": 0.9, "page": 16, "every": 2},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "write", "plan", "release"])
    if op == "attend":
        c = {"op": op, "hkv": rng.randint(1, 8), "group": rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16]), "d": rng.choice([64, 128]),
             "page": rng.choice([16, 32, 64, 128, 256]), "dtype": rng.choice(["bf16", "fp16"])}
        kind = rng.choice(["decode", "drafted", "mixed", "chunk", "states"])
        if kind in ("decode", "drafted"):
            c.update(seqs=_log(rng, 1, 96), long=0, q=1, q_rest=1 if kind == "decode" else rng.randint(2, 9), causal=True)
            c["q"] = c["q_rest"]
            room = 1.2e9 / (c["seqs"] * c["hkv"] * c["d"] * 4)
            c["kv"] = _log(rng, c["q"], int(max(c["q"] + 1, min(40000, room))))
        elif kind == "mixed":
            c.update(seqs=rng.randint(2, 24), long=1, q=_log(rng, 8, 700), q_rest=1, causal=True)
            room = 1.5e9 / (c["seqs"] * c["q"] * c["hkv"] * c["group"])
            c["kv"] = _log(rng, c["q"], int(max(c["q"] + 1, min(6000, room))))
        else:
            causal = kind == "chunk"
            c.update(seqs=rng.randint(1, 4), q_rest=1, q=_log(rng, 16, 2500), causal=causal)
            c["long"] = c["seqs"]
            room = 1.5e9 / (c["seqs"] * c["q"] * c["hkv"] * c["group"])
            lo = c["q"] if causal else 1
            c["kv"] = _log(rng, lo, int(max(lo + 1, min(16000, room))))
        c["spread"] = round(rng.uniform(0.0, 0.9), 2)
        c["pad"] = rng.choice([0, 0, 1, 7, 33])
        return c
    if op == "write":
        return {"op": op, "rows": _log(rng, 1, 16000), "pad": rng.choice([0, 0, 3, 50]), "hkv": rng.randint(1, 8),
                "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128, 256]), "pages": rng.randint(1100, 2000),
                "dtype": rng.choice(["bf16", "fp16"])}
    if op == "plan":
        seqs = _log(rng, 1, 500)
        return {"op": op, "seqs": seqs, "long": rng.randint(0, min(seqs, 30)), "q": _log(rng, 1, 2000), "q_rest": rng.randint(0, 7),
                "kv": _log(rng, 2000, 16000), "spread": round(rng.uniform(0.0, 0.9), 2), "page": rng.choice([16, 32, 64, 128, 256]),
                "pad": rng.choice([0, 0, 5, 64])}
    return {"op": op, "seqs": _log(rng, 1, 770), "kv": _log(rng, 1, 16000), "spread": round(rng.uniform(0.0, 0.9), 2),
            "page": rng.choice([16, 32, 64, 128, 256]), "every": rng.randint(1, 9)}


def _lengths(c):
    """(new tokens, keys with them) of each sequence: the first `long` bring q tokens, the others q_rest."""
    n = [c["q"] if b < c["long"] else c["q_rest"] for b in range(c["seqs"])]
    kv = [int(c["kv"] - c["kv"] * c["spread"] * ((b * 379) % 1000) / 1000) for b in range(c["seqs"])]
    return n, [max(k, m, 1) if c.get("causal", True) else max(k, 1) for k, m in zip(kv, n)]


def _pages(tokens, page):
    return (tokens + page - 1) // page


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(kv, page, columns, order):
    """A block table whose rows take the pages of `order` in turn, and how many were taken."""
    rows, at = [], 0
    for n in kv:
        m = _pages(n, page)
        rows.append(order[at:at + m] + [-1] * (columns - m))
        at += m
    return _i32(rows), at


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    st = {"case": c}
    if c["op"] == "attend":
        dt = _TYPES[c["dtype"]]
        n, kv = _lengths(c)
        columns = _pages(max(kv), c["page"])
        total = sum(_pages(k, c["page"]) for k in kv)
        order = torch.randperm(total + 3, generator=g, device="cuda").tolist()
        st["table"], _ = _table(kv, c["page"], columns, order)
        st["cu_q"] = _i32([sum(n[:b]) for b in range(len(n) + 1)])
        st["kv_len"] = _i32(kv)
        rows = sum(n) + c["pad"]
        hq = c["hkv"] * c["group"]
        st["q"] = normal(rows, hq, c["d"]).to(dt)
        # a page holds its tokens' heads side by side; the library sees (page, head, slot, d)
        for name in ("k", "v"):
            st[name] = normal(total + 3, c["page"], c["hkv"], c["d"]).to(dt).transpose(1, 2)
        st["out"] = torch.zeros(rows, hq, c["d"], dtype=dt, device="cuda")
        st["lse"] = torch.zeros(hq, rows, dtype=torch.float32, device="cuda")
        st["max_q"] = max(n)
    elif c["op"] == "write":
        dt = _TYPES[c["dtype"]]
        rows = c["rows"] + c["pad"]
        for name in ("k", "v"):
            st[name] = normal(rows, c["hkv"], c["d"]).to(dt)
            st[name + "_cache"] = torch.zeros(c["pages"], c["page"], c["hkv"], c["d"], dtype=dt, device="cuda").transpose(1, 2)
        slots = torch.randperm(c["pages"] * c["page"], generator=g, device="cuda")[:c["rows"]].to(torch.int32)
        st["slots"] = torch.cat([slots, torch.full((c["pad"],), -1, dtype=torch.int32, device="cuda")])
        st["rows"] = c["rows"]
    elif c["op"] == "plan":
        n, kv = _lengths(c)
        old = [k - m for k, m in zip(kv, n)]
        columns = _pages(max(kv), c["page"]) + 2
        total = sum(_pages(k, c["page"]) for k in kv) + 5
        order = torch.randperm(total, generator=g, device="cuda").tolist()
        st["table"], taken = _table(old, c["page"], columns, order)
        free = order[taken:]
        st["free_pages"] = _i32(free + [0] * taken)
        st["free_count"] = _i32([len(free)])
        st["q_len"], st["kv_len"] = _i32(n), _i32(old)
        st["rows"] = sum(n) + c["pad"]
    else:
        kv = _lengths(dict(c, q=0, q_rest=0, long=0))[1]
        columns = _pages(max(kv), c["page"])
        total = sum(_pages(k, c["page"]) for k in kv) + 9
        order = torch.randperm(total, generator=g, device="cuda").tolist()
        st["table"], taken = _table(kv, c["page"], columns, order)
        st["free_pages"] = _i32(order[taken:] + [0] * taken)
        st["free_count"] = _i32([total - taken])
        st["kv_len"] = _i32(kv)
        st["done"] = _i32([1 if b % c["every"] == 0 else 0 for b in range(c["seqs"])])
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    return _RUN[state["case"]["op"]](state)


def _attend(st):
    c = st["case"]
    if own:
        from attn_fwd_03_gb300 import attn_paged
        out, lse = attn_paged(st["q"], st["k"], st["v"], st["table"], st["cu_q"], st["kv_len"], causal=c["causal"],
                              max_q=st["max_q"], out=st["out"], lse=st["lse"])
        return {"out": out, "lse": lse}
    q, cu, kv_len, table = st["q"], st["cu_q"].long(), st["kv_len"].long(), st["table"].long().clamp(min=0)
    rows, hq, d = q.shape
    seqs, hkv, group, longest = table.shape[0], c["hkv"], c["group"], st["max_q"]
    keys = table.shape[1] * c["page"]
    # (seq, kv head, key, d)
    k, v = (st[x][table].permute(0, 2, 1, 3, 4).reshape(seqs, hkv, keys, d).float() for x in ("k", "v"))
    at = torch.arange(longest, device=q.device)
    row = (cu[:-1, None] + at).clamp(max=rows - 1)
    qs = q[row].float().view(seqs, longest, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, group * longest, d)
    s = torch.matmul(qs, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(seqs, hkv, group, longest, keys)
    new = cu[1:] - cu[:-1]
    last = (kv_len - new)[:, None] + at if c["causal"] else (kv_len - 1)[:, None].expand(seqs, longest)
    last = torch.minimum(last, kv_len[:, None] - 1)
    key = torch.arange(keys, device=q.device)
    s.masked_fill_((key > last[:, :, None])[:, None, None], float("-inf"))
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


def _write(st):
    if own:
        from attn_fwd_03_gb300 import attn_pages_write
        attn_pages_write(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"])
        return {"k": st["k_cache"], "v": st["v_cache"]}
    slots = st["slots"][:st["rows"]].long()
    page, slot = slots // st["case"]["page"], slots % st["case"]["page"]
    st["k_cache"].transpose(1, 2)[page, slot] = st["k"][:st["rows"]]
    st["v_cache"].transpose(1, 2)[page, slot] = st["v"][:st["rows"]]
    return {"k": st["k_cache"], "v": st["v_cache"]}


def _plan(st):
    page = st["case"]["page"]
    if own:
        from attn_fwd_03_gb300 import attn_pages_plan
        cu_q, new_len, slots, positions, free_left = attn_pages_plan(st["q_len"], st["kv_len"], st["table"], st["free_pages"],
                                                                     st["free_count"], page, st["rows"])
        return {"cu_q": cu_q, "new_len": new_len, "slots": slots, "positions": positions, "free_left": free_left,
                "table": st["table"]}
    n, old, table, count = st["q_len"].long(), st["kv_len"].long(), st["table"], st["free_count"].long()
    cu = torch.cat([torch.zeros_like(count), n.cumsum(0)])
    new = old + n
    had, has = (old + page - 1) // page, (new + page - 1) // page
    first = (has - had).cumsum(0) - (has - had)  # pages taken by the sequences before
    col = torch.arange(table.shape[1], device=table.device)
    taken = (count - 1 - first[:, None] - (col - had[:, None])).clamp(0, st["free_pages"].numel() - 1)
    table = torch.where((col >= had[:, None]) & (col < has[:, None]), st["free_pages"][taken], table)
    t = torch.arange(st["rows"], device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=n.numel() - 1)
    pos = old[seq] + t - cu[seq]
    held = t < cu[-1]
    slot = table[seq, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    none = torch.full_like(t, -1)
    return {"cu_q": cu.int(), "new_len": new.int(), "slots": torch.where(held, slot, none).int(),
            "positions": torch.where(held, pos, none).int(), "free_left": (count - (has - had).sum()).int(), "table": table}


def _release(st):
    page = st["case"]["page"]
    if own:
        from attn_fwd_03_gb300 import attn_pages_release
        new_len, free_left = attn_pages_release(st["done"], st["kv_len"], st["table"], st["free_pages"], st["free_count"], page)
        return {"new_len": new_len, "free_left": free_left, "free_pages": st["free_pages"]}
    gone, table, count = st["done"] != 0, st["table"], st["free_count"].long()
    pages = torch.where(gone, (st["kv_len"].long() + page - 1) // page, 0)
    first = count + pages.cumsum(0) - pages
    col = torch.arange(table.shape[1], device=table.device)
    spare = st["free_pages"].numel()
    to = torch.where(col < pages[:, None], first[:, None] + col, spare)
    free = torch.cat([st["free_pages"], st["free_pages"][:1]])  # one place more, for what is not given back
    free[to.reshape(-1)] = table.reshape(-1)
    return {"new_len": torch.where(gone, 0, st["kv_len"]).int(), "free_left": (count + pages.sum()).int(),
            "free_pages": free[:spare]}


_RUN = {"attend": _attend, "write": _write, "plan": _plan, "release": _release}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "attend":
        n, kv = _lengths(c)
        hq, row = c["hkv"] * c["group"], c["d"] * 2
        pairs = sum(m * k - (m * (m - 1) // 2 if c["causal"] else 0) for m, k in zip(n, kv))
        tables = 4 * (2 * len(n) + 1 + sum(_pages(k, c["page"]) for k in kv))
        return {"bytes": 2 * sum(n) * hq * row + 4 * sum(n) * hq + 2 * sum(kv) * c["hkv"] * row + tables,
                "flops": 4 * c["d"] * hq * pairs}
    if c["op"] == "write":
        return {"bytes": c["rows"] * (2 * 2 * c["hkv"] * c["d"] * 2 + 4), "flops": 0}
    if c["op"] == "plan":
        n, kv = _lengths(c)
        new = sum(_pages(k, c["page"]) - _pages(k - m, c["page"]) for m, k in zip(n, kv))
        return {"bytes": 4 * (4 * len(n) + 1 + 2 + 2 * (sum(n) + c["pad"]) + 2 * new), "flops": 0}
    kv = _lengths(dict(c, q=0, q_rest=0, long=0))[1]
    gone = sum(_pages(k, c["page"]) for b, k in enumerate(kv) if b % c["every"] == 0)
    return {"bytes": 4 * (3 * len(kv) + 2 + 2 * gone), "flops": 0}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    """Attention sequence by sequence and head by head in float64; the other operators move whole values."""
    if case["op"] != "attend":
        return None
    c, st = case, prepare(case, seed)
    n, kv = _lengths(c)
    out, lse = st["out"].double(), st["lse"].double()
    start = 0
    for b in range(c["seqs"]):
        for h in range(c["hkv"]):
            ids = st["table"][b, :_pages(kv[b], c["page"])].long()
            k, v = (st[x][ids, h].reshape(-1, c["d"])[:kv[b]].double() for x in ("k", "v"))
            for g in range(c["group"]):
                hq = h * c["group"] + g
                for r0 in range(0, n[b], 2048):
                    r1 = min(n[b], r0 + 2048)
                    s = (st["q"][start + r0:start + r1, hq].double() @ k.t()) / math.sqrt(c["d"])
                    if c["causal"]:
                        i = torch.arange(r0, r1, device=s.device)[:, None] + (kv[b] - n[b])
                        s = s.masked_fill(torch.arange(kv[b], device=s.device)[None] > i, -math.inf)
                    z = torch.logsumexp(s, 1)
                    out[start + r0:start + r1, hq] = torch.exp(s - z[:, None]) @ v
                    lse[hq, start + r0:start + r1] = z
        start += n[b]
    return {"out": out, "lse": lse}
