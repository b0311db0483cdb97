"""The operators of a verification step whose target attends through a sliding window and whose drafts were
sampled, as they are measured: page tables and slot maps from request lengths, packed keys and values into their
slots, attention with a window and sinks over the paged cache (single tokens, draft trees, prompts), and the
verification of drafted tokens against the target's probabilities.  Each case runs in a plain form (elementary torch
operations in 32 bits, 64 where the decision needs them) or, where ``own`` is true, through the framework's entry
points.

Cache format: a page holds ``P`` tokens of all key/value heads; per head one chunk of P * dh * 9 / 8 bytes:
key codes [P][dh/2], key scales [P][dh/16], value codes, value scales.  A code is e2m1 (two per byte, the even
dimension in the low half), a scale is e4m3 for 16 dimensions.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token behind a short window: latency
        dict(name="slide_one", op="window", form="token", R=1, n=1, len=1000, window=512, sinks=4, Hq=32, Hkv=8,
             dh=128, P=64),
        # next tokens of a busy server, long conversations
        dict(name="slide_batch", op="window", form="token", R=64, n=1, len=60000, window=4096, sinks=4, Hq=32, Hkv=8,
             dh=128, P=64),
        # the verification of a batch of trees (the batch build's requests and budget), small pages
        dict(name="slide_trees", op="window", form="tree", R=32, n=65, len=9000, window=2048, sinks=4, Hq=32, Hkv=8,
             dh=128, P=16),
        # two prompts through the cache
        dict(name="slide_prompt", op="window", form="chain", R=2, n=8192, len=0, window=2048, sinks=4, Hq=32, Hkv=8,
             dh=128, P=64),
        # a step of a server: a piece of a prompt and other users' next tokens, packed
        dict(name="slide_mixed", op="window", form="packed", R=33, n=2001, len=12000, window=4096, sinks=16, Hq=32,
             Hkv=8, dh=128, P=64),
        # pages and slots of one step's trees
        dict(name="plan_step", op="plan", R=32, n=65, long=0, len=9000, window=2048, sinks=4, P=16),
        # pages and slots of a large server's step: prompts among single tokens and drafts
        dict(name="plan_server", op="plan", R=1024, n=9, long=2000, len=32000, window=4096, sinks=4, P=64),
        # the keys and values of one step's trees
        dict(name="put_step", op="put", R=8, n=129, long=0, len=1000, Hkv=8, dh=128, P=64),
        # the keys and values of pieces of several prompts
        dict(name="put_prompts", op="put", R=8, n=4000, long=0, len=4000, Hkv=8, dh=128, P=64),
        # one user's drafted chain (the smallest build's vocabulary)
        dict(name="verify_one", op="verify", R=1, B=8, kids=1, depth=8, V=32000, bf16=False, mix="plain"),
        # a server's drafted chains, requests with settings of their own
        dict(name="verify_chains", op="verify", R=64, B=7, kids=1, depth=7, V=151936, bf16=True, mix="mixed"),
        # sampled trees of a batch
        dict(name="verify_trees", op="verify", R=16, B=128, kids=4, depth=16, V=151936, bf16=True, mix="plain"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["token", "token", "tree", "chain", "packed", "plan", "put", "verify", "verify", "verify"])
    dh, P = rng.choice([128, 128, 64]), rng.choice([16, 32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    window, sinks = _log(rng, 1, 5000), rng.choice([0, 1, 4, 4, 16, 100])
    win = dict(op="window", form=op, window=window, sinks=sinks, Hq=Hkv * g, Hkv=Hkv, dh=dh, P=P)
    if op == "token":
        return dict(win, R=_log(rng, 1, 64), n=1, len=_log(rng, 1, 60000))
    if op == "tree":
        R, n = _log(rng, 1, 32), 1 + _log(rng, 1, 256)
        win["window"] = min(window, max(64, 32 * 65 * 4 * 2048 // (R * n * g)))
        return dict(win, R=R, n=n, len=_log(rng, 1, 20000))
    if op == "chain":
        R = _log(rng, 1, 8)
        n = _log(rng, 2, 16384 // R)
        win["window"] = min(window, max(1, 8192 * 2048 * 64 // (R * n * Hkv * g)))
        return dict(win, R=R, n=n, len=rng.choice([0, _log(rng, 1, 9000)]))
    if op == "packed":
        win["window"] = min(window, 4096)
        return dict(win, R=_log(rng, 2, 48), n=_log(rng, 2, 2000), len=_log(rng, 1, 12000))
    if op == "plan":
        R = _log(rng, 1, 1024)
        return dict(op="plan", R=R, n=_log(rng, 1, 129), long=rng.choice([0, _log(rng, 130, 2000)]),
                    len=_log(rng, 1, 32000), window=rng.choice([0, window]), sinks=sinks, P=P)
    if op == "put":
        R = _log(rng, 1, 64)
        return dict(op="put", R=R, n=_log(rng, 1, 32000 // R), long=0, len=_log(rng, 1, 4000), Hkv=Hkv, dh=dh, P=P)
    V, R = _log(rng, 500, 152000), _log(rng, 1, 64)
    kids = rng.choice([1, 1, 2, 3, 4])
    B = _log(rng, 1, 16) if kids == 1 else _log(rng, 2, 128 if R <= 16 else 16)
    return dict(op="verify", R=R, B=B, kids=kids, depth=B if kids == 1 else min(B, rng.randint(1, 16)), V=V,
                bf16=rng.random() < 0.5, mix=rng.choice(["plain", "plain", "mixed", "nucleus", "topk"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _nibble_pairs(g):
    """65536 byte values in the frequencies in which normal data, scaled by its block's largest value, has them."""
    x = torch.randn(4096, 16, generator=g, device=DEV)
    x = x * (6.0 / x.abs().amax(1, keepdim=True))
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    nib = torch.bucketize(x.abs(), mid).to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)
    nib = nib.reshape(-1)
    other = nib[torch.randperm(nib.numel(), generator=g, device=DEV)]
    return nib | (other << 4)


def _pool(g, pages, Hkv, dh, P):
    """One layer's pages as quantised data fills them: [1, pages, Hkv * P * dh * 9 / 8] bytes."""
    lut = _nibble_pairs(g)
    chunk = P * dh * 9 // 8
    pool = torch.empty(1, pages, Hkv, chunk, dtype=torch.uint8, device=DEV)
    half = chunk // 2
    code = P * dh // 2
    for at in (0, half):
        i = torch.randint(0, 65536, (1, pages, Hkv, code), generator=g, device=DEV, dtype=torch.int32)
        pool[..., at:at + code] = lut[i]
        s = torch.randint(0x21, 0x2C, (1, pages, Hkv, half - code), generator=g, device=DEV, dtype=torch.uint8)
        pool[..., at + code:at + half] = s           # scales 0.14 .. 0.34
    return pool.view(1, pages, Hkv * chunk)


def _lens(rs, R, most):
    n = rs.randint(max(0, most // 4), most + 1, R)
    n[0] = most
    return n


def _mask(rs, R, B):
    """Random trees in canonical order: the nodes' numbers and the ancestor masks."""
    n = rs.randint(max(1, (3 * B) // 4), B + 1, R)
    n[0] = B
    anc = np.zeros((R, B, B), bool)
    for i in range(B):
        parent = (rs.random_sample(R) * (i + 1)).astype(np.int64) - 1
        anc[:, i] = np.where(parent[:, None] >= 0, anc[np.arange(R), np.maximum(parent, 0)], False)
        anc[:, i, i] = True
        anc[i >= n, i] = False
    words = (B + 31) // 32
    bits = np.zeros((R, B, words * 32), np.uint64)
    bits[:, :, :B] = anc
    mask = (bits.reshape(R, B, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return n, torch.from_numpy(mask.view(np.int32)).to(DEV)


def _counts(rs, c):
    """Tokens per request: up to n, and `long` (a piece of a prompt) for every eighth request."""
    count = rs.randint(max(1, c["n"] // 2), c["n"] + 1, c["R"])
    count[0] = c["n"]
    if c["long"]:
        count[::8] = rs.randint(c["long"] // 2, c["long"] + 1, len(count[::8]))
        count[0] = c["long"]
    return count


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tables(rs, first, last, pages, width):
    """Page tables whose row r holds its first[r] first pages and those in [.., ..) of last[r], in no order."""
    ids = rs.permutation(pages)
    table = np.full((len(first), width), -1, np.int32)
    at = 0
    for r in range(len(first)):
        slots = np.concatenate([np.arange(min(first[r], last[r][0])), np.arange(last[r][0], last[r][1])])
        table[r, slots] = ids[at:at + len(slots)]
        at += len(slots)
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    return table, refs


def prepare(case, seed):
    c = case
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 32))
    s = dict(case=c)
    if c["op"] == "verify":
        return _prepare_verify(c, g, rs, s)
    R, P = c["R"], c["P"]
    lens = _lens(rs, R, c["len"])
    if c["op"] == "window":
        return _prepare_window(c, g, rs, s, lens)
    count = _counts(rs, c)
    T = R * c["n"] + (-(-R // 8) * c["long"])
    s.update(T=T, count=_int(count), most=max(c["n"], c["long"]))
    window, sinks = c.get("window", 0), c.get("sinks", 0)
    # the step before this one held its own window's pages, `back` tokens before this one's
    back = 64
    f = lens
    have = -(-lens // P)
    lo = np.maximum(0, (f - back - window + 1) // P) if window else np.zeros(R, np.int64)
    lo = np.minimum(lo, have)
    first = np.full(R, -(-sinks // P)) if window else np.zeros(R, np.int64)
    width = int((lens + max(c["n"], c["long"])).max()) // P + 2
    per = (-(-sinks // P) + (window + back) // P + 2) if window else c["len"] // P + 1
    pages = R * (min(per, c["len"] // P + 2) + max(c["n"], c["long"]) // P + 2)
    table, refs = _tables(rs, first, list(zip(lo, have)), pages, width)
    s.update(lens=_int(lens), rows=_int(np.arange(R)), table=_int(table), refs=_int(refs))
    if c["op"] == "put":
        mag = torch.exp(torch.randn(2, 1, c["Hkv"], c["dh"], generator=g, device=DEV) * 0.5)
        x = torch.randn(2, T, c["Hkv"], c["dh"], generator=g, device=DEV)
        x.mul_(mag)
        # pages of the tokens to come, and the packed tokens' slots
        free = np.flatnonzero(refs == 0)
        at = 0
        slot = np.full(T, -1, np.int64)
        start = np.concatenate([[0], np.cumsum(count)])
        for r in range(R):
            lack = [j for j in range(lens[r] // P, -(-(lens[r] + count[r]) // P)) if table[r, j] < 0]
            table[r, lack] = free[at:at + len(lack)]
            refs[table[r, lack]] = 1
            at += len(lack)
            pos = lens[r] + np.arange(count[r])
            slot[start[r]:start[r + 1]] = table[r, pos // P].astype(np.int64) * P + pos % P
        s.update(K=x[0].to(torch.bfloat16), V=x[1].to(torch.bfloat16), slot=_int(slot), table=_int(table),
                 refs=_int(refs), start=_int(start))
    Hkv, dh = c.get("Hkv", 1), c.get("dh", 64)
    s["pool"] = torch.zeros(1, pages, Hkv * P * dh * 9 // 8, dtype=torch.uint8, device=DEV)
    if own:
        from speculative_decoding_draft_06_gb300 import dartree
        s["cache"] = dartree.KVCache(1, pages, page_tokens=P, Hkv=Hkv, dh=dh, pool=s["pool"], refs=s["refs"])
    return s


def _prepare_window(c, g, rs, s, lens):
    """Row 0 of a request is at position lens: the tokens of the step are in the cache behind the prefix."""
    R, n, P, Hq, Hkv, dh, W, S = (c[k] for k in ("R", "n", "P", "Hq", "Hkv", "dh", "window", "sinks"))
    count = np.full(R, n)
    if c["form"] == "tree":
        nodes, mask = _mask(rs, R, n - 1)
        count = nodes + 1
        s.update(mask=mask, n_nodes=_int(nodes))
    elif c["form"] == "chain":
        count = rs.randint(max(1, (3 * n) // 4), n + 1, R)
        count[0] = n
        s["n_nodes"] = _int(count - 1)
    elif c["form"] == "packed":
        count = np.ones(R, np.int64)
        count[R // 2] = n
        s["start"] = _int(np.concatenate([[0], np.cumsum(count)]))
    held = -(-(lens + n) // P)
    lo = np.minimum(np.maximum(0, (lens - W + 1) // P), held)
    width = int(held.max()) + 1
    pages = R * (-(-S // P) + (min(W, c["len"] + n) + n) // P + 3) + 1
    table, refs = _tables(rs, np.full(R, -(-S // P)), list(zip(lo, held)), pages, width)
    T = int(count.sum()) if c["form"] == "packed" else R * n
    shape = (T, Hq, dh) if c["form"] == "packed" else (R, n, Hq, dh)
    s.update(pool=_pool(g, pages, Hkv, dh, P), table=_int(table), refs=_int(refs), lens=_int(lens),
             count=[int(x) for x in count], max_len=c["len"] + n,
             Q=torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16),
             O=torch.zeros(*shape, dtype=torch.bfloat16, device=DEV))
    if own:
        from speculative_decoding_draft_06_gb300 import dartree
        s["cache"] = dartree.KVCache(1, pages, page_tokens=P, Hkv=Hkv, dh=dh, pool=s["pool"], refs=s["refs"])
    return s


def _prepare_verify(c, g, rs, s):
    R, B, V, kids = c["R"], c["B"], c["V"], c["kids"]
    # trees of nodes with at most `kids` children and `depth` levels, parents first
    n = rs.randint(max(1, (3 * B) // 4), B + 1, R)
    n[0] = B
    parent = np.full((R, B), -1)
    has, deep = np.zeros((R, B + 1), np.int64), np.zeros((R, B + 1), np.int64)
    nth = np.zeros((R, B), np.int64)
    for i in range(B):
        may = (has[:, :i + 1] < kids) & (deep[:, :i + 1] < c["depth"])
        n[~may.any(1) & (n > i)] = i
        row = np.argmax(rs.random_sample((R, i + 1)) * may, 1)
        parent[:, i], nth[:, i] = row - 1, has[np.arange(R), row]
        has[np.arange(R), row] += 1
        deep[:, i + 1] = deep[np.arange(R), row] + 1
    live = np.arange(B)[None] < n[:, None]
    parent[~live] = -1
    D = B if kids == 1 else B + 1
    t = torch.bfloat16 if c["bf16"] else torch.float32
    zipf = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
    logits = torch.empty(R, B + 1, V, dtype=t, device=DEV)
    draft = torch.empty(R, D, V, dtype=t, device=DEV)
    T = np.full(R, 0.8)
    k, p, m = np.zeros(R), np.ones(R), np.zeros(R)
    if c["mix"] == "topk":
        T, k = np.full(R, 0.6), np.full(R, 20)
    elif c["mix"] == "nucleus":
        p = np.full(R, 0.95)
    elif c["mix"] == "mixed":
        T, k = rs.choice([0.0, 0.6, 0.7, 1.0, 1.3], R), rs.choice([0, 0, 0, 20, 1000], R)
        p, m = rs.choice([0.9, 0.95, 1.0, 1.0], R), rs.choice([0.0, 0.0, 0.05], R)
    Td = np.where(T > 0, T, 1.0)
    token = torch.full((R, B), -1, dtype=torch.int32, device=DEV)
    for r in range(R):
        x = torch.randn(B + 1, V, generator=g, device=DEV) * 2.0
        x += 20.0 + zipf[torch.randperm(V, generator=g, device=DEV)]
        logits[r] = x
        x = x[:D]
        x += torch.randn(D, V, generator=g, device=DEV) * 0.7           # the drafter is near the target
        draft[r] = x
        # the children of a row: drawn from its distribution one after the other, without replacement
        e = torch.empty(D, V, device=DEV).exponential_(generator=g)
        drawn = torch.topk(draft[r].float() / Td[r] - torch.log(e), min(kids, V), dim=1).indices
        i = np.flatnonzero(live[r])
        token[r, torch.from_numpy(i).to(DEV)] = drawn[torch.from_numpy(parent[r, i] + 1).to(DEV),
                                                      torch.from_numpy(nth[r, i]).to(DEV)].int()
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV)  # noqa: E731
    s.update(parent=_int(parent), token=token, n_out=_int(n), logits=logits, draft=draft,
             u=torch.rand(R, B + 1, generator=g, device=DEV), temperature=f(T), top_k=_int(k), top_p=f(p),
             min_p=f(m), draft_temperature=f(Td))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from speculative_decoding_draft_06_gb300 import dartree
        if op == "verify":
            out = dartree.verify(s["parent"], s["token"], s["n_out"], s["logits"], s["draft"], s["u"],
                                 max_len=c["depth"], temperature=s["temperature"], top_k=s["top_k"],
                                 top_p=s["top_p"], min_p=s["min_p"], draft_temperature=s["draft_temperature"])
            return [out["len"], out["nodes"], out["bonus"], out["prob"]]
        cache, table, lens = s["cache"], s["table"], s["lens"]
        if op == "window":
            more = dict(start=s["start"], max_rows=c["n"]) if c["form"] == "packed" else \
                dict(n_nodes=s.get("n_nodes"), mask=s.get("mask"))
            return [cache.window_attention(0, s["Q"], table, lens, max_len=s["max_len"], window=c["window"],
                                           sinks=c["sinks"], offset=0, out=s["O"], **more)]
        if op == "plan":
            cache.release(table, lens, s["rows"], lens)
            out = cache.plan(table, lens, s["count"], max_tokens=s["T"], offset=0, window=c["window"] or None,
                             sinks=c["sinks"])
            return [out["ok"], out["start"], out["row"], out["pos"], out["slot"], table, s["refs"]]
        cache.append_slots(0, s["K"], s["V"], s["slot"])
        return list(cache.read(0, table, lens, s["most"], count=s["count"]))
    return {"verify": _verify, "window": _window, "plan": _plan, "put": _put}[op](s)


# ------------------------------------------------------------------ plain forms
def _token_values(s, page, tok, second):
    """The fp32 values [..., Hkv, dh] of the keys (or values) of tokens `tok` of pages `page`."""
    c = s["case"]
    P, Hkv, dh = c["P"], c["Hkv"], c["dh"]
    chunk = s["pool"][0].view(-1, Hkv, P * dh * 9 // 8)
    at, code = (chunk.shape[-1] // 2 if second else 0), P * dh // 2
    byte = chunk[..., at:at + code].unflatten(-1, (P, dh // 2))[page, :, tok]
    scale = chunk[..., at + code:at + code + P * dh // 16].unflatten(-1, (P, dh // 16))[page, :, tok]
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    two = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)              # byte -> both values
    x = two[byte.int()].flatten(-2).unflatten(-1, (dh // 16, 16))
    return (x * scale.contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _window_rows(s, Q, reqs, i0, mask=None):
    """Rows i0 .. of the requests in the slice, Q [requests, rows, Hq, dh] -> O in 32 bits."""
    c = s["case"]
    P, Hkv, dh, W, S = (c[k] for k in ("P", "Hkv", "dh", "window", "sinks"))
    R, rows = Q.shape[:2]
    table, base = s["table"][reqs], s["lens"][reqs].long()                    # position of row 0
    n = s["n_nodes"][reqs].long() if "n_nodes" in s else None
    far = torch.arange(rows, device=DEV)[None] + i0                           # a row's distance from row 0
    if mask is not None:
        # node i's depth is the number of bits of its mask row
        bits = (mask[:, :, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        bits = bits.flatten(2)[:, :, :rows - 1]                               # [R, nodes, nodes]
        depth = torch.cat([torch.zeros(R, 1, device=DEV, dtype=torch.long), bits.sum(2)], 1)
        q_at = base[:, None] + depth
    else:
        q_at = base[:, None] + far
    # keys: the sinks, then the window's range; where they lie and at which position
    span = torch.arange(min(W, s["max_len"]) - 1 + rows, device=DEV)
    lo = (base + i0 - W + 1).clamp(min=0)[:, None]
    place = torch.cat([torch.arange(S, device=DEV).expand(R, S), lo + span], 1)
    sink = torch.arange(place.shape[1], device=DEV)[None] < S
    node = place - base[:, None] - 1                                          # place -> node (row - 1)
    if mask is not None:
        at = torch.where(node >= 0, base[:, None] + depth.gather(1, (node + 1).clamp(0, rows - 1)), place)
        tree = torch.cat([torch.zeros_like(bits[:, :1]), bits], 1).gather(
            2, node.clamp(0, rows - 2)[:, None].expand(R, rows, -1)) == 1
        seen = (node < 0)[:, None] | (tree & (node < rows - 1)[:, None])
    else:
        at = place
        seen = place[:, None] <= q_at[:, :, None]
    dup = torch.where(sink, False, place < S)                                 # already among the sinks
    seen = seen & ~dup[:, None] & ((at[:, None] > q_at[:, :, None] - W) | (at < S)[:, None])
    slot = (place // P).clamp(max=table.shape[1] - 1)
    page = table.gather(1, slot).clamp(min=0).long()
    tok = place % P
    K = _token_values(s, page, tok, False).transpose(1, 2)                    # [R, Hkv, keys, dh]
    q = Q.float().view(R, rows, Hkv, -1, dh).permute(0, 2, 1, 3, 4).reshape(R, Hkv, -1, dh)
    Z = (q @ K.transpose(2, 3)).mul_(dh ** -0.5).view(R, Hkv, rows, -1, place.shape[1])
    del K
    Z.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = Z.amax(-1, keepdim=True)
    Z = torch.exp_(Z.sub_(torch.where(top == -math.inf, 0.0, top)))
    V = _token_values(s, page, tok, True).transpose(1, 2)
    total = Z.sum(-1, keepdim=True)
    O = (Z.flatten(2, 3) @ V).view(R, Hkv, rows, -1, dh) / torch.where(total > 0, total, 1.0)
    O = O.permute(0, 2, 1, 3, 4).reshape(R, rows, -1, dh).to(torch.bfloat16)
    return O, None if n is None else far <= n[:, None]


def _window(s):
    c = s["case"]
    R, n = c["R"], c["n"]
    if c["form"] == "packed":
        at = 0
        for r, k in enumerate(s["count"]):
            for i in range(0, k, 256):
                j = min(k, i + 256)
                s["O"][at + i:at + j] = _window_rows(s, s["Q"][None, at + i:at + j], slice(r, r + 1), i)[0][0]
            at += k
        return [s["O"]]
    step = n if c["form"] != "chain" else max(1, min(n, 512 // max(1, R // 2)))
    for i in range(0, n, step):
        j = min(n, i + step)
        O, row = _window_rows(s, s["Q"][:, i:j], slice(0, R), i, s.get("mask"))
        if row is None:
            s["O"][:, i:j] = O
        else:
            s["O"][:, i:j] = torch.where(row[:, :, None, None], O, s["O"][:, i:j])
    return [s["O"]]


def _plan(s):
    c = s["case"]
    P, W, S, T = c["P"], c["window"], c["sinks"], s["T"]
    table, refs, lens, count = s["table"], s["refs"], s["lens"], s["count"].long()
    R, width = table.shape
    slot = torch.arange(width, device=DEV)[None]
    f = lens.long()
    # pages behind the lengths go back, then those that the window has left behind
    gone = (slot >= ((f + P - 1) // P)[:, None]) & (table >= 0)
    if W:
        gone |= (table >= 0) & (slot * P >= S) & (slot * P + P - 1 <= (f - W)[:, None])
    refs -= torch.bincount(torch.where(gone, table, refs.numel()).view(-1), minlength=refs.numel() + 1)[:-1].int()
    table.masked_fill_(gone, -1)
    upto = torch.cumsum(count, 0)
    valid = (lens >= 0) & (count >= 0) & ((upto <= T) | (count == 0))
    have = torch.where(valid, count, 0)
    end = torch.cumsum(have, 0)
    start = torch.cat([torch.zeros(1, device=DEV, dtype=torch.long), end])
    # the lowest free pages, in the rows' order
    need = (slot >= (f // P)[:, None]) & (slot < ((f + have + P - 1) // P)[:, None])
    held = need & (table >= 0)
    bad = ~valid | ((f + have + P - 1) // P > width) | (held & (refs[table.clamp(min=0).long()] > 1)).any(1)
    lack = need & (table < 0) & ~bad[:, None]
    want = lack.sum(1)
    taken = torch.cumsum(want, 0)
    ok = ~bad & ((want == 0) | (taken <= (refs == 0).sum()))
    free = torch.argsort(refs != 0, stable=True)
    at = (taken - want)[:, None] + torch.cumsum(lack, 1) - 1
    lack &= ok[:, None]
    page = free[at.clamp(0, refs.numel() - 1)].int()
    table[:] = torch.where(lack, page, table)
    refs += torch.bincount(torch.where(lack, page, refs.numel()).view(-1), minlength=refs.numel() + 1)[:-1].int()
    t = torch.arange(T, device=DEV)
    row = torch.searchsorted(end, t, right=True)
    inside = row < R
    r = row.clamp(max=R - 1)
    pos = f[r] + t - start[r]
    where = table[r, (pos // P).clamp(0, width - 1)].long() * P + pos % P
    return [ok.int(), start.int(), torch.where(inside, row, -1).int(), torch.where(inside, pos, -1).int(),
            torch.where(inside & ok[r], where, -1).int(), table, refs]


def _quantised(x):
    """The values that [..., dh] has in 4 bits: e4m3 scales of 16 dimensions, e2m1 codes, ties to even."""
    y = x.float().unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    a = y.abs() / torch.where(scale > 0, scale, 1.0)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    up = torch.bucketize(a, mid, right=False)                # the code below a tie ...
    odd_tie = (a == mid[up.clamp(max=6)]) & (up % 2 == 1)    # ... or the even one above it
    code = torch.tensor(E2M1, device=x.device)[up + odd_tie]
    return (torch.copysign(code, y) * scale).flatten(-2).to(torch.bfloat16)


def _padded(s, x):
    """Packed rows as [R, most], zeros behind a request's."""
    i = torch.arange(s["most"], device=DEV)[None]
    at = (s["start"][:-1, None].long() + i).clamp(max=x.shape[0] - 1)
    return torch.where((i < s["count"][:, None])[:, :, None, None], x[at], 0.0)


def _put(s):
    return [_padded(s, _quantised(s["K"])), _padded(s, _quantised(s["V"]))]


def _target(s, x):
    """The target's probabilities of logits [R, V], in 64 bits."""
    T, k, p, m = (s[name][:, None] for name in ("temperature", "top_k", "top_p", "min_p"))
    V = x.shape[1]
    order = None
    if s["case"]["mix"] != "plain":
        x, order = torch.sort(x, dim=1, descending=True, stable=True)
    x = x.double()
    top = x.amax(1, keepdim=True)
    x = torch.exp_(x.sub_(top).div_(torch.where(T > 0, T.double(), 1.0)))
    if order is not None:
        rank = torch.arange(V, device=DEV)[None]
        x.masked_fill_((rank >= torch.where(T <= 0, 1, torch.where(k > 0, k, V))) | (x < m.double()), 0.0)
        before = torch.cumsum(x, 1).sub_(x)
        total = (before[:, -1] + x[:, -1])[:, None]
        x.masked_fill_((before >= p.double() * total) & (p < 1), 0.0)
        x = torch.zeros_like(x).scatter_(1, order, x)
    return x.div_(x.sum(1, keepdim=True))


def _verify(s):
    c = s["case"]
    R, B, kids, depth = c["R"], c["B"], c["kids"], c["depth"]
    D = s["draft"].shape[1]
    parent, token, u = s["parent"].long(), s["token"].long(), s["u"].double()
    node = torch.arange(B, device=DEV)[None]
    there = node < s["n_out"][:, None]
    each = torch.arange(R, device=DEV)
    cur = torch.zeros(R, dtype=torch.long, device=DEV)
    done = torch.zeros(R, dtype=torch.bool, device=DEV)
    length = torch.zeros(R, dtype=torch.long, device=DEV)
    nodes = torch.full((R, depth), -1, dtype=torch.long, device=DEV)
    bonus, prob = torch.full_like(length, -1), torch.zeros(R, dtype=torch.float64, device=DEV)
    for _ in range(depth + 1):
        p = _target(s, s["logits"][each, cur])
        q = s["draft"][each, cur.clamp(max=D - 1)].double().div_(s["draft_temperature"].double()[:, None])
        q = torch.softmax(q, 1)
        mine = there & (parent == cur[:, None] - 1)
        nth = torch.cumsum(mine, 1)
        rest, A = p, torch.zeros(R, dtype=torch.float64, device=DEV)
        N, Z = torch.ones_like(A), torch.ones_like(A)
        took = torch.full((R,), -1, dtype=torch.long, device=DEV)
        for k in range(1, kids + 1):
            hit = mine & (nth == k)
            i = hit.int().argmax(1)
            x = token[each, i].clamp(min=0)
            qx, px = q[each, x], p[each, x]
            live = hit.any(1) & ~done & (took < 0) & (qx > 0)
            a = N / Z
            yes = live & (u[each, i + 1] * a * qx < px - A * qx)
            took = torch.where(yes, i, took)
            no = live & ~yes
            A, Z = torch.where(no, A + a, A), torch.where(no, Z - qx, Z)
            rest = torch.where(no[:, None], (p - A[:, None] * q).clamp_(min=0.0), rest)
            N = torch.where(no, rest.sum(1), N)
        # rows where no child was accepted end here, with a token of what is left
        end = ~done & (took < 0)
        rest = torch.where((N > 0)[:, None], rest, p)
        upto = torch.cumsum(rest, 1)
        total = upto[:, -1]
        x = (upto <= (u[:, 0] * total)[:, None]).sum(1)
        last = c["V"] - 1 - (rest.flip(1) > 0).int().argmax(1)
        x = torch.minimum(x, last)
        bonus, prob = torch.where(end, x, bonus), torch.where(end, rest[each, x] / total, prob)
        done |= end
        nodes.scatter_(1, length.clamp(max=depth - 1)[:, None],
                       torch.where(took >= 0, took, nodes[each, length.clamp(max=depth - 1)])[:, None])
        length += took >= 0
        cur = torch.where(took >= 0, took + 1, cur)
    return [length.int(), nodes.int(), bonus.int(), prob.float()]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "verify":
        # the rows on the path: a drafted token is accepted about seven times in ten, more often with siblings
        keep = 1 - 0.3 ** c["kids"]
        rows = c["R"] * sum(keep ** i for i in range(min(c["depth"], 6 if c["kids"] > 1 else 99) + 1))
        return {"bytes": rows * 2 * c["V"] * (2 if c["bf16"] else 4), "flops": rows * 4 * c["V"]}
    R = c["R"]
    if c["op"] == "plan" or c["op"] == "put":
        tokens = R * c["n"] * 0.75 + (R / 8) * c["long"] * 0.75
        if c["op"] == "plan":
            return {"bytes": 12 * (R * c["n"] + (R + 7) // 8 * c["long"]) + 20 * R + 16 * tokens / c["P"],
                    "flops": 8 * tokens}
        row = c["Hkv"] * c["dh"]
        return {"bytes": tokens * 2 * (4 * row + 9 * row / 8), "flops": tokens * row * 8}
    n, W, S, Hq, Hkv, dh = (c[k] for k in ("n", "window", "sinks", "Hq", "Hkv", "dh"))
    mean = c["len"] * (0.625 + 0.375 / R)       # the requests' lengths lie between a quarter of the largest and it
    rows = {"token": R, "tree": 0.875 * R * n, "chain": 0.875 * R * n, "packed": R - 1 + n}[c["form"]]
    if c["form"] == "packed":
        keys = (R - 1) * min(W + S, mean + 1) + min(W + S + n, mean + n)
    else:
        keys = R * min(W + S + n, mean + n)
    seen = min(W + S, mean + n / 2)
    return {"bytes": keys * Hkv * dh * 9 / 8 + 4 * rows * Hq * dh, "flops": 4 * rows * Hq * dh * seen}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None                       # whole numbers only
    if c["op"] == "window":
        rows = c["R"] + c["n"] if c["form"] == "packed" else c["R"] * c["n"]
        if 4 * rows * c["Hq"] * c["dh"] * min(c["window"] + c["n"], c["len"] + c["n"]) > 3e12:
            return None
    s = prepare(case, seed)
    if c["op"] == "put":
        K, V = _nearest(s["K"]), _nearest(s["V"])
        out = [torch.zeros(c["R"], s["most"], c["Hkv"], c["dh"], dtype=torch.float64, device=DEV) for _ in range(2)]
        at = s["start"].tolist()
        for r in range(c["R"]):
            for o, x in zip(out, (K, V)):
                o[r, :at[r + 1] - at[r]] = x[at[r]:at[r + 1]]
        return out
    if c["op"] == "verify":
        return [None, None, None, _exact_verify(s)]
    return [_exact_window(s)]


def _nearest(x):
    """4-bit values by search: the nearest scale and the nearest code among all, the even one of two as near."""
    f8 = torch.arange(0, 127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    code = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def near(v, grid):
        hi = torch.searchsorted(grid, v).clamp(1, len(grid) - 1)
        lo = hi - 1
        a, b = v - grid[lo], grid[hi] - v
        return grid[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]

    y = x.double().unflatten(-1, (-1, 16))
    sc = near(y.abs().amax(-1, keepdim=True) / 6, f8)
    v = near((y.abs() / sc.clamp(min=2.0 ** -40)).clamp(max=6.0), code)
    return (v * y.sign() * sc).flatten(-2)


def _exact_window(s):
    c = s["case"]
    n, P, Hkv, dh, W, S, g = (*(c[k] for k in ("n", "P", "Hkv", "dh", "window", "sinks")), c["Hq"] // c["Hkv"])
    code, sc = P * dh // 2, P * dh // 16
    val = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    O = torch.zeros(s["O"].shape, dtype=torch.float64, device=DEV)

    def part(b, at):
        raw = b[:, at:at + code].reshape(-1, dh // 2)                        # [tokens, dh / 2]
        x = torch.stack([val[(raw & 15).int()], val[(raw >> 4).int()]], -1).view(-1, dh // 16, 16)
        e = b[:, at + code:at + code + sc].reshape(-1, dh // 16, 1)
        man, ex = (e & 7).double(), (e >> 3).double()
        return (x * torch.where(ex > 0, (1 + man / 8) * 2 ** (ex - 7), man * 2.0 ** -9)).view(-1, dh)

    first = 0
    for r, rows in enumerate(s["count"]):
        L = int(s["lens"][r])
        depth = np.arange(rows)
        up = np.tril(np.ones((rows, rows), bool))        # row i sees row j
        if c["form"] == "tree":
            words = s["mask"][r].cpu().numpy().view(np.uint32)
            bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:rows - 1, :rows - 1].astype(bool)
            up = np.zeros((rows, rows), bool)
            up[:, 0] = True
            up[1:, 1:] = bits
            depth = np.concatenate([[0], bits.sum(1)])
        # the places that any row sees: the sinks, and from the first row's window on
        place = np.unique(np.concatenate([np.arange(min(S, L + rows)), np.arange(max(0, L - W + 1), L + rows)]))
        at = np.where(place > L, L + depth[np.clip(place - L, 0, rows - 1)], place)
        at, place = torch.from_numpy(at).to(DEV), torch.from_numpy(place).to(DEV)
        slot = s["table"][r].long()[place // P]
        up, far = torch.from_numpy(up).to(DEV), torch.from_numpy(depth).to(DEV)
        for h in range(Hkv):
            b = s["pool"][0].view(-1, Hkv, P * dh * 9 // 8)[:, h]
            held = torch.unique(slot[slot >= 0])
            K, V = part(b[held], 0), part(b[held], code + sc)
            i = torch.searchsorted(held, slot) * P + place % P
            i = i.clamp(max=len(K) - 1)
            K, V = K[i], V[i]
            for a in range(0, rows, 2048):
                e = min(rows, a + 2048)
                use = slice(int(torch.searchsorted(place, max(S, L + a - W + 1))) if c["form"] != "tree" else 0,
                            int(torch.searchsorted(place, L + e)) if c["form"] != "tree" else len(place))
                pick = torch.cat([torch.arange(min(S, use.start), device=DEV), torch.arange(use.start, use.stop, device=DEV)])
                qp = (L + far[a:e])[:, None]
                kp, kl = at[pick][None], place[pick][None]
                see = (kl <= L) | up[a:e].gather(1, (kl - L).clamp(0, rows - 1).expand(e - a, -1))
                see &= (kp < S) | (qp - kp < W)
                q = (s["Q"][first + a:first + e] if c["form"] == "packed" else s["Q"][r, a:e])[:, h * g:(h + 1) * g].double()
                z = torch.einsum("ngd,ld->ngl", q, K[pick]) / math.sqrt(dh)
                w = torch.softmax(z.masked_fill(~see[:, None], -math.inf), -1).nan_to_num(0.0)
                o = torch.einsum("ngl,ld->ngd", w, V[pick])
                if c["form"] == "packed":
                    O[first + a:first + e, h * g:(h + 1) * g] = o
                else:
                    O[r, a:e, h * g:(h + 1) * g] = o
        first += rows
    return O


def _exact_verify(s):
    """The drawn token's probability, request by request: residuals made one after the other, each of the last."""
    c = s["case"]
    out = torch.zeros(c["R"], dtype=torch.float64, device=DEV)
    for r in range(c["R"]):
        parent, token = s["parent"][r].tolist(), s["token"][r].tolist()
        u, n = s["u"][r].tolist(), int(s["n_out"][r])
        T, k, p, m = (float(s[x][r]) for x in ("temperature", "top_k", "top_p", "min_p"))
        row = 0
        while True:
            l = s["logits"][r, row].double()
            if T <= 0:
                t = torch.zeros_like(l)
                t[int(torch.argmax(l))] = 1.0
            else:
                t = torch.softmax(l / T, 0)
                val, idx = torch.sort(t, descending=True, stable=True)
                keep = c["V"] if k <= 0 else min(int(k), c["V"])
                keep = min(keep, int((val >= m * val[0]).sum()))
                mass = torch.cumsum(val[:keep], 0)
                if p < 1:
                    keep = min(keep, int((mass < p * mass[-1]).sum()) + 1)
                t = torch.zeros_like(l)
                t[idx[:keep]] = val[:keep]
                t /= t.sum()
            q, nxt = None, -1
            for i in range(n):
                if parent[i] != row - 1:
                    continue
                if q is None:
                    q = torch.softmax(s["draft"][r, row].double() / float(s["draft_temperature"][r]), 0)
                x = token[i]
                if float(q[x]) <= 0:
                    continue
                if u[i + 1] * float(q[x]) < float(t[x]):
                    nxt = i
                    break
                left = (t - q).clamp(min=0)
                if float(left.sum()) > 0:
                    t = left / left.sum()
                q[x] = 0.0
                q = q / q.sum()
            if nxt < 0:
                upto = torch.cumsum(t, 0)
                j = int((upto <= u[0] * float(upto[-1])).sum())
                j = min(j, int(torch.nonzero(t > 0)[-1]))
                out[r] = t[j] / upto[-1]
                break
            row = nxt + 1
    return out
