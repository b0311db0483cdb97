"""The operators of a verification step over a paged key/value cache in 4 bits, as they are measured:
attention over the cache (single tokens and draft trees), writing and reading it, its page operations, and
sampling the target's tokens.  Each case runs in a plain form (elementary torch operations in 32 bits, 64 where
the decision needs them) or, where ``own`` is true, through the framework's entry points.

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
        # one user's next token, a short conversation: latency
        dict(name="decode_one", op="attention", R=1, B=0, len=1000, Hq=32, Hkv=8, dh=128, P=64),
        # next tokens of a busy server, conversations of many lengths
        dict(name="decode_batch", op="attention", R=64, B=0, len=16001, Hq=32, Hkv=8, dh=128, P=64),
        # one user with a long document
        dict(name="decode_long", op="attention", R=1, B=0, len=131072, Hq=32, Hkv=8, dh=128, P=64),
        # the verification of one draft tree (the default build's budget)
        dict(name="tree_one", op="attention", R=1, B=128, len=4099, Hq=32, Hkv=8, dh=128, P=64),
        # the verification of a batch of trees (the batch build's requests and budget), small pages
        dict(name="tree_batch", op="attention", R=32, B=64, len=2500, Hq=32, Hkv=8, dh=128, P=16),
        # the keys and values of one step's trees into the cache, and back
        dict(name="write_step", op="write", R=8, n=129, len=1000, Hkv=8, dh=128, P=64),
        # a prompt's keys and values into the cache, and back
        dict(name="write_prompt", op="write", R=2, n=16000, len=0, Hkv=8, dh=128, P=64),
        # one request's accepted path moves to the end of its prefix, pages for the next tree
        dict(name="commit_one", op="commit", R=1, B=128, len=1000, layers=32, accept=7, Hkv=8, dh=128, P=64),
        # the same for a batch
        dict(name="commit_batch", op="commit", R=32, B=64, len=500, layers=32, accept=6, Hkv=8, dh=128, P=64),
        # requests continued in several ways: their last pages are copied, the others shared
        dict(name="fork_batch", op="fork", R=8, ways=4, len=700, layers=32, Hkv=8, dh=128, P=64),
        # the target's tokens of one tree (the smallest build's vocabulary and budget)
        dict(name="sample_small", op="sample", R=1, n=17, V=32000, bf16=False, mix="nucleus"),
        # the target's tokens of a batch of trees, requests with settings of their own
        dict(name="sample_batch", op="sample", R=16, n=129, V=151936, bf16=True, mix="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "tree", "tree", "write", "commit", "fork", "sample", "sample"])
    dh, P = rng.choice([128, 128, 64]), rng.choice([16, 32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "decode":
        R, g = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        return dict(op="attention", R=R, B=0, len=_log(rng, 1, min(100000, 700000 // R)), Hq=Hkv * g, Hkv=Hkv, dh=dh, P=P)
    if op == "tree":
        R, g, B = _log(rng, 1, 32), rng.choice([1, 2, 4, 8]), _log(rng, 1, 256)
        most = max(2, min(16000, 32 * 65 * 4 * 2500 // (R * (B + 1) * g)))
        return dict(op="attention", R=R, B=B, len=_log(rng, 1, most), Hq=Hkv * g, Hkv=Hkv, dh=dh, P=P)
    if op == "write":
        R = _log(rng, 1, 32)
        return dict(op="write", R=R, n=_log(rng, 1, 24000 // R), len=_log(rng, 1, 2000) - 1, Hkv=Hkv, dh=dh, P=P)
    if op == "commit":
        B = _log(rng, 1, 256)
        return dict(op="commit", R=_log(rng, 1, 32), B=B, len=_log(rng, 1, 500), layers=rng.randint(1, 32),
                    accept=rng.randint(0, min(B, 16)), Hkv=Hkv, dh=dh, P=P)
    if op == "fork":
        return dict(op="fork", R=_log(rng, 1, 8), ways=rng.randint(1, 4), len=_log(rng, 1, 700),
                    layers=rng.randint(1, 32), Hkv=Hkv, dh=dh, P=P)
    V = _log(rng, 500, 152000)
    R = _log(rng, 1, 16)
    return dict(op="sample", R=R, n=_log(rng, 1, 129), V=V, bf16=rng.random() < 0.5,
                mix=rng.choice(["mixed", "nucleus", "topk", "full"]))


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


def _pool(g, layers, pages, Hkv, dh, P):
    """Pages as quantised data fills them: [layers, pages, Hkv * P * dh * 9 / 8] bytes."""
    lut = _nibble_pairs(g)
    chunk = P * dh * 9 // 8
    pool = torch.empty(layers, pages, Hkv, chunk, dtype=torch.uint8, device=DEV)
    half = chunk // 2
    code = P * dh // 2
    for at in (0, half):
        i = torch.randint(0, 65536, (layers, pages, Hkv, code), generator=g, device=DEV, dtype=torch.int32)
        pool[..., at:at + code] = lut[i]
        s = torch.randint(0x21, 0x2C, (layers, pages, Hkv, half - code), generator=g, device=DEV, dtype=torch.uint8)
        pool[..., at + code:at + half] = s           # scales 0.14 .. 0.34
    return pool.view(layers, pages, Hkv * chunk)


def _lens(rs, R, most):
    n = rs.randint(max(0, most // 4), most + 1, R)
    n[0] = most
    return n


def _trees(rs, R, B):
    """Random trees in canonical order: the nodes' numbers, the parents (rank or -1) and the ancestor masks."""
    n = rs.randint(max(1, (3 * B) // 4), B + 1, R) if B else np.zeros(R, np.int64)
    if B:
        n[0] = B
    parent = np.full((R, max(B, 1)), -1)
    anc = np.zeros((R, max(B, 1), max(B, 1)), bool)
    for i in range(B):
        parent[:, i] = (rs.random_sample(R) * (i + 1)).astype(np.int64) - 1
        up = np.where(parent[:, i, None] >= 0, anc[np.arange(R), np.maximum(parent[:, i], 0)], False)
        anc[:, i] = up
        anc[:, i, i] = True
        anc[i >= n, i] = False
    words = max(1, (B + 31) // 32)
    bits = np.zeros((R, max(B, 1), words * 32), np.uint64)
    bits[:, :, :anc.shape[2]] = anc
    mask = (bits.reshape(R, -1, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return n, parent, torch.from_numpy(mask.view(np.int32)).to(DEV)


def _table(rs, held, pages, width):
    """Page tables whose row r holds held[r] pages, in no order, and the counts of the pages' holders."""
    ids = rs.permutation(pages)
    table = np.full((len(held), width), -1, np.int32)
    at = 0
    for r, k in enumerate(held):
        table[r, :k] = ids[at:at + k]
        at += k
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    return torch.from_numpy(table).to(DEV), torch.from_numpy(refs).to(DEV)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def prepare(case, seed):
    c = case
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 32))
    s = dict(case=c)
    if c["op"] == "sample":
        return _prepare_sample(c, g, rs, s)
    R, P, Hkv, dh = c["R"], c["P"], c["Hkv"], c["dh"]
    lens = _lens(rs, R, c["len"])
    layers, spare = c.get("layers", 1), 0
    if c["op"] == "attention":
        n, _, mask = _trees(rs, R, c["B"])
        held = -(-(lens + c["B"]) // P)
        width = int(held.max()) + 1
        s.update(mask=mask, n_nodes=_int(n), max_len=c["len"] + c["B"],
                 Q=torch.randn(R, c["B"] + 1, c["Hq"], dh, generator=g, device=DEV).to(torch.bfloat16),
                 O=torch.zeros(R, c["B"] + 1, c["Hq"], dh, dtype=torch.bfloat16, device=DEV))
    elif c["op"] == "write":
        held = -(-(lens + c["n"]) // P)
        width = int(held.max())
        mag = torch.exp(torch.randn(2, 1, 1, Hkv, dh, generator=g, device=DEV) * 0.5)    # channels differ in size
        x = torch.randn(2, R, c["n"], Hkv, dh, generator=g, device=DEV)
        x.mul_(mag)
        s.update(K=x[0].to(torch.bfloat16), V=x[1].to(torch.bfloat16))
    elif c["op"] == "commit":
        B = c["B"]
        n, parent, _ = _trees(rs, R, B)
        L = max(1, c["accept"])
        nodes = np.full((R, L), -1)
        length = np.zeros(R, np.int64)
        for r in range(R):          # a path of rising ranks
            k = min(int(rs.randint(c["accept"] // 2, c["accept"] + 1)), int(n[r]))
            nodes[r, :k] = np.sort(rs.choice(int(n[r]), k, replace=False))
            length[r] = k
        held = -(-(lens + B) // P)
        width = int(held.max()) + 2
        spare = R * (-(-B // P) + 2)
        s.update(nodes=_int(nodes), length=_int(length), rows=_int(np.arange(R)), keep=_int(lens),
                 want=_int(np.full(R, B)), B=B)
    else:
        ways = c["ways"]
        held = np.concatenate([-(-lens // P), np.zeros(R * ways, np.int64)])
        lens = np.concatenate([lens, np.zeros(R * ways, np.int64)])
        width = max(1, int(held.max()))
        spare = R * ways + 8
        s.update(src=_int(np.repeat(np.arange(R), ways)), dst=_int(R + np.arange(R * ways)),
                 none=_int(np.zeros(R * ways)))
    pages = R * -(-(c["len"] + c.get("B", c.get("n", 0))) // P) + spare + 1      # enough for every seed's lengths
    table, refs = _table(rs, held, pages, width)
    s.update(pool=_pool(g, layers, pages, Hkv, dh, P), table=table, refs=refs, lens=_int(lens))
    if own:
        from speculative_decoding_draft_06_gb300 import dartree
        s["cache"] = dartree.KVCache(layers, pages, page_tokens=P, Hkv=Hkv, dh=dh, pool=s["pool"], refs=refs)
    return s


def _prepare_sample(c, g, rs, s):
    R, n, V = c["R"], c["n"], c["V"]
    zipf = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
    logits = torch.empty(R, n, V, dtype=torch.bfloat16 if c["bf16"] else torch.float32, device=DEV)
    for r in range(R):
        x = torch.randn(n, V, generator=g, device=DEV) * 2.0
        x += 20.0 + zipf[torch.randperm(V, generator=g, device=DEV)]
        if r % 8 == 5:              # a grammar allows few tokens
            x.masked_fill_((torch.rand(V, generator=g, device=DEV) > 0.002)[None], -math.inf)
        logits[r] = x
    logits[:, :, V - V // 500:] = -math.inf      # rows of the projection that stand for no token
    T, k, p, m = np.full(R, 0.8), np.zeros(R), np.full(R, 0.95), np.zeros(R)
    if c["mix"] == "topk":
        T, k = np.full(R, 0.6), np.full(R, 20)
    elif c["mix"] == "full":
        T, p = np.full(R, 1.0), np.full(R, 1.0)
    elif c["mix"] == "mixed":
        T, k = rs.choice([0.0, 0.6, 0.7, 1.0, 1.3], R), rs.choice([0, 0, 20, 50, 1000], R)
        p, m = rs.choice([0.8, 0.9, 0.95, 1.0], R), rs.choice([0.0, 0.0, 0.05], R)
        if R * n >= 16:
            logits[R - 1, n - 1] = -math.inf     # a row with nothing left to choose from
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV)  # noqa: E731
    s.update(logits=logits.view(R * n, V), u=torch.rand(R * n, generator=g, device=DEV), temperature=f(T),
             top_k=_int(k), top_p=f(p), min_p=f(m))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        from speculative_decoding_draft_06_gb300 import dartree
        c = s["case"]
        if op == "sample":
            out = dartree.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                 top_p=s["top_p"], min_p=s["min_p"], rows_per_req=c["n"])
            return [out["token"], out["prob"]]
        cache, table, lens = s["cache"], s["table"], s["lens"]
        if op == "attention":
            return [cache.attention(0, s["Q"], table, lens, mask=s["mask"] if c["B"] else None,
                                    n_nodes=s["n_nodes"], max_len=s["max_len"], out=s["O"])]
        if op == "write":
            cache.append(0, s["K"], s["V"], table, lens)
            return list(cache.read(0, table, lens, c["n"]))
        if op == "commit":
            cache.release(table, lens, s["rows"], s["keep"])
            ok = cache.reserve(table, lens, s["want"])
            cache.commit(table, lens, s["nodes"], s["length"], extra=1)
            return [ok, table, lens, s["refs"], s["pool"]]
        cache.release(table, lens, s["dst"], s["none"])
        ok = cache.fork(table, lens, s["src"], s["dst"])
        return [ok, table, lens, s["refs"], s["pool"]]
    return {"sample": _sample, "attention": _attention, "write": _write, "commit": _commit, "fork": _fork}[op](s)


# ------------------------------------------------------------------ plain forms
def _values(chunk, P, dh, second):
    """The fp32 values [..., P, dh] of the keys (or values) in chunks [..., P * dh * 9 / 8]."""
    at, code = (chunk.shape[-1] // 2 if second else 0), P * dh // 2
    byte = chunk[..., at:at + code].reshape(*chunk.shape[:-1], P, dh // 16, 8)
    scale = chunk[..., at + code:at + code + P * dh // 16].contiguous().view(torch.float8_e4m3fn).float()
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=chunk.device)
    two = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)              # byte -> both values
    x = two[byte.int()].view(*byte.shape[:-1], 16)
    return (x * scale.view(*byte.shape[:-1], 1)).view(*chunk.shape[:-1], P, dh)


def _attention(s):
    c = s["case"]
    R, B, Hq, Hkv, dh, P = (c[k] for k in ("R", "B", "Hq", "Hkv", "dh", "P"))
    np_ = -(-s["max_len"] // P)
    page = s["table"][:, :np_]
    got = s["pool"][0].view(-1, Hkv, P * dh * 9 // 8)[page.clamp(min=0).long()]         # [R, pages, Hkv, chunk]
    K = _values(got, P, dh, False).transpose(1, 2).reshape(R, Hkv, np_ * P, dh)
    j = torch.arange(np_ * P, device=DEV)
    lens, n = s["lens"].long()[:, None], s["n_nodes"].long()[:, None]
    seen = (j < lens)[:, None].repeat(1, B + 1, 1)                                       # [R, B+1, L]
    if B:
        node = (j - lens).clamp(0, B - 1)                                                # [R, L]
        bit = (s["mask"].long().gather(2, (node >> 5)[:, None].expand(R, B, -1)) >> (node & 31)[:, None]) & 1
        seen[:, 1:] |= (bit == 1) & ((j >= lens) & (j < lens + n))[:, None]
    Q = s["Q"].float().view(R, B + 1, Hkv, Hq // Hkv, dh).permute(0, 2, 1, 3, 4).reshape(R, Hkv, -1, dh)
    S = (Q @ K.transpose(2, 3)).mul_(dh ** -0.5).view(R, Hkv, B + 1, Hq // Hkv, -1)
    S.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = S.amax(-1, keepdim=True)
    W = torch.exp(S - torch.where(top == -math.inf, 0.0, top))
    del S, K
    V = _values(got, P, dh, True).transpose(1, 2).reshape(R, Hkv, np_ * P, dh)
    total = W.sum(-1, keepdim=True)
    O = (W.view(R, Hkv, -1, np_ * P) @ V).view(R, Hkv, B + 1, Hq // Hkv, dh) / torch.where(total > 0, total, 1.0)
    O = O.permute(0, 2, 1, 3, 4).reshape(R, B + 1, Hq, dh).to(torch.bfloat16)
    row = torch.arange(B + 1, device=DEV)[None] <= n
    s["O"][row] = O[row]
    return [s["O"]]


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


def _write(s):
    return [_quantised(s["K"]), _quantised(s["V"])]


def _drop(s, rows, keep):
    """Pages beyond keep tokens of the rows go back."""
    P, table, refs, lens = s["case"]["P"], s["table"], s["refs"], s["lens"]
    rows = rows.long()
    mine = table[rows]
    gone = (torch.arange(table.shape[1], device=DEV) >= ((keep + P - 1) // P)[:, None]) & (mine >= 0)
    refs -= torch.bincount(torch.where(gone, mine, refs.numel()).view(-1), minlength=refs.numel() + 1)[:-1].int()
    table[rows] = torch.where(gone, -1, mine)
    lens[rows] = torch.minimum(lens[rows], keep)


def _take(refs, need):
    """Which of the needs are met, in order, and the pages [len(need), most] that each gets (lowest first)."""
    upto = torch.cumsum(need, 0)
    free = torch.argsort(refs != 0, stable=True)
    ok = (need == 0) | (upto <= (refs == 0).sum())
    return ok, free, upto - need


def _commit(s):
    c = s["case"]
    P, table, refs, lens = c["P"], s["table"], s["refs"], s["lens"]
    _drop(s, s["rows"], s["keep"])
    slot = torch.arange(table.shape[1], device=DEV)
    wanted = -(-(lens + s["want"]) // P)
    lack = (slot < wanted[:, None]) & (table < 0)
    ok, free, first = _take(refs, lack.sum(1))
    at = first[:, None] + torch.cumsum(lack, 1) - 1
    page = free[at.clamp(0, refs.numel() - 1)].int()
    lack &= ok[:, None]
    table[:] = torch.where(lack, page, table)
    refs += torch.bincount(torch.where(lack, page, refs.numel()).view(-1), minlength=refs.numel() + 1)[:-1].int()
    # the accepted tokens, all layers at once
    chunk = P * c["dh"] * 9 // 8
    pool = s["pool"].view(c["layers"], -1, c["Hkv"], chunk)
    k = torch.arange(s["nodes"].shape[1], device=DEV)
    live = k < s["length"][:, None]
    r = torch.arange(len(lens), device=DEV)[:, None].expand(live.shape)[live]
    src, dst = (lens[:, None] + s["nodes"])[live].long(), (lens[:, None] + k)[live].long()
    code, sc = P * c["dh"] // 2, P * c["dh"] // 16
    edge = [0, code, code + sc, 2 * code + sc, 2 * (code + sc)]
    for a, b in zip(edge, edge[1:]):
        part = pool[..., a:b].unflatten(-1, (P, -1))                        # [layers, pages, Hkv, P, bytes]
        part[:, table[r, dst // P].long(), :, dst % P] = part[:, table[r, src // P].long(), :, src % P]
    lens += s["length"] + 1
    return [ok.int(), table, lens, refs, s["pool"]]


def _fork(s):
    P, table, refs, lens = s["case"]["P"], s["table"], s["refs"], s["lens"]
    _drop(s, s["dst"], s["none"])
    src, dst = s["src"].long(), s["dst"].long()
    whole, rest = lens[src] // P, (lens[src] % P != 0).int()
    ok, free, first = _take(refs, rest)
    slot = torch.arange(table.shape[1], device=DEV)[None]
    share = (slot < whole[:, None]) & ok[:, None]
    mine = torch.where(share, table[src], -1)
    refs += torch.bincount(torch.where(share, mine, refs.numel()).view(-1), minlength=refs.numel() + 1)[:-1].int()
    part = ok & (rest == 1)
    page = free[first[part]]
    refs[page] = 1
    s["pool"][:, page] = s["pool"][:, table[src[part], whole[part].long()].long()]
    mine[part] = torch.where(slot == whole[part][:, None], page[:, None].int(), mine[part])
    table[dst[ok]] = mine[ok]
    lens[dst[ok]] = lens[src[ok]]
    return [ok.int(), table, lens, refs, s["pool"]]


def _sample(s):
    rows, V = s["logits"].shape
    per = lambda t: t.repeat_interleave(rows // t.numel())[:, None]  # noqa: E731
    T, k, p, m = (per(s[x]) for x in ("temperature", "top_k", "top_p", "min_p"))
    x, order = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    x = x.double()
    top = x[:, :1].clone()
    greedy = T <= 0
    x.sub_(torch.where(top == -math.inf, 0.0, top)).div_(torch.where(greedy, 1.0, T.double())).exp_()   # the weights
    rank = torch.arange(V, device=DEV)[None]
    x.masked_fill_((rank >= torch.where(greedy, 1, torch.where(k > 0, k, V))) | (x < m.double()), 0.0)
    before = torch.cumsum(x, 1).sub_(x)
    total = (before[:, -1] + x[:, -1])[:, None]
    x.masked_fill_((before >= p.double() * total) & (p < 1), 0.0)
    del before
    w = torch.zeros_like(x).scatter_(1, order, x)
    del x, order
    upto = torch.cumsum(w, 1)
    total = upto[:, -1:]
    token = (upto <= s["u"].double()[:, None] * total).sum(1).clamp(max=V - 1)
    prob = w.gather(1, token[:, None])[:, 0] / torch.where(total > 0, total, 1.0)[:, 0]
    none = top[:, 0] == -math.inf
    return [torch.where(none, -1, token).int(), torch.where(none, 0.0, prob).float()]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "sample":
        n = c["R"] * c["n"]
        return {"bytes": n * (c["V"] * (2 if c["bf16"] else 4) + 12), "flops": 2 * n * c["V"]}
    R, Hkv, dh, P = c["R"], c["Hkv"], c["dh"], c["P"]
    token = Hkv * dh * 9 // 8
    mean = c["len"] * (0.625 + 0.375 / R)       # the requests' lengths lie between a quarter of the largest and it
    if c["op"] == "attention":
        B = c["B"]
        io = 4 * R * (B + 1) * c["Hq"] * dh
        return {"bytes": R * (mean + 0.875 * B) * token + io, "flops": 4 * R * (B + 1) * c["Hq"] * dh * mean}
    if c["op"] == "write":
        return {"bytes": R * c["n"] * 2 * (token + 4 * Hkv * dh), "flops": R * c["n"] * Hkv * dh * 8}
    if c["op"] == "commit":
        return {"bytes": 2 * c["layers"] * R * 0.75 * c["accept"] * token + 8 * R * 8, "flops": R}
    n = R * c["ways"]
    return {"bytes": 2 * c["layers"] * n * P * token + 8 * n * (mean // P + 1), "flops": n}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("commit", "fork"):
        return None                       # whole numbers only
    s = prepare(case, seed)
    if op == "write":
        return [_nearest(s["K"]), _nearest(s["V"])]
    if op == "sample":
        return _exact_sample(s) if s["logits"].numel() <= 400_000_000 else None
    return [_exact_attention(s)]


def _nearest(x):
    """4-bit values by search: the nearest scale and the nearest code among all, the even one of two as near."""
    f8 = torch.arange(0, 127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    code = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def near(v, grid):
        hi = torch.searchsorted(grid, v).clamp(1, len(grid) - 1)
        lo = hi - 1
        a, b = v - grid[lo], grid[hi] - v
        return grid[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]

    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for r in range(x.shape[0]):
        y = x[r].double().unflatten(-1, (-1, 16))
        sc = near(y.abs().amax(-1, keepdim=True) / 6, f8)
        v = near((y.abs() / sc.clamp(min=2.0 ** -40)).clamp(max=6.0), code)
        out[r] = (v * y.sign() * sc).flatten(-2)
    return out


def _exact_attention(s):
    c = s["case"]
    B, Hkv, dh, P, g = c["B"], c["Hkv"], c["dh"], c["P"], c["Hq"] // c["Hkv"]
    code, sc = P * dh // 2, P * dh // 16
    val = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    O = torch.zeros(s["O"].shape, dtype=torch.float64, device=DEV)

    def part(b, at):
        raw = b[:, at:at + code].reshape(-1, dh // 2)                        # [tokens, dh / 2]
        x = torch.stack([val[(raw & 15).int()], val[(raw >> 4).int()]], -1).view(-1, dh // 16, 16)
        e = b[:, at + code:at + code + sc].reshape(-1, dh // 16, 1)
        man, ex = (e & 7).double(), (e >> 3).double()
        return (x * torch.where(ex > 0, (1 + man / 8) * 2 ** (ex - 7), man * 2.0 ** -9)).view(-1, dh)

    for r in range(c["R"]):
        L, n = int(s["lens"][r]), int(s["n_nodes"][r])
        page = s["table"][r, :-(-(L + n) // P)].long()
        words = s["mask"][r].cpu().numpy().view(np.uint32)
        see = torch.zeros(n + 1, L + n, dtype=torch.bool, device=DEV)
        see[:, :L] = True
        if n:
            bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")
            see[1:, L:] = torch.from_numpy(bits[:n, :n].astype(bool)).to(DEV)
        for h in range(Hkv):
            b = s["pool"][0, page].view(len(page), Hkv, -1)[:, h]
            K, V = part(b, 0)[:L + n], part(b, code + sc)[:L + n]
            q = s["Q"][r, :n + 1, h * g:(h + 1) * g].double()
            z = torch.einsum("ngd,ld->ngl", q, K) / math.sqrt(dh)
            w = torch.softmax(z.masked_fill(~see[:, None], -math.inf), -1).nan_to_num(0.0)
            O[r, :n + 1, h * g:(h + 1) * g] = torch.einsum("ngl,ld->ngd", w, V)
    return O


def _exact_sample(s):
    """The probability of the drawn token, row by row, from the sorted weights' definition; tokens are whole numbers."""
    rows, V = s["logits"].shape
    per = rows // s["temperature"].numel()
    prob = torch.zeros(rows, dtype=torch.float64, device=DEV)
    for i in range(rows):
        r = i // per
        l = s["logits"][i].double()
        T, k, p, m = (float(s[x][r]) for x in ("temperature", "top_k", "top_p", "min_p"))
        if float(l.max()) == -math.inf:
            continue
        if T <= 0:
            prob[i] = 1.0
            continue
        q = torch.softmax(l / T, 0)
        val, idx = torch.sort(q, descending=True, stable=True)
        n = V if k <= 0 else min(int(k), V)
        n = min(n, int((val >= m * val[0]).sum()))
        mass = torch.cumsum(val[:n], 0)
        if p < 1:
            n = min(n, int((mass < p * mass[-1]).sum()) + 1)
        kept = torch.sort(idx[:n]).values
        pick = torch.cumsum(q[kept], 0)
        j = int((pick <= float(s["u"][i]) * pick[-1]).sum())
        prob[i] = q[kept[min(j, n - 1)]] / pick[-1]
    return [None, prob]
