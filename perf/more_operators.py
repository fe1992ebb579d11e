"""Cases of the operators of one speculative decoding step, for timing.

A small model drafts a tree of tokens for each request; the large one checks
the whole tree at once.  Row 0 of a request is the last token that is certain,
the rows after it are drafted tokens, each with the row of its parent (a
smaller one; -1 for row 0).  Three operators, in the order of a step:

* ``attend``  -- attention of the rows over the paged cache: a row sees every
  key before the draft, its own and its ancestors' (16-bit, E4M3 and 4-bit
  caches);
* ``verify``  -- which drafted tokens stand, from the large model's
  probabilities and given random numbers, and the token that follows them;
* ``compact`` -- the keys and values of the rows that stand, moved together at
  the end of the context, in every layer's cache.

``run`` computes a case in plain torch operations, or, with ``own`` set, by
the package's operators.
"""
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
K_SCALE, V_SCALE = 0.0021, 0.0017       # 4-bit cache
K_SCALE8, V_SCALE8 = 0.02, 0.013        # E4M3 cache
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------- cases

def _attend(name, batch, nodes, keys, hq, hkv, d, **kw):
    c = dict(name=name, op="attend", batch=batch, n_lo=nodes[0],
             n_hi=nodes[1], k_lo=keys[0], k_hi=keys[1], hq=hq, hkv=hkv, d=d,
             bs=16, reach=4, window=-1, softcap=0.0, dtype="bf16",
             cache="auto", lens=319)
    c.update(kw)
    return c


def _verify(name, batch, nodes, vocab, **kw):
    c = dict(name=name, op="verify", batch=batch, n_lo=nodes[0],
             n_hi=nodes[1], vocab=vocab, reach=1, sampled=True, sharp=3.0,
             dtype="f32", lens=319)
    c.update(kw)
    return c


def _compact(name, batch, nodes, keys, layers, hkv, d, **kw):
    c = dict(name=name, op="compact", batch=batch, n_lo=nodes[0],
             n_hi=nodes[1], k_lo=keys[0], k_hi=keys[1], layers=layers,
             hkv=hkv, d=d, bs=16, dtype="bf16", lens=319)
    c.update(kw)
    return c


def listed():
    return [
        # two short chats on a small model: latency-bound
        _attend("attend tiny", 2, (7, 7), (37, 50), 4, 2, 64, lens=318),
        # one user with a long conversation and a large tree
        _attend("attend single", 1, (61, 61), (16384, 16384), 32, 8, 128,
                reach=16, lens=322),
        # a batch of 64 chats with small trees
        _attend("attend batch", 64, (16, 16), (512, 4096), 32, 8, 128),
        # a few long documents with large trees: the matrix products count
        _attend("attend wide", 4, (64, 64), (65536, 65536), 64, 8, 128,
                bs=64, reach=16, lens=320),
        # sliding window and soft-cap, chains of drafted tokens
        _attend("attend window", 124, (2, 8), (1024, 16384), 16, 8, 256,
                bs=32, window=4095, softcap=50.0, reach=1, dtype="f16",
                lens=321),
        # an E4M3 cache
        _attend("attend fp8", 48, (12, 12), (512, 8192), 32, 8, 128,
                cache="fp8"),
        # one user, four drafted tokens of a look-up (the draft has no
        # probabilities of its own)
        _verify("verify single", 1, (5, 5), 32001, sampled=False),
        # a batch with chains sampled from a draft model
        _verify("verify chains", 64, (5, 5), 131072),
        # a batch with trees of the draft's most likely tokens
        _verify("verify trees", 48, (16, 16), 131072, reach=4,
                sampled=False),
        # trees sampled from a draft model, 16-bit probabilities of an odd
        # vocabulary
        _verify("verify sampled trees", 24, (9, 24), 100003, reach=4,
                dtype="bf16"),
        # one user, two layers: latency-bound
        _compact("compact single", 1, (7, 7), (37, 50), 2, 2, 64),
        # a batch after a step of trees, every layer's cache
        _compact("compact batch", 64, (24, 32), (16, 64), 16, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng: random.Random):
    op = rng.choice(["attend", "attend", "attend", "verify", "verify",
                     "compact"])
    hkv = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128, 256])
    bs = rng.choice([16, 32, 48, 64, 128])
    lens = rng.randint(0, 1 << 20)
    if op == "verify":
        n_hi = rng.choice([1, rng.randint(2, 6), _log(rng, 7, 64)])
        vocab = _log(rng, 1000, 160000)
        sampled = rng.random() < 0.5
        rows = 60_000_000 // vocab // (2 if sampled else 1)
        return _verify("", max(1, min(_log(rng, 1, 128), rows // n_hi)),
                       (max(1, n_hi // 3), n_hi), vocab,
                       reach=rng.choice([1, 2, 4, 8]), sampled=sampled,
                       sharp=rng.choice([1.0, 3.0, 5.0]),
                       dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                       lens=lens)
    n_hi = rng.choice([rng.randint(1, 8), _log(rng, 9, 100)])
    nodes = (max(1, n_hi // 3), n_hi)
    dtype = rng.choice(["bf16", "f16"])
    if op == "compact":
        batch = _log(rng, 1, 64)
        layers = _log(rng, 1, max(1, min(40, 120_000 // (batch * hkv *
                                                         d // 64 * 5))))
        return _compact("", batch, nodes, (1, rng.randint(2, 64)), layers,
                        hkv, d, bs=bs, dtype=dtype, lens=lens)
    g = rng.choice([1, 2, 3, 4, 8])
    batch = _log(rng, 1, 128)
    top = 800_000_000 // (batch * n_hi * g * hkv)
    k_hi = _log(rng, 16, max(32, min(100_000, top, 2_000_000 // batch)))
    return _attend("", batch, nodes, (max(1, k_hi // 8), k_hi), g * hkv, hkv,
                   d, bs=bs, reach=rng.choice([1, 2, 4, 16]),
                   window=rng.choice([-1, -1, rng.randint(1, 5000)]),
                   softcap=rng.choice([0.0, 0.0, 30.0]), dtype=dtype,
                   cache=rng.choice(["auto", "auto", "fp8", "fp4"]),
                   lens=lens)


def _lengths(case):
    """Rows of each request and keys before the draft, from the case alone."""
    r = np.random.default_rng([case["lens"], 2])
    n = r.integers(case["n_lo"], case["n_hi"], size=case["batch"],
                   endpoint=True)
    if case["op"] == "verify":
        return n, None
    return n, r.integers(case["k_lo"], case["k_hi"], size=case["batch"],
                         endpoint=True)


def work(case):
    n, ctx = _lengths(case)
    t = int(n.sum())
    if case["op"] == "verify":
        # the row of the last token that stands, and what it was drafted from
        e = 4 if case["dtype"] == "f32" else 2
        rows = case["batch"] * (2 if case["sampled"] else 1)
        return {"bytes": rows * case["vocab"] * e + 12 * t + 8 * t,
                "flops": 2 * rows * case["vocab"]}
    row = {"auto": 2 * case["d"], "fp8": case["d"],
           "fp4": case["d"] // 2 + case["d"] // 16}
    if case["op"] == "compact":
        stand = sum(min(4, (int(x) - 1) // 2) for x in n) // 2   # (on average)
        return {"bytes": 2 * stand * 2 * case["layers"] * case["hkv"] *
                row["auto"] + 8 * t, "flops": 0}
    keys = ctx if case["window"] < 0 else np.minimum(ctx, case["window"])
    reads = int((keys + n).sum())
    pairs = int((keys * n + n * 3).sum())
    return {"bytes": reads * case["hkv"] * 2 * row[case["cache"]] +
            t * case["hq"] * (4 * case["d"] + 4) + 4 * t +
            4 * int((-(-(ctx + n) // case["bs"])).sum()),
            "flops": 4 * case["d"] * case["hq"] * pairs}


# --------------------------------------------------------------------- inputs

def _trees(host, counts, reach):
    """Parent rows of every request's rows: each row's parent is one of the
    `reach` rows before it (1: a chain)."""
    out = []
    for n in counts.tolist():
        i = np.arange(n)
        back = host.integers(1, reach, size=n, endpoint=True)
        out.append(np.where(i > 0, np.maximum(i - back, 0), -1))
    return np.concatenate(out).astype(np.int32)


def _cu(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])
                            .astype(np.int32)).to(DEV)


def _paged(case, host, keys):
    """Block count and table of requests with this many keys."""
    blocks = -(-keys // case["bs"])
    nb = int(blocks.sum()) + 3
    perm = host.permutation(nb)
    table = np.full((len(keys), int(blocks.max())), perm[-1], np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return nb, torch.from_numpy(table).to(DEV)


def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def _cache(case, gen, nb, scale8, scale4):
    """One matrix of a cache filled with N(0, 1) rows (codes of such rows),
    its block scales and its scale."""
    shape = (nb, case["bs"], case["hkv"], case["d"])
    if case["cache"] == "auto":
        x = torch.empty(shape, dtype=DTYPES[case["dtype"]], device=DEV)
        return x.normal_(generator=gen), None, None
    if case["cache"] == "fp8":
        x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        x = (x.normal_(generator=gen) / scale8).to(torch.float8_e4m3fn)
        return x, None, torch.tensor([scale8], device=DEV)
    codes = torch.randint(0, 256, shape[:3] + (shape[3] // 2,), generator=gen,
                          dtype=torch.uint8, device=DEV)
    sf = torch.rand(shape[:3] + (shape[3] // 16,), generator=gen, device=DEV)
    sf = (sf * 80 + 80).to(torch.float8_e4m3fn)
    # each (block, head) contiguous
    codes, sf = (t.transpose(1, 2).contiguous().transpose(1, 2)
                 for t in (codes, sf.view(torch.uint8)))
    return codes, sf.view(torch.float8_e4m3fn), \
        torch.tensor([scale4], device=DEV)


def _prepare_attend(case, gen, host):
    n, ctx = _lengths(case)
    keys = ctx + n
    nb, table = _paged(case, host, keys)
    t, dtype = int(n.sum()), DTYPES[case["dtype"]]
    span = int(keys.max())
    if case["window"] >= 0:
        span = min(span, case["window"] + int(n.max()))
    k, v = (_cache(case, gen, nb, *s) for s in ((K_SCALE8, K_SCALE),
                                                (V_SCALE8, V_SCALE)))
    return dict(q=_normal(gen, dtype, t, case["hq"], case["d"]), k=k, v=v,
                table=table, k_len=torch.from_numpy(keys.astype(np.int32))
                .to(DEV), max_k=int(keys.max()), span=span,
                out=torch.empty((t, case["hq"], case["d"]), dtype=dtype,
                                device=DEV))


def _prepare_verify(case, gen, host, s):
    n = s["counts"]
    t, vocab = int(n.sum()), case["vocab"]
    dtype = DTYPES[case["dtype"]]
    target = torch.empty((t, vocab), dtype=dtype, device=DEV)
    draft = torch.empty_like(target) if case["sampled"] else None
    tokens = torch.zeros(t, dtype=torch.int64, device=DEV)
    start = np.repeat(np.cumsum(n) - n, n)
    par = s["parents"].cpu().numpy()
    # place of each row among its parent's children
    place, seen = np.zeros(t, np.int64), {}
    for i in range(t):
        key = (int(start[i]), int(par[i]))
        place[i] = seen.get(key, 0)
        seen[key] = int(place[i]) + 1
    most = max(1, int(place.max()) + 1)
    guess = torch.empty((t, most), dtype=torch.int64, device=DEV)
    step = max(1, (1 << 26) // vocab)
    for i in range(0, t, step):            # the rows in pieces
        m = min(step, t - i)
        logits = case["sharp"] * torch.randn((m, vocab), generator=gen,
                                             device=DEV)
        target[i:i + m] = torch.softmax(logits, -1).to(dtype)
        logits += torch.randn((m, vocab), generator=gen, device=DEV) * 0.7
        p = torch.softmax(logits, -1).to(dtype)
        if draft is not None:
            draft[i:i + m] = p
            guess[i:i + m] = torch.multinomial(p.float(), most, True,
                                               generator=gen)
        else:
            guess[i:i + m] = p.topk(most, -1).indices
    node = torch.from_numpy(np.flatnonzero(par >= 0)).to(DEV)
    up = torch.from_numpy((start + par)[par >= 0]).to(DEV)
    tokens[node] = guess[up, torch.from_numpy(place[par >= 0]).to(DEV)]
    return dict(target=target, draft=draft,
                tokens=tokens.to(torch.int32),
                uniform=torch.rand(t, generator=gen, device=DEV))


def _prepare_compact(case, gen, host, s):
    n, ctx = s["counts"], s["context"]
    nb, table = _paged(case, host, ctx + n)
    shape = (nb, case["bs"], case["hkv"], case["d"])
    caches = [torch.empty(shape, dtype=DTYPES[case["dtype"]], device=DEV)
              .normal_(generator=gen) for _ in range(2 * case["layers"])]
    # rows that stand: row 0 and some behind the last place that is filled
    # (a second pass finds them as the first did)
    rows = np.full((len(n), int(n.max())), -1, np.int32)
    count = np.ones(len(n), np.int32)
    for b, m in enumerate(n.tolist()):
        k = int(host.integers(0, min(4, (m - 1) // 2), endpoint=True))
        rows[b, 0] = 0
        rows[b, 1:k + 1] = np.sort(host.permutation(
            np.arange(k + 1, m))[:k])
        count[b] = k + 1
    return dict(caches=caches, table=table,
                rows=torch.from_numpy(rows).to(DEV),
                count=torch.from_numpy(count).to(DEV),
                k_len=torch.from_numpy((ctx + n).astype(np.int32)).to(DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = np.random.default_rng(seed)
    n, ctx = _lengths(case)
    s = {"case": case, "cu": _cu(n), "max_n": int(n.max()), "counts": n,
         "context": ctx}
    if case["op"] != "compact":
        par = _trees(host, n, case["reach"])
        s["parents"] = torch.from_numpy(par).to(DEV)
        # longest way from a row to row 0
        depth = np.zeros(len(par), np.int64)
        base = np.repeat(np.cumsum(n) - n, n)
        for i in np.flatnonzero(par >= 0):
            depth[i] = depth[base[i] + par[i]] + 1
        s["depth"] = int(depth.max())
    if case["op"] == "attend":
        s.update(_prepare_attend(case, gen, host))
        s["lut"] = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    elif case["op"] == "verify":
        s.update(_prepare_verify(case, gen, host, s))
    else:
        s.update(_prepare_compact(case, gen, host, s))
    return s


# ----------------------------------------------------------------- plain forms

def _values(s, which, at):
    """Rows of one matrix of the cache, float32."""
    x, sf, scale = s[which]
    x = x[at]
    if sf is not None:
        x = s["lut"][torch.stack([x & 15, x >> 4], -1).flatten(-2).int()]
        sf = sf.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
        return (x.unflatten(-1, (-1, 16)) * sf[..., None]).flatten(-2) * scale
    return x.float() if scale is None else x.float() * scale


def _attend_plain(s):
    """Padded to the longest request: [batch, rows, keys]."""
    case = s["case"]
    hkv, bs, window = case["hkv"], case["bs"], case["window"]
    q, k_len, cu = s["q"], s["k_len"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    ctx = k_len - n
    t = torch.arange(q.shape[0], device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    # which of its request's rows each row sees, and how deep it is
    sees = torch.zeros((q.shape[0], s["max_n"]), dtype=torch.bool, device=DEV)
    deep, here = torch.zeros_like(t), t
    for i in range(s["depth"] + 1):
        if window < 0 or i <= window:
            sees[t, here - cu[b]] = True
        up = s["parents"].long()[here]
        deep = deep + (up >= 0)
        here = torch.where(up >= 0, cu[b] + up, here)
    first = (k_len - s["span"]).clamp(min=0)
    key = first[:, None] + torch.arange(s["span"], device=DEV)
    blk = (key // bs).clamp(max=s["table"].shape[1] - 1)
    at = (torch.gather(s["table"].long(), 1, blk), key % bs)
    k = _values(s, "k", at)
    i = torch.arange(s["max_n"], device=DEV)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    g = case["hq"] // hkv
    rows = q[row].float().unflatten(2, (hkv, g))      # [b, i, h, g, d]
    rows = rows.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [b, h, g*i, d]
    x = rows @ k.permute(0, 2, 3, 1) * case["d"] ** -0.5
    del k
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    before = (key < ctx[:, None])[:, None].expand(-1, s["max_n"], -1)
    if window >= 0:
        before = before & (key[:, None] >=
                           (ctx[:, None] + deep[row] - window)[..., None])
    rel = (key - ctx[:, None])[:, None].expand(-1, s["max_n"], -1)
    mine = torch.gather(sees[row], 2, rel.clamp(0, s["max_n"] - 1))
    seen = before | (mine & (rel >= 0) & (key < k_len[:, None])[:, None])
    x = x.unflatten(2, (g, -1)).masked_fill_(~seen[:, None, None],
                                             float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(x.sub_(top))
    del x
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]            # [b, h, g, i]
    o = p.flatten(2, 3) @ _values(s, "v", at).permute(0, 2, 1, 3)
    o = o.unflatten(2, (g, -1)) / total.clamp(min=1e-38)
    i = t - cu[b]                                     # back to a row a token
    out = o.permute(0, 3, 1, 2, 4)[b, i].flatten(1, 2)
    return out.to(q.dtype), lse.permute(0, 3, 1, 2)[b, i].flatten(1).T


def _verify_plain(s):
    """All requests side by side, one row of each at a time, in 64 bits
    (the answers are whole numbers that turn on sums over the vocabulary)."""
    cu = s["cu"].long()
    start, n = cu[:-1], cu[1:] - cu[:-1]
    target, draft = s["target"], s["draft"]
    tokens, u = s["tokens"].long(), s["uniform"].double()
    batch, top = len(n), target.shape[0] - 1
    lane = torch.arange(batch, device=DEV)
    at = torch.zeros_like(n)                          # row that stands last
    rest = target[start].double()                     # what is left of it
    mass = torch.ones(batch, dtype=torch.float64, device=DEV)
    count = torch.ones_like(n)
    out = torch.full((batch, s["max_n"] + 1), -1, dtype=torch.int64,
                     device=DEV)
    rows = out.clone()
    rows[:, 0] = 0
    for i in range(1, s["max_n"]):
        row = (start + i).clamp(max=top)
        asked = (i < n) & (s["parents"].long()[row] == at)
        x = tokens[row]
        have = rest[lane, x]
        likely = draft[start + at, x].double() if draft is not None else 1.0
        stands = asked & (u[row] * likely * mass < have)
        falls = asked & ~stands
        if draft is not None:
            left = (rest - mass[:, None] * draft[start + at].double()) \
                .clamp(min=0.0)
            rest = torch.where(falls[:, None], left, rest)
            mass = torch.where(falls, rest.sum(-1), mass)
        else:
            mass = torch.where(falls, mass - have, mass)
            rest[lane, x] = torch.where(falls, 0.0, have)
        end = torch.where(stands, count, s["max_n"])  # (the spare column)
        out[lane, end - 1] = torch.where(stands, x, out[lane, end - 1])
        rows[lane, end] = torch.where(stands, i, -1)
        count = count + stands
        at = torch.where(stands, i, at)
        rest = torch.where(stands[:, None], target[row].double(), rest)
        mass = torch.where(stands, 1.0, mass)
    whole = target[start + at].double()
    rest = torch.where((rest.sum(-1) > 0)[:, None], rest, whole)
    run_sum = rest.cumsum(-1)
    over = run_sum > (u[start] * run_sum[:, -1])[:, None]
    out[lane, count - 1] = over.int().argmax(-1)
    return (out[:, :s["max_n"]].int(), rows[:, :s["max_n"]].int(),
            count.int())


def _compact_plain(s):
    bs = s["case"]["bs"]
    table, rows = s["table"].long(), s["rows"].long()
    cu = s["cu"].long()
    ctx = (s["k_len"].long() - (cu[1:] - cu[:-1]))[:, None]
    i = torch.arange(rows.shape[1], device=DEV)
    # places past the count take row 0 to itself
    live = i < s["count"].long()[:, None]
    src = ctx + torch.where(live, rows, 0)
    dst = ctx + torch.where(live, i, 0)
    src, dst = ((torch.gather(table, 1, x // bs), x % bs)
                for x in (src, dst))
    for c in s["caches"]:
        c[dst] = c[src]
    return s["caches"]


# ------------------------------------------------------------------------ run

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"attend": _attend_plain, "verify": _verify_plain,
                "compact": _compact_plain}[op](s)
    from paged_kv_cache_318_gb300 import api
    if op == "attend":
        (k, k_sf, k_scale), (v, v_sf, v_scale) = s["k"], s["v"]
        return api.flash_attn_varlen_func(
            s["q"], k, v, s["max_n"], s["cu"], s["max_k"],
            seqused_k=s["k_len"], causal=True,
            window_size=(case["window"], -1), softcap=case["softcap"],
            block_table=s["table"], return_softmax_lse=True, out=s["out"],
            k_descale=k_scale, v_descale=v_scale, k_block_scale=k_sf,
            v_block_scale=v_sf, tree_parents=s["parents"])
    if op == "verify":
        return api.verify_draft_tokens(
            s["target"], s["tokens"], s["cu"], s["max_n"], s["uniform"],
            tree_parents=s["parents"], draft_probs=s["draft"])
    api.compact_draft_cache(s["caches"], s["table"], s["cu"], s["k_len"],
                            s["rows"], s["count"])
    return s["caches"]


# ---------------------------------------------------------------------- exact

def _exact_rows(s, which, pages, keep):
    x, sf, scale = s[which]
    c = x[pages].flatten(0, 1)[:keep]
    if sf is not None:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).int()
        e, m = (c >> 1) & 3, (c & 1).double()
        val = torch.where(e == 0, 0.5 * m,
                          (1 + 0.5 * m) * torch.exp2(e.double() - 1))
        val = torch.where(c >= 8, -val, val)
        f = sf.view(torch.uint8)[pages].flatten(0, 1)[:keep]
        f = f.view(torch.float8_e4m3fn).float().double()
        val = val * f.repeat_interleave(16, -1)
    else:
        val = c.float().double()
    return val if scale is None else val * scale.double()


def _exact_attend(case, s):
    g = case["hq"] // case["hkv"]
    cu, par = s["cu"].tolist(), s["parents"].tolist()
    outs, lses = [], []
    for b, n_k in enumerate(s["k_len"].tolist()):
        n = cu[b + 1] - cu[b]
        ctx = n_k - n
        sees = np.zeros((n, n), bool)
        deep = np.zeros(n, np.int64)
        for i in range(n):
            j, far = i, 0
            while j >= 0:
                sees[i, j] = case["window"] < 0 or far <= case["window"]
                j, far = par[cu[b] + j], far + 1
            deep[i] = far - 1
        lo = 0 if case["window"] < 0 else \
            max(0, ctx - case["window"]) // case["bs"]
        base = lo * case["bs"]
        pages = s["table"][b, lo:-(-n_k // case["bs"])].long()
        k, v = (_exact_rows(s, w, pages, n_k - base) for w in "kv")
        key = torch.arange(base, ctx, device=DEV)[None]
        hide = torch.zeros((n, ctx - base), dtype=torch.bool, device=DEV)
        if case["window"] >= 0:
            hide = key < torch.from_numpy(ctx + deep).to(DEV)[:, None] - \
                case["window"]
        hide = torch.cat([hide, torch.from_numpy(~sees).to(DEV)], 1)
        q = s["q"][cu[b]:cu[b + 1]].double()
        out = torch.empty((n, case["hq"], case["d"]), dtype=torch.float64,
                          device=DEV)
        lse = torch.empty((case["hq"], n), dtype=torch.float64, device=DEV)
        for h in range(case["hq"]):
            x = q[:, h] @ k[:, h // g].T / case["d"] ** 0.5
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            x = x.masked_fill(hide, float("-inf"))
            lse[h] = torch.logsumexp(x, 1)
            out[:, h] = torch.softmax(x, 1) @ v[:, h // g]
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses, 1)


def _exact_verify(case, s):
    """One request at a time, with numpy on the host."""
    cu, par = s["cu"].tolist(), s["parents"].tolist()
    tok, u = s["tokens"].tolist(), s["uniform"].double().tolist()
    batch, most = len(cu) - 1, s["max_n"]
    out = np.full((batch, most), -1, np.int32)
    rows = np.full((batch, most), -1, np.int32)
    count = np.zeros(batch, np.int32)

    def dist(t, r):
        return t[r].double().cpu().numpy()

    for b in range(batch):
        first, n = cu[b], cu[b + 1] - cu[b]
        path, said, node = [0], [], 0
        left, total = dist(s["target"], first), 1.0
        while True:
            nxt = -1
            kids = [i for i in range(node + 1, n) if par[first + i] == node]
            q = None
            if kids and s["draft"] is not None:
                q = dist(s["draft"], first + node)
            for i in kids:
                x = tok[first + i]
                bar = u[first + i] * total * (1.0 if q is None else q[x])
                if bar < left[x]:
                    nxt = i
                    break
                if q is None:
                    total -= left[x]
                    left[x] = 0.0
                else:
                    left = np.maximum(left - total * q, 0.0)
                    total = float(left.sum())
            if nxt < 0:
                break
            said.append(tok[first + nxt])
            path.append(nxt)
            node = nxt
            left, total = dist(s["target"], first + node), 1.0
        if not left.sum() > 0:
            left = dist(s["target"], first + node)
        c = np.cumsum(left)
        said.append(int(np.searchsorted(c, u[first] * c[-1], side="right")))
        out[b, :len(said)], rows[b, :len(path)] = said, path
        count[b] = len(path)
    return tuple(torch.from_numpy(x).to(DEV) for x in (out, rows, count))


def _exact_compact(case, s):
    cu, k_len = s["cu"].tolist(), s["k_len"].tolist()
    rows, count = s["rows"].tolist(), s["count"].tolist()
    table = s["table"].tolist()
    moves = []
    for b in range(len(k_len)):
        ctx = k_len[b] - (cu[b + 1] - cu[b])
        for i in range(count[b]):
            moves.append([(table[b][x // case["bs"]], x % case["bs"])
                          for x in (ctx + i, ctx + rows[b][i])])
    answer = []
    to = torch.tensor([m[0] for m in moves], device=DEV).T
    of = torch.tensor([m[1] for m in moves], device=DEV).T
    for c in s["caches"]:
        x = c.double()
        x[to[0], to[1]] = c[of[0], of[1]].double()
        answer.append(x)
    return answer


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "verify": _exact_verify,
            "compact": _exact_compact}[case["op"]](case, s)
