"""Cases of the operators around a 4-bit paged KV cache, for timing.

Four operators, in the order a serving step runs them:

* ``norm_rope``   -- RMS norm of every query and key head and the rotary
  position rotation, in one pass;
* ``rope_append`` -- the same on q and k, with the rotated keys and the
  values appended to a paged cache (16-bit, E4M3 or 4-bit);
* ``append``      -- keys and values appended to a 4-bit cache as they are,
  and the cache read back in the model's type (as ``rope_append`` does too,
  where its cache has 4 bits);
* ``attend``      -- attention over a 4-bit paged cache.

The 4-bit cache holds E2M1 codes, two to a byte (the lower index in the lower
four bits), with one E4M3 scale for each 16 values of a row and one float32
scale for the whole cache: value = code * block_scale * scale.

``run`` computes a case in plain torch operations, or, with ``own`` set, by
the package's operators.
"""
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"
K_SCALE, V_SCALE = 0.0021, 0.0017       # 4-bit cache: about amax / (6 * 448)
K_SCALE8, V_SCALE8 = 0.02, 0.013        # E4M3 cache
EPS = 1e-6


# ---------------------------------------------------------------------- cases

def _rope(name, op, tokens, hq, hkv, d, **kw):
    c = dict(name=name, op=op, tokens=tokens, pad=0, hq=hq, hkv=hkv, d=d,
             rot=d, neox=True, sections="", woven=False, norm=True,
             offset=0.0, dtype="bf16", table="f32", max_pos=16384,
             order="prompt", cache="", bs=16)
    c.update(kw)
    return c


def _attend(name, batch, q, k, hq, hkv, d, **kw):
    c = dict(name=name, op="attend", batch=batch, q_lo=q[0], q_hi=q[1],
             k_lo=k[0], k_hi=k[1], hq=hq, hkv=hkv, d=d, bs=16, window=-1,
             softcap=0.0, dtype="bf16", lens=319)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of 64 requests: 64 tokens, latency-bound
        _rope("norm_rope step", "norm_rope", 64, 32, 8, 128, order="step"),
        # image and video tokens with (time, height, width) positions
        _rope("norm_rope 3 axes", "norm_rope", 8192, 16, 8, 256,
              sections="40,44,44", woven=True, dtype="f16", table="16",
              order="grid"),
        # one decode step into a 16-bit cache; half of each head rotates, in
        # adjacent pairs, and the model has no head norms
        _rope("rope_append step", "rope_append", 64, 32, 8, 128, rot=64,
              neox=False, norm=False, order="step", cache="auto"),
        # a batch of prompts into an E4M3 cache, norm weights stored around 0,
        # with the padded tail of a captured batch size
        _rope("rope_append fp8 prompt", "rope_append", 8103, 16, 8, 256,
              pad=89, offset=1.0, cache="fp8", bs=32),
        # a batch of prompts into the 4-bit cache
        _rope("rope_append fp4 prompt", "rope_append", 11207, 32, 8, 128,
              cache="fp4"),
        # one decode step of 124 requests into the 4-bit cache
        _rope("append step", "append", 124, 0, 8, 256, order="step",
              cache="fp4", bs=32, norm=False),
        # a batch of prompts into the 4-bit cache
        _rope("append prompt", "append", 11207, 0, 8, 128, cache="fp4",
              norm=False, dtype="f16"),
        # two short chats on a small model: latency-bound
        _attend("attend tiny", 2, (1, 1), (37, 50), 4, 2, 64, lens=318),
        # one decode step of a batch of 64
        _attend("attend batch", 64, (1, 1), (512, 4096), 32, 8, 128),
        # decoding after very long prompts
        _attend("attend long", 8, (1, 1), (131072, 131072), 64, 8, 128,
                bs=64, lens=322),
        # sliding window and soft-cap, two drafted tokens a request
        _attend("attend window", 124, (2, 2), (1024, 16384), 16, 8, 256,
                bs=32, window=4095, softcap=50.0, lens=321),
        # prompts that extend what the cache already holds
        _attend("attend prompt", 8, (256, 2048), (512, 2048), 32, 8, 128,
                lens=320),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng: random.Random):
    op = rng.choice(["norm_rope", "rope_append", "append", "attend",
                     "attend"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 8])
    bs = rng.choice([16, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op != "attend":
        tokens = _log(rng, 1, 12000 * 5120 // ((g + 2) * hkv * d) if
                      (g + 2) * hkv * d > 5120 else 12000)
        rot = rng.choice([d, d, d // 2, d // 4])
        axes = rng.choice([1, 1, 2, 3]) if op != "append" else 1
        half = rot // 2
        a = half // axes
        sections = "" if axes == 1 else ",".join(
            str(x) for x in [half - a * (axes - 1)] + [a] * (axes - 1))
        return _rope("", op, tokens, 0 if op == "append" else g * hkv, hkv, d,
                     pad=rng.choice([0, 0, rng.randint(1, 40)]), rot=rot,
                     neox=rng.random() < 0.7, sections=sections,
                     woven=axes > 1 and rng.random() < 0.5,
                     norm=op != "append" and rng.random() < 0.6,
                     offset=rng.choice([0.0, 1.0]), dtype=dtype,
                     table=rng.choice(["f32", "16"]),
                     max_pos=_log(rng, 64, 40000),
                     order="grid" if axes > 1 else
                     rng.choice(["step", "prompt"]),
                     cache="" if op == "norm_rope" else "fp4"
                     if op == "append" else rng.choice(["auto", "fp8", "fp4"]),
                     bs=bs)
    window = rng.choice([-1, -1, rng.randint(1, 5000)])
    q_hi = rng.choice([1, 1, 1, rng.randint(2, 4), _log(rng, 17, 700)])
    most = 2_000_000 if q_hi <= 4 else 40_000
    batch = _log(rng, 1, 160 if q_hi <= 4 else 10)
    k_hi = _log(rng, max(16, q_hi), max(64, q_hi * 2, most // batch // hkv))
    return _attend("", batch, (max(1, q_hi // 3), q_hi),
                   (max(1, k_hi // 8), k_hi), g * hkv, hkv, d, bs=bs,
                   window=window, softcap=rng.choice([0.0, 0.0, 30.0]),
                   dtype=dtype, lens=rng.randint(0, 1 << 20))


def _lengths(case):
    """Query and key counts of each request, from the case alone."""
    r = np.random.default_rng([case["lens"], 2])
    n = case["batch"]
    q = r.integers(case["q_lo"], case["q_hi"], size=n, endpoint=True)
    k = r.integers(case["k_lo"], case["k_hi"], size=n, endpoint=True)
    return q, np.maximum(k, q) if case["q_hi"] <= 4 else q + k


def _sections(case):
    return [int(x) for x in case["sections"].split(",") if x]


def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "attend":
        q, k = _lengths(case)
        pairs = reads = 0
        for a, b in zip(q.tolist(), k.tolist()):
            pos = np.arange(b - a, b)
            lo = np.zeros_like(pos) if case["window"] < 0 else \
                np.maximum(pos - case["window"], 0)
            pairs += int((pos + 1 - lo).sum())
            reads += b - int(lo[0])
        t = int(q.sum())
        blocks = int(sum(-(-int(x) // case["bs"]) for x in k))
        return {"bytes": reads * hkv * 2 * (d // 2 + d // 16) +
                t * hq * (4 * d + 4) + 4 * blocks + 8 * len(q),
                "flops": 4 * d * hq * pairs}
    t = case["tokens"]
    row = {"": 2 * d, "auto": 2 * d, "fp8": d, "fp4": d // 2 + d // 16}
    if case["op"] == "append":
        return {"bytes": t * hkv * 2 * (2 * d + row["fp4"]) + 8 * t,
                "flops": 4 * t * hkv * 2 * d}
    axes = max(1, len(_sections(case)))
    table = min(case["max_pos"], t * axes) * case["rot"] * \
        (4 if case["table"] == "f32" else 2)
    n = t * hq * 4 * d + t * hkv * (2 * d + row[case["cache"]])
    if case["op"] == "rope_append":
        n += t * hkv * (2 * d + row[case["cache"]]) + 8 * t
    return {"bytes": n + table + 8 * t * axes,
            "flops": t * (hq + hkv) * (3 * case["rot"] +
                                       (5 * d if case["norm"] else 0))}


# --------------------------------------------------------------------- inputs

def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def _fp4_cache(nb, bs, hkv, d):
    """Codes [NB, BS, Hkv, D/2] and block scales [NB, BS, Hkv, D/16] of one
    matrix; each (block, head) is contiguous in memory."""
    codes = torch.zeros((nb, hkv, bs, d // 2), dtype=torch.uint8, device=DEV)
    sf = torch.zeros((nb, hkv, bs, d // 16), dtype=torch.uint8, device=DEV)
    return (codes.permute(0, 2, 1, 3),
            sf.view(torch.float8_e4m3fn).permute(0, 2, 1, 3))


def _prepare_attend(case, gen, host):
    d, hkv, bs = case["d"], case["hkv"], case["bs"]
    dtype = DTYPES[case["dtype"]]
    q_len, k_len = _lengths(case)
    blocks = -(-k_len // bs)
    nb = int(blocks.sum()) + 3
    perm = host.permutation(nb)
    table = np.full((len(k_len), int(blocks.max())), perm[-1], np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    s = {"caches": []}
    for scale in (K_SCALE, V_SCALE):
        codes, sf = _fp4_cache(nb, bs, hkv, d)
        step = max(1, (1 << 26) // (bs * hkv * d))
        for i in range(0, nb, step):       # N(0,1) rows, quantized in pieces
            x = _normal(gen, dtype, min(step, nb - i), bs, hkv, d)
            codes[i:i + step], f = _quantize(x.float(), scale)
            sf[i:i + step] = f.to(torch.float8_e4m3fn)
        s["caches"].append((codes, sf))
    t = int(q_len.sum())
    cu = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    span = int(k_len.max())
    if case["window"] >= 0:
        span = min(span, case["window"] + int(q_len.max()))
    s.update(q=_normal(gen, dtype, t, case["hq"], d),
             table=torch.from_numpy(table).to(DEV),
             cu=torch.from_numpy(cu).to(DEV),
             k_len=torch.from_numpy(k_len.astype(np.int32)).to(DEV),
             max_q=int(q_len.max()), max_k=int(k_len.max()), span=span,
             out=torch.empty((t, case["hq"], d), dtype=dtype, device=DEV))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = np.random.default_rng(seed)
    d, hkv, hq, bs = case["d"], case["hkv"], case["hq"], case["bs"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "attend":
        s = _prepare_attend(case, gen, host)
    else:
        n = case["tokens"] + case["pad"]
        heads = hq + 2 * hkv
        # the projection's output holds q, k and v side by side
        qkv = _normal(gen, dtype, n, heads, d) * 1.3
        s = {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv],
             "v": qkv[:, hq + hkv:], "n": case["tokens"]}
        if case["op"] != "append":
            s.update(_prepare_rope(case, gen, host, n))
        if case["cache"]:
            nb = -(-case["tokens"] // bs) + 2
            if case["order"] == "step":    # a slot anywhere in a larger pool
                nb = case["tokens"] + 2
                slots = host.permutation(nb)[:case["tokens"]] * bs + \
                    host.integers(0, bs, case["tokens"])
            else:                          # whole blocks in shuffled order
                t = np.arange(case["tokens"])
                slots = host.permutation(nb)[t // bs] * bs + t % bs
            slots = np.concatenate([slots, np.full(case["pad"], -1)])
            s["slots"] = torch.from_numpy(slots.astype(np.int64)).to(DEV)
            if case["cache"] == "fp4":
                s["caches"] = [_fp4_cache(nb, bs, hkv, d) for _ in "kv"]
                s["back"] = [torch.empty((nb, bs, hkv, d), dtype=dtype,
                                         device=DEV) for _ in "kv"]
            else:
                kind = torch.float8_e4m3fn if case["cache"] == "fp8" else dtype
                s["caches"] = [(torch.zeros((nb, bs, hkv, d), device=DEV)
                                .to(kind), None) for _ in "kv"]
    scales = {"fp8": (K_SCALE8, V_SCALE8)}.get(case.get("cache"),
                                               (K_SCALE, V_SCALE))
    s["case"] = case
    s["scale"] = [torch.tensor([x], dtype=torch.float32, device=DEV)
                  for x in scales]
    # the two values of each code byte, for reading a 4-bit cache back
    byte = torch.arange(256, device=DEV)
    s["lut"] = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    s["pairs"] = torch.stack([s["lut"][byte & 15], s["lut"][byte >> 4]], -1) \
        .to(dtype).contiguous().view(torch.int32).reshape(256)
    return s


def _prepare_rope(case, gen, host, n):
    rot, dtype = case["rot"], DTYPES[case["dtype"]]
    freq = 1e4 ** (-torch.arange(0, rot, 2, device=DEV,
                                 dtype=torch.float64) / rot)
    angle = torch.arange(case["max_pos"], device=DEV,
                         dtype=torch.float64)[:, None] * freq
    table = torch.cat([angle.cos(), angle.sin()], -1)
    axes = max(1, len(_sections(case)))
    top = case["max_pos"]
    if case["order"] == "prompt":
        pos = np.arange(n) % min(top, 2048)
    elif case["order"] == "step":
        pos = host.integers(0, top, n)
    else:                                  # a grid of patches per frame
        side = max(1, min(top, 48))
        t = np.arange(n)
        pos = np.stack([t // (side * side) % top, t // side % side,
                        t % side][:axes])
    pos = torch.from_numpy(np.ascontiguousarray(pos).astype(np.int64)).to(DEV)
    weight = [None, None]
    if case["norm"]:
        mid = 1.0 - case["offset"]
        weight = [(mid + 0.2 * torch.randn(case["d"], generator=gen,
                                           device=DEV)).to(dtype)
                  for _ in "qk"]
    kept = {"positions": pos, "weight": weight,
            "table": table.to(torch.float32 if case["table"] == "f32"
                              else dtype)}
    kept["axis"] = torch.tensor(_axis_of_pair(case), device=DEV)
    kept["q_out"] = torch.empty((n, case["hq"], case["d"]), dtype=dtype,
                                device=DEV)
    kept["k_out"] = torch.empty((n, case["hkv"], case["d"]), dtype=dtype,
                                device=DEV)
    return kept


# ----------------------------------------------------------------- plain forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1(lut, code):
    """Value of a 4-bit code, float32."""
    return lut[code.long()]


def _quantize(x, scale):
    """4-bit codes (two to a byte) and block scales of rows [..., D]."""
    g = x.unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    scale = torch.as_tensor(scale, dtype=torch.float32, device=x.device)
    sf = (top * (1.0 / (scale * 6.0))).clamp(max=448.0) \
        .to(torch.float8_e4m3fn).float()
    step = sf * scale
    inv = torch.where(step > 0, 1.0 / step, 0.0)[..., None]
    y = g * inv
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) +
            (a > 2.5) + (a >= 3.5) + (a > 5.0)) | ((y < 0).byte() << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf


def _read_back(state, which):
    """The values a 4-bit cache stands for, in the model's type."""
    codes, sf = state["caches"][which]
    if own:
        from paged_kv_cache_318_gb300 import api
        return api.dequantize_fp4_cache(codes, sf, state["scale"][which],
                                        out=state["back"][which])
    dtype = DTYPES[state["case"]["dtype"]]
    v = state["pairs"][codes.int()].view(dtype)
    v = v.unflatten(-1, (-1, 16)) * sf.to(dtype)[..., None]
    return (v * (K_SCALE, V_SCALE)[which]).flatten(-2)


def _pairwise_sum(x):
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x


def _axis_of_pair(case):
    """Which axis' position rotates each pair of dimensions."""
    sections, half = _sections(case), case["rot"] // 2
    if not case["woven"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    n = len(sections)
    return [i % n if i < n * sections[i % n] else 0 for i in range(half)]


def _norm_rope(state, x, weight):
    """Rows x [n, heads, d] normed and rotated, float32."""
    case, positions, table = state["case"], state["positions"], state["table"]
    x = x.float()
    if weight is not None:
        mean = _pairwise_sum(x * x) / case["d"]
        x = x * (1.0 / torch.sqrt(mean + EPS)) * \
            (weight.float() + case["offset"])
    rot, half = case["rot"], case["rot"] // 2
    if case["sections"]:
        i = torch.arange(half, device=x.device)
        at = positions[state["axis"]].T              # [n, half]
        c, s = table[at, i].float(), table[at, i + half].float()
    else:
        row = table[positions].float()
        c, s = row[:, :half], row[:, half:]
    c, s = c[:, None], s[:, None]
    if case["neox"]:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _store(state, which, x):
    """Rows x [n, heads, d], float32, into a paged cache at the slots."""
    case, n = state["case"], state["n"]
    codes, sf = state["caches"][which]
    slots = state["slots"][:n]
    at = (slots // case["bs"], slots % case["bs"])
    if case["cache"] == "fp4":
        codes[at], f = _quantize(x, state["scale"][which])
        sf.view(torch.uint8)[at] = f.to(torch.float8_e4m3fn).view(torch.uint8)
    elif case["cache"] == "fp8":
        y = (x / state["scale"][which]).clamp(-448.0, 448.0)
        codes.view(torch.uint8)[at] = \
            y.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes[at] = x.to(codes.dtype)


def _dequantize(lut, codes, sf, scale):
    v = torch.stack([_e2m1(lut, codes & 15), _e2m1(lut, codes >> 4)], -1)
    v = v.flatten(-2)
    v = v.unflatten(-1, (-1, 16)) * sf.float()[..., None]
    return v.flatten(-2) * scale


def _attend_plain(s):
    """Padded to the longest request: [batch, queries, keys]."""
    case = s["case"]
    d, hkv, bs = case["d"], case["hkv"], case["bs"]
    q, k_len, cu = s["q"], s["k_len"].long(), s["cu"].long()
    n_q = cu[1:] - cu[:-1]
    first = (k_len - s["span"]).clamp(min=0)
    key = first[:, None] + torch.arange(s["span"], device=DEV)
    blk = (key // bs).clamp(max=s["table"].shape[1] - 1)
    at = (torch.gather(s["table"].long(), 1, blk), key % bs)
    k, v = (_dequantize(s["lut"], codes[at], sf.view(torch.uint8)[at]
                        .view(torch.float8_e4m3fn), scale)
            for (codes, sf), scale in zip(s["caches"], s["scale"]))
    i = torch.arange(s["max_q"], device=DEV)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    pos = (k_len - n_q)[:, None] + i                  # [batch, queries]
    g = case["hq"] // hkv
    rows = q[row].float().unflatten(2, (hkv, g))      # [b, i, h, g, d]
    rows = rows.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [b, h, g*i, d]
    x = rows @ k.permute(0, 2, 3, 1) * d ** -0.5      # [b, h, g*i, j]
    del k
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    seen = (key[:, None] <= pos[..., None]) & \
        (key < k_len[:, None])[:, None]
    if case["window"] >= 0:
        seen &= key[:, None] >= pos[..., None] - case["window"]
    x = x.unflatten(2, (g, -1)).masked_fill_(~seen[:, None, None],
                                             float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]            # [b, h, g, i]
    o = p.flatten(2, 3) @ v.permute(0, 2, 1, 3)
    o = o.unflatten(2, (g, -1)) / total.clamp(min=1e-38)
    # back to one row a token
    t = torch.arange(q.shape[0], device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[b]
    out = o.permute(0, 3, 1, 2, 4)[b, i].flatten(1, 2)
    return out.to(q.dtype), lse.permute(0, 3, 1, 2)[b, i].flatten(1).T


# ------------------------------------------------------------------------ run

def _own_rope(s):
    case = s["case"]
    sections = _sections(case)
    return dict(q_weight=s["weight"][0], k_weight=s["weight"][1], eps=EPS,
                is_neox=case["neox"], mrope_section=sections or None,
                mrope_interleaved=case["woven"],
                weight_offset=case["offset"], q_out=s["q_out"])


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        from paged_kv_cache_318_gb300 import api
        if op == "norm_rope":
            return api.qk_norm_rope(s["q"], s["k"], s["positions"],
                                    s["table"], k_out=s["k_out"],
                                    **_own_rope(s))
        (kc, k_sf), (vc, v_sf) = s["caches"]
        if op == "attend":
            return api.flash_attn_varlen_func(
                s["q"], kc, vc, s["max_q"], s["cu"], s["max_k"],
                seqused_k=s["k_len"], causal=True,
                window_size=(case["window"], -1), softcap=case["softcap"],
                block_table=s["table"], return_softmax_lse=True,
                out=s["out"], k_descale=s["scale"][0],
                v_descale=s["scale"][1], k_block_scale=k_sf,
                v_block_scale=v_sf)
        if op == "append":
            api.reshape_and_cache_flash(
                s["k"], s["v"], kc, vc, s["slots"], "fp4", s["scale"][0],
                s["scale"][1], k_block_scale=k_sf, v_block_scale=v_sf)
            return _read_back(s, 0), _read_back(s, 1)
        q = api.rope_reshape_and_cache(
            s["q"], s["k"], s["v"], kc, vc, s["slots"], s["positions"],
            s["table"], kv_cache_dtype=case["cache"], k_scale=s["scale"][0],
            v_scale=s["scale"][1], k_block_scale=k_sf, v_block_scale=v_sf,
            **_own_rope(s))
    else:
        if op == "attend":
            return _attend_plain(s)
        if op != "append":
            q, k = (_norm_rope(s, x, w)
                    for x, w in zip((s["q"], s["k"]), s["weight"]))
            q = q.to(s["q"].dtype)
            if op == "norm_rope":
                return q, k.to(s["k"].dtype)
        else:
            k = s["k"].float()
        _store(s, 0, k[:s["n"]])
        _store(s, 1, s["v"][:s["n"]].float())
        if op == "append":
            return _read_back(s, 0), _read_back(s, 1)
    if case["cache"] == "fp4":
        return q, _read_back(s, 0), _read_back(s, 1)
    return q, s["caches"][0][0], s["caches"][1][0]


# ---------------------------------------------------------------------- exact

def _round_to(x, bits, lowest, most):
    """float64 x on the grid of a small float: `bits` of significand, lowest
    exponent `lowest`, ties to even, largest value `most`."""
    e = torch.frexp(x.abs())[1].double() - 1
    step = torch.exp2(e.clamp(min=lowest) - (bits - 1))
    return (torch.round(x / step) * step).clamp(-most, most)


def _exact_fp4(x, scale):
    """Rows x [..., d], float64, as the 4-bit cache gives them back."""
    shape = x.shape
    x = x.reshape(-1, 16)
    sf = _round_to(x.abs().max(1, keepdim=True).values / (6 * scale), 4, -6,
                   448)
    unit = torch.where(sf > 0, sf * scale, 1.0)
    y = torch.where(sf > 0, _round_to(x / unit, 2, 0, 6), 0.0)
    return (y * sf * scale).reshape(shape)


def _exact_rope(case, x, weight, positions, table):
    n = x.shape[0]
    out = x.double().clone()
    if weight is not None:
        w = weight.double() + case["offset"]
        out = out * w * torch.rsqrt((out ** 2).mean(2, keepdim=True) + EPS)
    src = out.clone()
    half = case["rot"] // 2
    sections = _sections(case)
    axis_of = []
    if not sections:
        axis_of = [0] * half
    elif not case["woven"]:
        for a, count in enumerate(sections):
            axis_of += [a] * count
    else:
        for i in range(half):
            a = i % len(sections)
            axis_of.append(a if i < len(sections) * sections[a] else 0)
    pos = positions if positions.dim() == 2 else positions[None]
    for i in range(half):
        row = table[pos[axis_of[i]]].double()
        c, s = row[:, i].reshape(n, 1), row[:, half + i].reshape(n, 1)
        a, b = (i, i + half) if case["neox"] else (2 * i, 2 * i + 1)
        out[:, :, a] = src[:, :, a] * c - src[:, :, b] * s
        out[:, :, b] = src[:, :, a] * s + src[:, :, b] * c
    return out


def _exact_attend(case, s):
    d, hkv, g = case["d"], case["hkv"], case["hq"] // case["hkv"]
    outs, lses = [], []
    cu = s["cu"].tolist()
    for b, n_k in enumerate(s["k_len"].tolist()):
        q = s["q"][cu[b]:cu[b + 1]].double()
        n_q = q.shape[0]
        lo = 0 if case["window"] < 0 else \
            max(0, n_k - n_q - case["window"]) // case["bs"]
        pages = s["table"][b, lo:-(-n_k // case["bs"])].long()
        base = lo * case["bs"]
        kv = []
        for (codes, sf), scale in zip(s["caches"], (K_SCALE, V_SCALE)):
            c = codes[pages].flatten(0, 1)[:n_k - base]
            c = torch.stack([c & 15, c >> 4], -1).flatten(-2).int()
            e, m = (c >> 1) & 3, (c & 1).double()
            val = torch.where(e == 0, 0.5 * m,
                              (1 + 0.5 * m) * torch.exp2(e.double() - 1))
            val = torch.where(c >= 8, -val, val)
            f = sf.view(torch.uint8)[pages].flatten(0, 1)[:n_k - base]
            f = f.view(torch.float8_e4m3fn).float().double()
            kv.append(val * f.repeat_interleave(16, -1) *
                      float(np.float32(scale)))
        pos = torch.arange(n_k - n_q, n_k, device=DEV)[:, None]
        key = torch.arange(base, n_k, device=DEV)[None]
        hide = key > pos
        if case["window"] >= 0:
            hide = hide | (key < pos - case["window"])
        out = torch.empty((n_q, case["hq"], d), dtype=torch.float64,
                          device=DEV)
        lse = torch.empty((case["hq"], n_q), dtype=torch.float64, device=DEV)
        for h in range(case["hq"]):
            x = q[:, h] @ kv[0][:, h // g].T / d ** 0.5
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            x = x.masked_fill(hide, float("-inf"))
            lse[h] = torch.logsumexp(x, 1)
            out[:, h] = torch.softmax(x, 1) @ kv[1][:, h // g]
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    answer = []
    k = s["k"].double()
    if case["op"] != "append":
        q, k = (_exact_rope(case, x, w, s["positions"], s["table"])
                for x, w in zip((s["q"], s["k"]), s["weight"]))
        answer.append(q)
        if case["op"] == "norm_rope":
            return q, k
    n, bs = s["n"], case["bs"]
    slots = s["slots"][:n]
    for which, x in enumerate((k[:n], s["v"][:n].double())):
        codes, _ = s["caches"][which]
        nb = codes.shape[0]
        if case["cache"] == "fp4":
            x = _exact_fp4(x, float(np.float32((K_SCALE, V_SCALE)[which])))
        elif case["cache"] == "fp8":
            x = _round_to(x / float(np.float32((K_SCALE8, V_SCALE8)[which])),
                          4, -6, 448)
        rows = torch.zeros((nb * bs, case["hkv"], case["d"]),
                           dtype=torch.float64, device=DEV)
        rows[slots] = x
        answer.append(rows.reshape(nb, bs, case["hkv"], case["d"]))
    return tuple(answer)
