"""Measured calls of the rotating cache writes and of the latent attention.

Four operators, each in a plain form (elementary torch operations) and, with
``own`` set, as the calls a user makes of this library:

  append   rope_append: new tokens' queries and keys are rotated by their
           positions, keys and values go to their slots of the paged caches.
  lappend  latent_append: the same for a latent cache, whose rows hold one
           vector and one rotated key for all heads.
  decode   latent_attn_decode: one query per sequence over the latent rows that
           its block table names (absorbed form: queries already in the latent
           space, values are the rows' latent part).
  prompt   latent_prompt_attn: causal attention over whole prompts with the keys
           and values expanded per head (expanded form), the rotated key shared.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
ROPE = 64  # dims of a latent row's shared key
F32, BF16, E4M3, E5M2 = "f32", "bf16", "e4m3", "e5m2"
TORCH = {F32: torch.float32, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
BYTES = {F32: 4, BF16: 2, E4M3: 1, E5M2: 1}
MOST = {E4M3: 448.0, E5M2: 57344.0}
KV_SCALE = 0.03125  # of the 8-bit caches
MAX_POS = 32768


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of the 8B layer: 64 tokens, each in a page of its own sequence.
        {"name": "append_decode_8b", "op": "append", "dtype": BF16, "cache": BF16, "heads": 32,
         "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "rows": 64, "decode": True,
         "lo": 16, "hi": 32768, "shape_seed": 1},
        # The prompts of a full chat batch of the 70B layer.
        {"name": "append_chat_70b", "op": "append", "dtype": BF16, "cache": BF16, "heads": 64,
         "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "rows": 128, "decode": False,
         "lo": 256, "hi": 512, "shape_seed": 2},
        # An fp8 cache, heads of 64 of which half the dims rotate in neighbouring pairs, ragged
        # prompts, some empty.
        {"name": "append_fp8_odd", "op": "append", "dtype": BF16, "cache": E4M3, "heads": 24,
         "kv_heads": 2, "dim": 64, "rot": 32, "interleaved": True, "rows": 37, "decode": False,
         "lo": 0, "hi": 1000, "shape_seed": 3},
        # One decode step into the latent cache.
        {"name": "latent_append_decode", "op": "lappend", "dtype": BF16, "heads": 32, "latent": 512,
         "interleaved": True, "rows": 64, "decode": True, "lo": 16, "hi": 32768, "shape_seed": 4},
        # The rows of a batch of documents.
        {"name": "latent_append_batch", "op": "lappend", "dtype": BF16, "heads": 32, "latent": 512,
         "interleaved": True, "rows": 16, "decode": False, "lo": 512, "hi": 4096, "shape_seed": 5},
        # One short chat on an idle server: the latency of a call.
        {"name": "latent_one_200", "op": "decode", "dtype": BF16, "heads": 32, "latent": 512, "rows": 1,
         "lens": "uniform", "lo": 200, "hi": 200, "shape_seed": 6},
        # A server's batch, 64 heads, contexts of very different lengths.
        {"name": "latent_batch_64h", "op": "decode", "dtype": BF16, "heads": 64, "latent": 512,
         "rows": 64, "lens": "lognormal", "lo": 0, "hi": 32768, "shape_seed": 7},
        # Four long contexts, 128 heads: as much arithmetic as bytes.
        {"name": "latent_long_128h", "op": "decode", "dtype": BF16, "heads": 128, "latent": 512,
         "rows": 4, "lens": "uniform", "lo": 32768, "hi": 32768, "shape_seed": 8},
        # A parity run in fp32, a smaller latent.
        {"name": "latent_f32", "op": "decode", "dtype": F32, "heads": 16, "latent": 256, "rows": 8,
         "lens": "uniform", "lo": 1, "hi": 4096, "shape_seed": 9},
        # One short question, expanded.
        {"name": "latent_prompt_one", "op": "prompt", "dtype": BF16, "heads": 32, "nope": 128, "rows": 1,
         "lo": 17, "hi": 17, "shape_seed": 10},
        # Documents of very different lengths.
        {"name": "latent_prompt_batch", "op": "prompt", "dtype": BF16, "heads": 32, "nope": 128,
         "rows": 16, "lo": 512, "hi": 4096, "shape_seed": 11},
        # One long prompt.
        {"name": "latent_prompt_long", "op": "prompt", "dtype": BF16, "heads": 32, "nope": 128,
         "rows": 1, "lo": 16384, "hi": 16384, "shape_seed": 12},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "append", "lappend", "decode", "decode", "decode", "prompt", "prompt"])
    seed = rng.randrange(1 << 30)
    if kind in ("append", "lappend"):
        decode = rng.random() < 0.4
        hi = MAX_POS if decode else _log_uniform(rng, 1, 8192)
        rows = _log_uniform(rng, 1, 512 if decode else max(1, min(128, 32768 // hi)))
        c = {"op": kind, "dtype": rng.choice([BF16, BF16, F32]), "interleaved": rng.random() < 0.5,
             "rows": rows, "decode": decode, "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi,
             "shape_seed": seed}
        if kind == "append":
            heads, kv_heads, dim = rng.choice([(4, 4, 64), (32, 8, 128), (64, 8, 128), (24, 2, 64),
                                               (12, 4, 128), (16, 1, 64), (7, 7, 128), (14, 2, 64)])
            c.update(cache=rng.choice([BF16, BF16, F32, E4M3, E5M2]), heads=heads, kv_heads=kv_heads,
                     dim=dim, rot=rng.choice([dim, dim, dim // 2, dim // 4]))
        else:
            c.update(heads=rng.choice([1, 5, 16, 32, 64, 128]), latent=rng.choice([256, 512, 512]))
        return c
    if kind == "decode":
        dtype = rng.choice([BF16, BF16, BF16, F32])
        heads = rng.choice([1, 8, 12, 16, 20, 32, 40, 64, 96, 128])
        latent = rng.choice([256, 512, 512])
        hi = _log_uniform(rng, 1, 32768 if dtype == BF16 else 4096)
        # Multiply-adds of rows full sequences: at most those of the largest listed case.
        cap = 4 * 32768 * 128 * 512 if dtype == BF16 else 8 * 4096 * 16 * 256
        rows = _log_uniform(rng, 1, max(1, min(256, int(cap / (hi * max(heads, 16) * latent)))))
        return {"op": "decode", "dtype": dtype, "heads": heads, "latent": latent, "rows": rows,
                "lens": rng.choice(["uniform", "uniform", "lognormal"]),
                "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi, "shape_seed": seed}
    dtype = rng.choice([BF16, BF16, BF16, F32])
    heads, nope = rng.choice([1, 4, 5, 16, 32, 40, 64]), rng.choice([64, 128, 128])
    hi = _log_uniform(rng, 1, 16384 if dtype == BF16 else 2048)
    cap = 16384 ** 2 * 32 * 128 // 2 if dtype == BF16 else 2048 ** 2 * 16 * 128
    while hi ** 2 * heads * nope > cap:
        hi = hi * 7 // 8
    rows = _log_uniform(rng, 1, max(1, min(96, 65536 // hi, cap // (hi ** 2 * heads * nope))))
    return {"op": "prompt", "dtype": dtype, "heads": heads, "nope": nope, "rows": rows,
            "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi, "shape_seed": seed}


def _lengths(case):
    r = np.random.RandomState(case["shape_seed"])
    n, lo, hi = case["rows"], case["lo"], case["hi"]
    if case.get("lens", "uniform") == "uniform":
        got = r.randint(lo, hi + 1, n)
    else:
        got = np.clip(np.round(min(2048, hi) * np.exp(0.8 * r.standard_normal(n))), lo, hi)
    if not got.any():
        got[0] = hi
    return got.astype(np.int64)


def _new_tokens(case):
    """Tokens that an append writes."""
    return case["rows"] if case["decode"] else int(_lengths(case).sum())


def _positions_met(case):
    lens = _lengths(case)
    if case["decode"]:
        return len(set(np.minimum(lens, MAX_POS - 1).tolist()))
    return int(lens.max())


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "append":
        n, d = _new_tokens(case), case["dim"]
        turned = n * (case["heads"] + case["kv_heads"]) * case["rot"] // 2
        return {"bytes": n * (2 * case["heads"] * d * b + 2 * case["kv_heads"] * d * (b + BYTES[case["cache"]])
                              + 12) + _positions_met(case) * case["rot"] * 4, "flops": 6 * turned}
    if case["op"] == "lappend":
        n = _new_tokens(case)
        row = case["latent"] + ROPE
        return {"bytes": n * (2 * row * b + 2 * case["heads"] * ROPE * b + 12) + _positions_met(case) * ROPE * 4,
                "flops": 6 * n * (case["heads"] + 1) * ROPE // 2}
    lens = _lengths(case)
    if case["op"] == "decode":
        h, r = case["heads"], case["latent"]
        tokens = int(lens.sum())
        return {"bytes": tokens * (r + ROPE) * b + int(((lens + PAGE - 1) // PAGE).sum()) * 4
                + case["rows"] * (h * (2 * r + ROPE) * b + 4), "flops": 2 * tokens * h * (2 * r + ROPE)}
    h, d = case["heads"], case["nope"]
    tokens, pairs = int(lens.sum()), int((lens * (lens + 1) // 2).sum())
    return {"bytes": tokens * (h * (4 * d + ROPE) + ROPE) * b + 4 * (case["rows"] + 1),
            "flops": 2 * pairs * h * (2 * d + ROPE)}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    return {"append": _prepare_append, "lappend": _prepare_append, "decode": _prepare_decode,
            "prompt": _prepare_prompt}[case["op"]](case, seed, dev, g)


def _table(rot, dev):
    """cos and sin of every position's angles, made in 64 bits as a model's start does."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    angle = torch.arange(MAX_POS, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _slots(case, seed):
    """Positions of the new tokens, their slots in a pool whose pages lie anywhere, the pool's pages."""
    r = np.random.RandomState(seed % (1 << 32))
    lens = _lengths(case)
    if case["decode"]:
        pos = np.minimum(lens, MAX_POS - 1)
        pages = case["rows"] + 8
        places = r.permutation(pages)[:case["rows"]].astype(np.int64)
        return pos, places * PAGE + pos % PAGE, pages
    held = (lens + PAGE - 1) // PAGE
    pages = int(held.sum()) + 8
    places = r.permutation(pages).astype(np.int64)
    first = np.cumsum(held) - held
    pos = np.concatenate([np.arange(n) for n in lens])
    row = np.repeat(np.arange(len(lens)), lens)
    return pos, places[first[row] + pos // PAGE] * PAGE + pos % PAGE, pages


def _prepare_append(case, seed, dev, g):
    pos, slots, pages = _slots(case, seed)
    T, h, dtype = len(pos), case["heads"], TORCH[case["dtype"]]
    s = {"case": case, "positions": torch.from_numpy(pos.astype(np.int32)).to(dev),
         "slots": torch.from_numpy(slots).to(dev)}
    if case["op"] == "append":
        hk, d = case["kv_heads"], case["dim"]
        qkv = torch.randn((T, h + 2 * hk, d), generator=g, device=dev).to(dtype)
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        s["q_out"] = torch.zeros((T, h, d), dtype=dtype, device=dev)
        for name in ("k_cache", "v_cache"):
            s[name] = torch.zeros((pages, hk, d, PAGE), device=dev).to(TORCH[case["cache"]])
        s["table"] = _table(case["rot"], dev)
    else:
        r = case["latent"]
        row = torch.randn((T, r + ROPE), generator=g, device=dev).to(dtype)
        s["latent"], s["k_rope"] = row[:, :r], row[:, r:]
        q = torch.randn((T, h, 128 + ROPE), generator=g, device=dev).to(dtype)
        s["q_rope"] = q[..., 128:]
        # The rotated part of the queries in the latent space, behind the part that a product fills.
        s["q_out"] = torch.zeros((T, h, r + ROPE), dtype=dtype, device=dev)[..., r:]
        s["cache"] = torch.zeros((pages, PAGE, r + ROPE), dtype=dtype, device=dev)
        s["table"] = _table(ROPE, dev)
    return s


def _prepare_decode(case, seed, dev, g):
    r = np.random.RandomState(seed % (1 << 32))
    lens, dtype = _lengths(case), TORCH[case["dtype"]]
    held = (lens + PAGE - 1) // PAGE
    pages = int(held.sum()) + max(8, int(held.sum()) // 10)
    places = r.permutation(pages).astype(np.int32)
    tables = np.full((case["rows"], max(1, int(held.max()))), -1, np.int32)
    at = 0
    for i, n in enumerate(held):
        tables[i, :n] = places[at:at + n]
        at += n
    h, row = case["heads"], case["latent"] + ROPE
    return {"case": case, "cache": torch.randn((pages, PAGE, row), generator=g, device=dev).to(dtype),
            "q": torch.randn((case["rows"], h, row), generator=g, device=dev).to(dtype),
            "tables": torch.from_numpy(tables).to(dev),
            "lens": torch.from_numpy(lens.astype(np.int32)).to(dev), "max_seq_len": int(lens.max()),
            "scale": 1.0 / math.sqrt(128 + ROPE),
            "out": torch.empty((case["rows"], h, case["latent"]), dtype=dtype, device=dev)}


def _prepare_prompt(case, seed, dev, g):
    lens, dtype = _lengths(case), TORCH[case["dtype"]]
    T, h, d = int(lens.sum()), case["heads"], case["nope"]
    q = torch.randn((T, h, d + ROPE), generator=g, device=dev).to(dtype)
    kv = torch.randn((T, h, 2 * d), generator=g, device=dev).to(dtype)  # the up-projection's rows
    row = torch.randn((T, 512 + ROPE), generator=g, device=dev).to(dtype)
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return {"case": case, "q": q, "k": kv[..., :d], "v": kv[..., d:], "k_rope": row[:, 512:],
            "q_start": torch.from_numpy(start).to(dev), "lens": [int(n) for n in lens],
            "max_q_len": int(lens.max()), "scale": 1.0 / math.sqrt(d + ROPE),
            "out": torch.empty((T, h, d), dtype=dtype, device=dev)}


# ------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import paged_kv_cache_225_gb300 as pkv
        if op == "append":
            scale = _kv_scale(s["case"])
            pkv.rope_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], s["k_cache"],
                            s["v_cache"], q_out=s["q_out"], interleaved=s["case"]["interleaved"],
                            k_scale=scale, v_scale=scale)
        elif op == "lappend":
            pkv.latent_append(s["latent"], s["k_rope"], s["positions"], s["table"], s["slots"], s["cache"],
                              q_rope=s["q_rope"], q_out=s["q_out"], interleaved=s["case"]["interleaved"])
        elif op == "decode":
            return pkv.latent_attn_decode(s["q"], s["cache"], s["tables"], s["lens"], s["scale"], s["out"],
                                          max_seq_len=s["max_seq_len"])
        else:
            return pkv.latent_prompt_attn(s["q"], s["k"], s["k_rope"], s["v"], s["q_start"], s["scale"],
                                          s["out"], max_q_len=s["max_q_len"])
        return _appended(s)
    if op == "append":
        _plain_append(s)
        return _appended(s)
    if op == "lappend":
        _plain_latent_append(s)
        return _appended(s)
    return _plain_decode(s) if op == "decode" else _plain_prompt(s)


def _appended(s):
    return {name: s[name] for name in ("q_out", "k_cache", "v_cache", "cache") if name in s}


def _kv_scale(case):
    return KV_SCALE if case["cache"] in MOST else 1.0


def _rotated(x, cos, sin, interleaved):
    """x [T, H, D] (32 or 64 bits) with its first dims turned by angles [T, 1, rot / 2]."""
    half = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    else:
        a, b = x[..., :half], x[..., half:2 * half]
    y = x.clone()
    first, second = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = first, second
    else:
        y[..., :half], y[..., half:2 * half] = first, second
    return y


def _angles(s, dtype):
    rows = s["table"][s["positions"].long()].to(dtype)[:, None]
    half = rows.shape[-1] // 2
    return rows[..., :half], rows[..., half:]


def _put(cache, block, offset, rows, kind, scale):
    """rows [T, H, D] into [N, H, D, 16] cells, rounded to the cache's type."""
    if kind in MOST:
        rows = (rows / scale).clamp(-MOST[kind], MOST[kind]).to(TORCH[kind])
        cache, rows = cache.view(torch.uint8), rows.view(torch.uint8)
    cache[block, :, :, offset] = rows.to(cache.dtype)


def _plain_append(s):
    c = s["case"]
    cos, sin = _angles(s, torch.float32)
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, c["interleaved"]))
    block, offset = s["slots"] // PAGE, s["slots"] % PAGE
    _put(s["k_cache"], block, offset, _rotated(s["k"].float(), cos, sin, c["interleaved"]), c["cache"],
         _kv_scale(c))
    _put(s["v_cache"], block, offset, s["v"].float(), c["cache"], _kv_scale(c))


def _plain_latent_append(s):
    c = s["case"]
    cos, sin = _angles(s, torch.float32)
    s["q_out"].copy_(_rotated(s["q_rope"].float(), cos, sin, c["interleaved"]))
    key = _rotated(s["k_rope"].float()[:, None], cos, sin, c["interleaved"])[:, 0]
    s["cache"][s["slots"] // PAGE, s["slots"] % PAGE] = torch.cat([s["latent"], key.to(s["latent"].dtype)], 1)


def _plain_decode(s):
    """All sequences at once, over as many pages as the longest has."""
    c, lens = s["case"], s["lens"]
    rows = s["cache"][s["tables"].clamp(min=0)]                       # [S, pages, 16, R + 64]
    rows = rows.view(c["rows"], -1, rows.shape[-1]).float()
    x = torch.matmul(s["q"].float(), rows.transpose(1, 2)) * s["scale"]
    seen = torch.arange(rows.shape[1], device=x.device)[None, None, :] < lens[:, None, None]
    x = torch.where(seen, x, -math.inf)
    e = torch.where(seen, torch.exp(x - x.amax(dim=-1, keepdim=True)), 0.0)
    o = torch.matmul(e, rows[..., :c["latent"]]) / e.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    s["out"].copy_(o)
    return s["out"]


def _plain_prompt(s):
    """Per sequence, and per block of its rows so that the scores fit."""
    c, out, at = s["case"], s["out"], 0
    h, d = c["heads"], c["nope"]
    for n in s["lens"]:
        if not n:
            continue
        r = slice(at, at + n)
        q = s["q"][r].float().permute(1, 0, 2)                                           # [h, n, d + 64]
        k = torch.cat([s["k"][r].float(), s["k_rope"][r].float()[:, None].expand(n, h, ROPE)], 2).permute(1, 0, 2)
        v = s["v"][r].float().permute(1, 0, 2)
        step = max(1, min(n, (1 << 28) // (h * n)))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            x = torch.matmul(q[:, lo:hi], k[:, :hi].transpose(1, 2)) * s["scale"]
            cols = torch.arange(hi, device=x.device)
            x = torch.where(cols[None, :] <= cols[lo:hi, None], x, -math.inf)
            e = torch.exp(x - x.amax(dim=-1, keepdim=True))
            o = torch.matmul(e, v[:, :hi]) / e.sum(dim=-1, keepdim=True)
            out[at + lo:at + hi] = o.permute(1, 0, 2)
        at += n
    return out


# ------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "lappend": _exact_append, "decode": _exact_decode,
            "prompt": _exact_prompt}[case["op"]](case, s)


def _turn(x, table, pos, interleaved):
    """The rotation as complex products."""
    x = x.double()
    half = table.shape[1] // 2
    w = torch.complex(table[pos, :half].double(), table[pos, half:].double())[:, None]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    pairs = head.unflatten(-1, (half, 2)) if interleaved else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * w)
    z = z if interleaved else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), rest], -1)


def _exact_append(case, s):
    pos, slots = s["positions"].long(), s["slots"]
    if case["op"] == "lappend":
        got = {"q_out": _turn(s["q_rope"], s["table"], pos, case["interleaved"])}
        cells = torch.zeros((s["cache"].shape[0] * PAGE, s["cache"].shape[2]), dtype=torch.float64,
                            device=slots.device)
        cells[slots, :case["latent"]] = s["latent"].double()
        cells[slots, case["latent"]:] = _turn(s["k_rope"][:, None], s["table"], pos, case["interleaved"])[:, 0]
        got["cache"] = cells.view(s["cache"].shape)
        return got
    got = {"q_out": _turn(s["q"], s["table"], pos, case["interleaved"])}
    for name, rows in (("k_cache", _turn(s["k"], s["table"], pos, case["interleaved"])),
                       ("v_cache", s["v"].double())):
        n, hk, d, _ = s[name].shape
        rows = rows / _kv_scale(case)
        if case["cache"] in MOST:
            rows = rows.clamp(-MOST[case["cache"]], MOST[case["cache"]])
        cells = torch.zeros((n * PAGE, hk, d), dtype=torch.float64, device=slots.device)
        cells[slots] = rows
        got[name] = cells.view(n, PAGE, hk, d).permute(0, 2, 3, 1).contiguous()
    return got


def _exact_decode(case, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    tables = s["tables"].long()
    for i, n in enumerate(int(x) for x in _lengths(case)):
        if n:
            rows = s["cache"][tables[i, :-(-n // PAGE)]].flatten(0, 1)[:n].double()
            p = torch.softmax(rows @ s["q"][i].double().T * s["scale"], dim=0)
            out[i] = p.T @ rows[:, :case["latent"]]
    return out


def _exact_prompt(case, s):
    lens = _lengths(case)
    d = case["nope"]
    if float((lens.astype(np.float64) ** 2).sum()) * case["heads"] * (2 * d + ROPE) * 2 > 1.2e13:
        return None
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    at = 0
    for n in (int(x) for x in lens):
        r = slice(at, at + n)
        shared = s["k_rope"][r].double()
        for h in range(case["heads"]):
            q, k, v = s["q"][r, h].double(), s["k"][r, h].double(), s["v"][r, h].double()
            for lo in range(0, n, 4096):
                hi = min(n, lo + 4096)
                x = (q[lo:hi, :d] @ k[:hi].T + q[lo:hi, d:] @ shared[:hi].T) * s["scale"]
                x[:, lo:].masked_fill_(torch.ones((hi - lo, hi - lo), dtype=torch.bool, device=x.device).triu(1),
                                       -math.inf)
                out[at + lo:at + hi, h] = torch.softmax(x, dim=1) @ v[:hi]
        at += n
    return out
