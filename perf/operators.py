"""Measured calls of the whole-prompt attention and of the device block tables.

Three operators, each in a plain form (elementary torch operations) and, with
``own`` set, as the calls a user makes of this library:

  prompt  prompt_attn: causal attention over whole prompts, packed one after
          another, with grouped heads.  Row i of a sequence attends its rows
          0 .. i.
  step    tables_step: one scheduling step of a paged cache kept on the GPU.
          Every row drops its last drop_lens tokens (pages that nobody holds any
          more return to the pool), then reserves new_lens tokens: block tables,
          lengths, reference counts, packed row starts and cache slots.
  fork    tables_fork: rows that start as copies of others and share their
          pages, followed by the step in which each of them takes a token, which
          gives it a page of its own (copy on write).

A pass of `step` and of `fork` drops what it reserved the time before, so that
every pass does the same work on the same state.
"""
import heapq
import math

import numpy as np
import torch

own = False

PAGE = 16
F32, BF16 = "f32", "bf16"
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
BYTES = {F32: 4, BF16: 2}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # The smallest layer: four short prompts, fp32, one KV head per query head.
        {"name": "prompt_tiny_f32", "op": "prompt", "dtype": F32, "heads": 4, "kv_heads": 4,
         "dim": 64, "fused": False, "rows": 4, "lens": "uniform", "lo": 1, "hi": 64,
         "shape_seed": 1},
        # One short question to an idle 8B server: the latency of a single call.
        {"name": "prompt_one_8b", "op": "prompt", "dtype": BF16, "heads": 32, "kv_heads": 8,
         "dim": 128, "fused": True, "rows": 1, "lens": "uniform", "lo": 17, "hi": 17,
         "shape_seed": 2},
        # A full chat batch of the 70B layer, every prompt 256 to 512 tokens.
        {"name": "prompt_chat_70b", "op": "prompt", "dtype": BF16, "heads": 64, "kv_heads": 8,
         "dim": 128, "fused": True, "rows": 128, "lens": "uniform", "lo": 256, "hi": 512,
         "shape_seed": 3},
        # Documents of very different lengths through the 8B layer.
        {"name": "prompt_batch_8b", "op": "prompt", "dtype": BF16, "heads": 32, "kv_heads": 8,
         "dim": 128, "fused": True, "rows": 16, "lens": "uniform", "lo": 512, "hi": 4096,
         "shape_seed": 4},
        # One prompt that fills the 32K context.
        {"name": "prompt_long_8b", "op": "prompt", "dtype": BF16, "heads": 32, "kv_heads": 8,
         "dim": 128, "fused": False, "rows": 1, "lens": "uniform", "lo": 32768, "hi": 32768,
         "shape_seed": 5},
        # Twelve query heads per KV head of dimension 64, ragged, some rows empty.
        {"name": "prompt_odd_groups", "op": "prompt", "dtype": BF16, "heads": 24, "kv_heads": 2,
         "dim": 64, "fused": True, "rows": 37, "lens": "uniform", "lo": 0, "hi": 1000,
         "shape_seed": 6},
        # The 8B layer in fp32, as a parity run uses it.
        {"name": "prompt_batch_f32", "op": "prompt", "dtype": F32, "heads": 32, "kv_heads": 8,
         "dim": 128, "fused": True, "rows": 8, "lens": "uniform", "lo": 256, "hi": 1024,
         "shape_seed": 7},
        # Speculative decoding of 128 requests: the four drafts of the last step
        # were rejected, four new ones and the token itself are reserved.
        {"name": "step_verify_128", "op": "step", "rows": 128, "lens": "lognormal", "lo": 16,
         "hi": 32768, "new_lo": 5, "new_hi": 5, "chunks": 0, "chunk": 0, "whole": False,
         "others": 0.1, "shape_seed": 8},
        # A batch of prompts leaves and the next one comes in.
        {"name": "step_admit_64", "op": "step", "rows": 64, "lens": "uniform", "lo": 512,
         "hi": 4096, "new_lo": 0, "new_hi": 0, "chunks": 0, "chunk": 0, "whole": True,
         "others": 0.3, "shape_seed": 9},
        # A large server: 512 requests, one token each but for 24 prompt chunks,
        # in a pool that other requests fragment.
        {"name": "step_mixed_512", "op": "step", "rows": 512, "lens": "lognormal", "lo": 16,
         "hi": 32768, "new_lo": 1, "new_hi": 1, "chunks": 24, "chunk": 2000, "whole": False,
         "others": 2.0, "shape_seed": 10},
        # Eight answers to each of 16 chat prompts.
        {"name": "fork_chat_16x8", "op": "fork", "rows": 16, "children": 7, "lens": "uniform",
         "lo": 256, "hi": 512, "others": 0.2, "shape_seed": 11},
        # Thirty-two beams over each of eight long contexts.
        {"name": "fork_long_8x32", "op": "fork", "rows": 8, "children": 31, "lens": "uniform",
         "lo": 8192, "hi": 32767, "others": 0.2, "shape_seed": 12},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "prompt", "step", "step", "fork"])
    seed = rng.randrange(1 << 30)
    if kind == "prompt":
        heads, kv_heads, dim = rng.choice([(4, 4, 64), (32, 8, 128), (64, 8, 128), (8, 8, 64),
                                           (24, 2, 64), (40, 8, 128), (12, 4, 128), (16, 1, 64),
                                           (16, 1, 128), (96, 8, 64), (14, 2, 64)])
        dtype = rng.choice([BF16, BF16, BF16, F32])
        hi = _log_uniform(rng, 1, 32768 if dtype == BF16 else 4096)
        # Multiply-adds of rows full sequences, at most half of the longest listed case.
        cap = 16384 ** 2 * 32 * 128 if dtype == BF16 else 4096 ** 2 * 32 * 128
        most = max(1, int(cap / (hi ** 2 * heads * dim)))
        most = max(1, min(most, 160, 131072 // hi))
        while hi ** 2 * heads * dim > cap:
            hi = hi * 7 // 8
        return {"op": "prompt", "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "fused": rng.random() < 0.6, "rows": _log_uniform(rng, 1, most),
                "lens": "uniform", "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi,
                "shape_seed": seed}
    if kind == "step":
        rows = _log_uniform(rng, 1, 512)
        whole = rng.random() < 0.3
        hi = _log_uniform(rng, 16, 4096 if whole else 32768)
        new = rng.choice([1, 1, 2, 5, 9])
        chunks = 0 if whole else rng.choice([0, 0, min(rows, 24), min(rows, 3)])
        return {"op": "step", "rows": min(rows, 128) if whole else rows,
                "lens": rng.choice(["uniform", "lognormal"]), "lo": min(hi, rng.choice([0, 1, 16])),
                "hi": hi, "new_lo": rng.choice([0, new]), "new_hi": new, "chunks": chunks,
                "chunk": rng.randrange(100, 2000) if chunks else 0, "whole": whole,
                "others": rng.choice([0.0, 0.1, 0.5, 2.0]), "shape_seed": seed}
    rows = _log_uniform(rng, 1, 64)
    return {"op": "fork", "rows": rows, "children": _log_uniform(rng, 1, max(1, 256 // rows)),
            "lens": "uniform", "lo": 1, "hi": _log_uniform(rng, 16, 32767),
            "others": rng.choice([0.0, 0.2, 1.0]), "shape_seed": seed}


def _lengths(case):
    r = np.random.RandomState(case["shape_seed"])
    n, lo, hi = case["rows"], case["lo"], case["hi"]
    if case["lens"] == "uniform":
        got = r.randint(lo, hi + 1, n)
    else:
        got = np.clip(np.round(2048 * np.exp(0.8 * r.standard_normal(n))), lo, hi).astype(np.int64)
    if case["op"] == "prompt" and not got.any():
        got[0] = max(1, hi)
    return got.astype(np.int64), r


def _step_counts(case):
    """Lengths before a step's tokens, and the tokens each row reserves."""
    lens, r = _lengths(case)
    if case["whole"]:
        return np.zeros_like(lens), lens
    new = r.randint(case["new_lo"], case["new_hi"] + 1, case["rows"]).astype(np.int64)
    at = r.permutation(case["rows"])[:case["chunks"]]
    new[at] = case["chunk"]
    return lens, new


def work(case):
    lens, _ = _lengths(case)
    if case["op"] == "prompt":
        tokens = int(lens.sum())
        pairs = int((lens * (lens + 1) // 2).sum())
        rows = 2 * case["heads"] + 2 * case["kv_heads"]
        return {"bytes": tokens * rows * case["dim"] * BYTES[case["dtype"]] + 4 * (case["rows"] + 1),
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "step":
        kept, new = _step_counts(case)
        pages = _pages(kept + new) - _pages(kept)
        n = case["rows"]
        # The reference counts once; per page taken and per page dropped a table entry and a
        # count; slots, row starts, lengths, counts asked for, copy pairs.
        return {"bytes": 4 * _pool(case) + int(pages.sum()) * 2 * 12 + 8 * int(new.sum())
                + 4 * (n + 1) + 8 * n + 8 * n + 8 * n, "flops": 0}
    pages = _pages(lens)
    n, kids = case["rows"], case["children"]
    # Each parent's table row once; per child its row written, and read when dropped, and the
    # counts of the parent's pages; the reference counts; slots and pairs.
    return {"bytes": 4 * _pool(case) + int(pages.sum()) * 4 * (1 + 2 * kids + 4)
            + n * (kids + 1) * 40, "flops": 0}


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _pool(case):
    """Pages of the case's pool: what its rows hold at most, what others hold, and a slack."""
    if case["op"] == "step":
        kept, new = _step_counts(case)
        mine = int(_pages(kept + new).sum())
    else:
        lens, _ = _lengths(case)
        mine = int(_pages(lens).sum()) + case["rows"] * case["children"]
    return mine + int(mine * case["others"]) + max(8, mine // 10)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    if case["op"] == "prompt":
        return _prepare_prompt(case, seed, dev)
    return _prepare_tables(case, seed, dev)


def _prepare_prompt(case, seed, dev):
    lens, _ = _lengths(case)
    T, hq, hk, d = int(lens.sum()), case["heads"], case["kv_heads"], case["dim"]
    g = torch.Generator(device=dev).manual_seed(seed)
    dtype = TORCH[case["dtype"]]
    qkv = torch.randn((T, hq + 2 * hk, d), generator=g, device=dev).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return {"case": case, "q": q, "k": k, "v": v, "q_start": torch.from_numpy(start).to(dev),
            "lens": [int(n) for n in lens], "max_q_len": int(lens.max()),
            "scale": 1.0 / math.sqrt(d), "out": torch.empty((T, hq, d), dtype=dtype, device=dev)}


def _layout(case, seed):
    """A pool with the rows' pages (and other owners') at random places, on the host."""
    r = np.random.RandomState(seed % (1 << 32))
    pool = _pool(case)
    if case["op"] == "step":
        kept, new = _step_counts(case)
        lens = kept + new          # the rows still hold what the pass drops first
        rows, drop = case["rows"], new
    else:
        parents, _ = _lengths(case)
        rows = case["rows"] * (case["children"] + 1)
        lens = np.zeros(rows, np.int64)
        lens[:case["rows"]] = parents
        new = np.zeros(rows, np.int64)
        new[case["rows"]:] = 1
        drop = np.zeros(rows, np.int64)
        drop[case["rows"]:] = 1 << 30
    places = r.permutation(pool)
    pages = _pages(lens)
    # Room in the tables: the longest row, and in a fork the token that its children add.
    width = int(pages.max()) + 1
    tables = np.full((rows, width), -1, np.int32)
    at = 0
    for s in range(rows):
        n = int(pages[s])
        tables[s, :n] = places[at:at + n]
        at += n
    ref = np.zeros(pool, np.int32)
    ref[places[:at]] = 1
    mine = at
    others = int(mine * case["others"])
    ref[places[at:at + others]] = r.randint(1, 4, min(others, pool - at))
    return {"tables": tables, "lens": lens.astype(np.int32), "ref": ref,
            "drop": drop.astype(np.int32), "new": new.astype(np.int32)}


def _prepare_tables(case, seed, dev):
    h = _layout(case, seed)
    s = {name: torch.from_numpy(a).to(dev) for name, a in h.items()}
    rows, tokens = h["lens"].size, max(1, int(h["new"].sum()))
    s["case"] = case
    s["q_start"] = torch.zeros(rows + 1, dtype=torch.int32, device=dev)
    s["slots"] = torch.zeros(tokens, dtype=torch.int64, device=dev)
    s["pairs"] = torch.full((rows, 2), -1, dtype=torch.int32, device=dev)
    if case["op"] == "fork":
        n, kids = case["rows"], case["children"]
        p = np.stack([np.repeat(np.arange(n), kids), n + np.arange(n * kids)], 1).astype(np.int32)
        s["forks"] = torch.from_numpy(p).to(dev)
    return s


# ------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        import paged_kv_cache_225_gb300 as pkv
        s = state
        if op == "prompt":
            return pkv.prompt_attn(s["q"], s["k"], s["v"], s["q_start"], s["scale"], s["out"],
                                   max_q_len=s["max_q_len"])
        if op == "step":
            pkv.tables_step(s["lens"], s["tables"], s["ref"], drop_lens=s["drop"],
                            new_lens=s["new"], q_start=s["q_start"], slot_mapping=s["slots"],
                            copy_pairs=s["pairs"])
        else:
            pkv.tables_step(s["lens"], s["tables"], s["ref"], drop_lens=s["drop"])
            pkv.tables_fork(s["forks"], s["lens"], s["tables"], s["ref"])
            pkv.tables_step(s["lens"], s["tables"], s["ref"], new_lens=s["new"],
                            q_start=s["q_start"], slot_mapping=s["slots"],
                            copy_pairs=s["pairs"])
        return _outputs(s)
    if op == "prompt":
        return _plain_prompt(state)
    if op == "step":
        _plain_drop(state)
        _plain_reserve(state)
    else:
        _plain_drop(state)
        _plain_fork(state)
        _plain_reserve(state)
    return _outputs(state)


def _outputs(s):
    return {"q_start": s["q_start"], "slots": s["slots"], "pairs": s["pairs"],
            "lens": s["lens"], "tables": s["tables"], "ref": s["ref"]}


def _plain_prompt(s):
    """Per sequence, and per block of its rows so that the scores fit: scores, mask, softmax,
    product, all in 32 bits."""
    c, out = s["case"], s["out"]
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    g = hq // hk
    at = 0
    for n in s["lens"]:
        if not n:
            continue
        q = s["q"][at:at + n].float().view(n, hk, g, d).permute(1, 2, 0, 3)      # [hk, g, n, d]
        k = s["k"][at:at + n].float().permute(1, 0, 2)[:, None]                   # [hk, 1, n, d]
        v = s["v"][at:at + n].float().permute(1, 0, 2)[:, None]
        step = max(1, min(n, (1 << 28) // (hq * n)))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            x = torch.matmul(q[:, :, lo:hi], k[:, :, :hi].transpose(2, 3)) * s["scale"]
            cols = torch.arange(hi, device=x.device)
            x = torch.where(cols[None, :] <= cols[lo:hi, None], x, -math.inf)
            e = torch.exp(x - x.amax(dim=-1, keepdim=True))
            o = torch.matmul(e, v[:, :, :hi]) / e.sum(dim=-1, keepdim=True)
            out[at + lo:at + hi] = o.permute(2, 0, 1, 3).reshape(hi - lo, hq, d).to(out.dtype)
        at += n
    return out


def _plain_drop(s):
    tables, ref, lens = s["tables"], s["ref"], s["lens"]
    kept = lens - torch.minimum(s["drop"], lens)
    col = torch.arange(tables.shape[1], device=lens.device)[None, :]
    gone = (col >= _pages(kept)[:, None]) & (col < _pages(lens)[:, None])
    ref.index_add_(0, torch.where(gone, tables, 0).view(-1), -gone.view(-1).to(torch.int32))
    tables.copy_(torch.where(gone, -1, tables))
    lens.copy_(kept)


def _plain_fork(s):
    tables, ref, lens = s["tables"], s["ref"], s["lens"]
    parent, child = s["forks"][:, 0].long(), s["forks"][:, 1].long()
    rows = tables[parent]
    held = torch.arange(tables.shape[1], device=lens.device)[None, :] < _pages(lens[parent])[:, None]
    ref.index_add_(0, torch.where(held, rows, 0).view(-1), held.view(-1).to(torch.int32))
    tables[child] = torch.where(held, rows, tables[child])
    lens[child] = lens[parent]


def _plain_reserve(s):
    tables, ref, lens = s["tables"], s["ref"], s["lens"]
    rows, width = tables.shape
    pool = ref.numel()
    dev = lens.device
    new = s["new"].long()
    old = lens.long()
    have = _pages(old)
    # A row whose last page is part full and shared takes a copy of it, but for the last
    # holder: row order decides who that is.
    last = tables.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long()
    grows = (new > 0) & (old % PAGE > 0)
    same = (last[:, None] == last[None, :]) & grows[None, :]
    before = torch.tril(same, -1).sum(dim=1)
    copies = grows & (ref[last.clamp(min=0)] - before > 1)
    first = have - copies.long()
    need = torch.where(new > 0, _pages(old + new) - first, 0)
    # Lowest free page first, in row order.
    free = ref == 0
    place = torch.where(free, torch.cumsum(free, 0) - 1, pool)
    listed_free = torch.zeros(pool + 1, dtype=torch.int64, device=dev)
    listed_free.scatter_(0, place, torch.arange(pool, device=dev))
    base = torch.cumsum(need, 0) - need
    ok = (need.sum() <= free.sum()).long()
    new, need, copies = new * ok, need * ok, copies & (ok > 0)
    col = torch.arange(width, device=dev)[None, :]
    fresh = (col >= first[:, None]) & (col < (first + need)[:, None])
    page = listed_free[(base[:, None] + col - first[:, None]).clamp(0, pool)]
    ref.index_add_(0, last.clamp(min=0), -copies.to(torch.int32))
    ref.index_add_(0, torch.where(fresh, page, 0).view(-1), fresh.view(-1).to(torch.int32))
    tables.copy_(torch.where(fresh, page, tables))
    dst = tables.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    s["pairs"][:, 0] = torch.where(copies, last, -1)
    s["pairs"][:, 1] = torch.where(copies, dst, -1)
    ends = torch.cumsum(new, 0)
    s["q_start"][0] = 0
    s["q_start"][1:] = ends
    i = torch.arange(s["slots"].numel(), device=dev)
    row = torch.searchsorted(ends, i, right=True).clamp(max=rows - 1)
    pos = old[row] + i - (ends - new)[row]
    slot = tables[row, (pos // PAGE).clamp(0, width - 1)].long() * PAGE + pos % PAGE
    s["slots"].copy_(torch.where(i < ends[-1], slot, -1))
    lens.copy_(old + new)


# ------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    if case["op"] == "prompt":
        return _exact_prompt(case, seed, dev)
    return _exact_tables(case, seed)


def _exact_prompt(case, seed, dev):
    s = _prepare_prompt(case, seed, dev)
    g = case["heads"] // case["kv_heads"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=dev)
    at = 0
    for n in s["lens"]:
        own_rows = slice(at, at + n)
        for h in range(case["heads"]):
            q, k, v = (s[x][own_rows, y].double() for x, y in
                       (("q", h), ("k", h // g), ("v", h // g)))
            for lo in range(0, n, 4096):
                hi = min(n, lo + 4096)
                p = q[lo:hi] @ k[:hi].T
                p.mul_(s["scale"])
                p[:, lo:].masked_fill_(torch.ones((hi - lo, hi - lo), dtype=torch.bool,
                                                  device=dev).triu(1), -math.inf)
                out[at + lo:at + hi, h] = torch.softmax(p, dim=1) @ v[:hi]
        at += n
    return out


def _exact_tables(case, seed):
    """The rows one after another, with a heap of free pages."""
    h = _layout(case, seed)
    table = [list(row[:n]) for row, n in zip(h["tables"], _pages(h["lens"]))]
    lens = [int(n) for n in h["lens"]]
    ref = h["ref"].copy()

    for s, d in enumerate(h["drop"]):
        lens[s] -= min(int(d), lens[s])
        while len(table[s]) > -(-lens[s] // PAGE):
            ref[table[s].pop()] -= 1
    if case["op"] == "fork":
        n, kids = case["rows"], case["children"]
        for i in range(n * kids):
            table[n + i], lens[n + i] = list(table[i // kids]), lens[i // kids]
            for p in table[n + i]:
                ref[p] += 1
    heap = [int(p) for p in np.flatnonzero(ref == 0)]
    heapq.heapify(heap)
    slots, starts = [], [0]
    pairs = np.full((len(lens), 2), -1, np.int32)
    for s, n in enumerate(int(x) for x in h["new"]):
        if n and lens[s] % PAGE and ref[table[s][-1]] > 1:
            src = table[s][-1]
            ref[src] -= 1
            table[s][-1] = heapq.heappop(heap)
            ref[table[s][-1]] += 1
            pairs[s] = src, table[s][-1]
        while len(table[s]) < -(-(lens[s] + n) // PAGE):
            table[s].append(heapq.heappop(heap))
            ref[table[s][-1]] += 1
        pos = np.arange(lens[s], lens[s] + n)
        slots.append(np.asarray(table[s], np.int64)[pos // PAGE] * PAGE + pos % PAGE
                     if n else np.empty(0, np.int64))
        lens[s] += n
        starts.append(starts[-1] + n)
    got = np.concatenate(slots)
    tables = np.full(h["tables"].shape, -1, np.int32)
    for s, row in enumerate(table):
        tables[s, :len(row)] = row
    all_slots = np.full(max(1, got.size), -1, np.int64)
    all_slots[:got.size] = got
    return {"q_start": np.asarray(starts, np.int32), "slots": all_slots, "pairs": pairs,
            "lens": np.asarray(lens, np.int32), "tables": tables, "ref": ref}
