"""Block tables, slots and reference counts built on the GPU (pkv_tables_step,
pkv_tables_fork) against a row-after-row model and against the host block
manager, exactly; and the pipeline they feed."""
import heapq
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_225_gb300 as pkv

from prompt_util import reference, tolerance

DEV = torch.device("cuda", 0)
OOR, NO_BLOCKS = 4, 7


def pages(n):
    return -(-n // 16)


class Model:
    """The pool as lists, one row after another."""

    def __init__(self, S, width, N):
        self.table, self.lens, self.ref = [[] for _ in range(S)], [0] * S, np.zeros(N, np.int64)
        self.width = width

    def drop(self, drop):
        for s, d in enumerate(drop):
            self.lens[s] -= min(d, self.lens[s])
            while len(self.table[s]) > pages(self.lens[s]):
                self.ref[self.table[s].pop()] -= 1

    def reserve(self, new, max_tokens):
        S = len(self.lens)
        slots, pairs = np.full(max_tokens, -1, np.int64), np.full((S, 2), -1, np.int32)
        if sum(new) > max_tokens or any(pages(a + b) > self.width for a, b in zip(self.lens, new)):
            return OOR, [0] * (S + 1), slots, pairs
        ref, heap = self.ref.copy(), [int(p) for p in np.flatnonzero(self.ref == 0)]
        table, at, starts = [list(t) for t in self.table], 0, [0]
        try:
            for s, n in enumerate(new):
                L = self.lens[s]
                if n and L % 16 and ref[table[s][-1]] > 1:
                    src = table[s][-1]
                    ref[src] -= 1
                    table[s][-1] = heapq.heappop(heap)
                    ref[table[s][-1]] = 1
                    pairs[s] = src, table[s][-1]
                while len(table[s]) < pages(L + n):
                    table[s].append(heapq.heappop(heap))
                    ref[table[s][-1]] = 1
                for t in range(L, L + n):
                    slots[at] = table[s][t // 16] * 16 + t % 16
                    at += 1
                starts.append(at)
        except IndexError:
            return NO_BLOCKS, [0] * (S + 1), np.full(max_tokens, -1, np.int64), np.full((S, 2), -1, np.int32)
        self.table, self.ref = table, ref
        self.lens = [a + b for a, b in zip(self.lens, new)]
        return 0, starts, slots, pairs

    def fork(self, parent, child):
        self.table[child], self.lens[child] = list(self.table[parent]), self.lens[parent]
        for p in self.table[child]:
            self.ref[p] += 1


class Pool:
    def __init__(self, S, width, N, max_tokens):
        i32 = dict(dtype=torch.int32, device=DEV)
        self.lens, self.ref = torch.zeros(S, **i32), torch.zeros(N, **i32)
        self.tables = torch.full((S, width), -1, **i32)
        self.q_start = torch.full((S + 1,), 77, **i32)
        self.slots = torch.full((max_tokens,), 77, dtype=torch.int64, device=DEV)
        self.pairs = torch.full((S, 2), 77, **i32)
        self.status = torch.zeros(1, **i32)

    def i32(self, a):
        return None if a is None else torch.tensor(a, dtype=torch.int32, device=DEV)

    def step(self, drop=None, new=None, **kw):
        self.status.zero_()
        args = dict(q_start=self.q_start, slot_mapping=self.slots, copy_pairs=self.pairs)
        args.update(kw)
        pkv.tables_step(self.lens, self.tables, self.ref, drop_lens=self.i32(drop),
                        new_lens=self.i32(new), status=self.status, **args)
        return int(self.status)

    def fork(self, pairs):
        self.status.zero_()
        pkv.tables_fork(self.i32(pairs).view(-1, 2), self.lens, self.tables, self.ref,
                        status=self.status)
        return int(self.status)

    def same(self, m):
        assert self.lens.tolist() == m.lens
        assert np.array_equal(self.ref.cpu().numpy(), m.ref)
        t = self.tables.cpu().numpy()
        for s, row in enumerate(m.table):
            assert t[s, :len(row)].tolist() == row and (t[s, len(row):] == -1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("S,N,width,max_tokens,seed", [
    (1, 1, 1, 16, 0), (3, 7, 4, 60, 1), (8, 40, 8, 300, 2), (37, 500, 12, 2000, 3),
    (64, 3001, 60, 6000, 4), (130, 20000, 300, 20000, 5), (600, 9000, 40, 60000, 6),
])
def test_random_steps(S, N, width, max_tokens, seed):
    r = np.random.RandomState(seed)
    m, g = Model(S, width, N), Pool(S, width, N, max_tokens)
    for it in range(40):
        kind = r.randint(4)
        if kind == 0 and S > 1:                     # forks of live rows into free ones
            free = [s for s in range(S) if m.lens[s] == 0]
            live = [s for s in range(S) if m.lens[s] > 0]
            if free and live:
                pairs = [(int(r.choice(live)), c) for c in free[:r.randint(1, len(free) + 1)]]
                assert g.fork(pairs) == 0
                for a, b in pairs:
                    m.fork(a, b)
                g.same(m)
        drop = [int(x) for x in r.randint(0, 40, S)] if kind != 1 else [0] * S
        for s in range(S):
            if r.rand() < 0.15:
                drop[s] = 1 << 30
        most = [1, 3, 20, 16 * width // 2][r.randint(4)]
        new = [int(x) for x in r.randint(0, most + 1, S)]
        m.drop(drop)
        st, q_start, slots, pairs = m.reserve(new, max_tokens)
        assert g.step(drop, new) == st
        assert g.q_start.tolist() == q_start
        assert np.array_equal(g.slots.cpu().numpy(), slots)
        assert np.array_equal(g.pairs.cpu().numpy(), pairs)
        g.same(m)


@pytest.mark.gpu
def test_same_pages_as_the_host_block_manager():
    r = np.random.RandomState(11)
    S, N, width = 24, 260, 32
    bm, g = pkv.BlockManager(N), Pool(S, width, N, 4096)
    lens = [0] * S
    for it in range(60):
        # Requests end, prompts come in one after another, then each row a token.
        ended = [s for s in range(S) if lens[s] and (r.rand() < 0.1 or lens[s] > 16 * width - 2)]
        free = [s for s in range(S) if lens[s] == 0]
        for s in ended:
            bm.free(s)
            lens[s] = 0
        came = [0] * S
        for s in free:
            if r.rand() < 0.4:
                n = int(r.randint(1, 150))
                if pages(n) + 2 * S < bm.num_free():
                    bm.add(s, n)
                    came[s] = n
        assert g.step([(1 << 30) if s in ended else 0 for s in range(S)], came) == 0
        lens = [a + b for a, b in zip(lens, came)]
        for s in [s for s in range(S) if lens[s] == 0 and s not in ended][:2]:
            live = [x for x in range(S) if lens[x]]
            if live and r.rand() < 0.7:
                p = int(r.choice(live))
                bm.fork(p, s)
                assert g.fork([(p, s)]) == 0
                lens[s] = lens[p]
        ids = [s for s in range(S) if 0 < lens[s] < 16 * width]
        if bm.num_free() < len(ids):
            continue
        slots, pairs = bm.append(ids) if ids else (np.empty(0, np.int64), np.empty((0, 2), np.int32))
        assert g.step(None, [1 if s in ids else 0 for s in range(S)]) == 0
        lens = [n + (s in ids) for s, n in enumerate(lens)]
        assert np.array_equal(g.slots.cpu().numpy()[:len(ids)], slots)
        got = g.pairs.cpu().numpy()
        assert np.array_equal(got[got[:, 0] >= 0], pairs)
        live = [s for s in range(S) if lens[s]]
        if live:
            t, n = bm.tables(live, width)
            assert np.array_equal(g.tables.cpu().numpy()[live], t)
            assert np.array_equal(g.lens.cpu().numpy()[live], n)
        assert int((g.ref == 0).sum()) == bm.num_free()


@pytest.mark.gpu
def test_too_few_pages_leaves_the_rows_alone():
    g = Pool(3, 8, 10, 200)
    assert g.step(None, [40, 40, 20]) == 0                       # 3 + 3 + 2 pages
    lens, tables, ref = g.lens.clone(), g.tables.clone(), g.ref.clone()
    assert g.step(None, [30, 1, 30]) == NO_BLOCKS                # 2 + 0 + 2 more than the 2 left
    assert torch.equal(lens, g.lens) and torch.equal(tables, g.tables) and torch.equal(ref, g.ref)
    assert (g.q_start == 0).all() and (g.slots == -1).all() and (g.pairs == -1).all()
    # The drops of the same call stand, and make the room.
    assert g.step([0, 40, 0], [30, 0, 30]) == 0
    assert g.lens.tolist() == [70, 0, 50]


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["negative", "overflow", "huge", "tokens", "length", "page", "free_page",
                                  "no_pairs"])
def test_invalid_rows_stop_the_reservation(what):
    g = Pool(4, 8, 64, 100)
    assert g.step(None, [20, 33, 7, 0]) == 0
    if what == "no_pairs":
        assert g.fork([(2, 3)]) == 0
    new, kw = [1, 1, 1, 1], {}
    if what == "negative":
        new[1] = -1
    elif what == "overflow":
        new[1] = 128 - 33 + 1
    elif what == "huge":
        new[0] = (1 << 31) - 1
    elif what == "tokens":
        new = [30, 30, 30, 11]
    elif what == "length":
        g.lens[1] = 129
    elif what == "page":
        g.tables[1, 2] = 64
    elif what == "free_page":
        g.ref[g.tables[1, 2]] = 0
    elif what == "no_pairs":
        kw["copy_pairs"] = None
        g.pairs.fill_(-1)
    lens, tables, ref = g.lens.clone(), g.tables.clone(), g.ref.clone()
    assert g.step(None, new, **kw) == OOR
    assert torch.equal(lens, g.lens) and torch.equal(tables, g.tables) and torch.equal(ref, g.ref)
    assert (g.q_start == 0).all() and (g.slots == -1).all() and (g.pairs == -1).all()


@pytest.mark.gpu
def test_bad_drops_are_reported_and_skipped():
    g = Pool(3, 8, 64, 200)
    assert g.step(None, [64, 64, 64]) == 0
    g.tables[0, 1] = 64                          # outside the pool
    g.tables[0, 2] = -5
    g.ref[g.tables[1, 0]] = 0                    # held by nobody
    free = int((g.ref == 0).sum())
    assert g.step([1 << 30, 1 << 30, -3], None) == OOR
    assert g.lens.tolist() == [0, 0, 64] and (g.tables[:2] == -1).all()
    assert int((g.ref == 0).sum()) == free + 2 + 3 and int(g.ref.min()) == 0
    g.lens[2] = -1
    assert g.step([0, 0, 5], None) == OOR
    assert g.lens.tolist() == [0, 0, -1]


@pytest.mark.gpu
def test_outputs_may_be_left_out():
    g = Pool(3, 8, 64, 100)
    assert g.step(None, [20, 0, 3], q_start=None, copy_pairs=None) == 0
    assert g.lens.tolist() == [20, 0, 3] and (g.q_start == 77).all() and (g.pairs == 77).all()
    assert g.step([5, 0, 3], None, q_start=None, copy_pairs=None, slot_mapping=None) == 0
    assert g.lens.tolist() == [15, 0, 0] and int((g.ref > 0).sum()) == 1
    assert g.step(None, None) == 0
    assert (g.q_start == 0).all() and (g.slots == -1).all() and (g.pairs == -1).all()
    # Tokens asked for without a place for their slots.
    assert g.step(None, [1, 0, 0], slot_mapping=None) == OOR


@pytest.mark.gpu
def test_no_rows():
    i32 = dict(dtype=torch.int32, device=DEV)
    q, slots = torch.full((1,), 7, **i32), torch.full((5,), 7, dtype=torch.int64, device=DEV)
    pkv.tables_step(torch.zeros(0, **i32), torch.zeros((0, 4), **i32), torch.zeros(8, **i32),
                    q_start=q, slot_mapping=slots)
    assert int(q) == 0 and (slots == -1).all()


@pytest.mark.gpu
def test_forks_that_are_refused():
    g = Pool(6, 8, 64, 200)
    assert g.step(None, [40, 20, 0, 0, 0, 0]) == 0
    ref = g.ref.clone()
    for bad in ([(6, 2)], [(0, 6)], [(-1, 2)], [(0, -1)], [(0, 0)], [(0, 1)]):
        assert g.fork(bad) == OOR
        assert g.lens.tolist() == [40, 20, 0, 0, 0, 0] and torch.equal(ref, g.ref)
    assert g.fork([(-1, -1), (-1, -1)]) == 0
    # A child listed twice: the first pair counts.  A child that is a parent too: not forked.
    assert g.fork([(0, 2), (1, 2), (1, 3), (2, 4)]) == OOR
    assert g.lens.tolist() == [40, 20, 0, 20, 0, 0]
    assert g.fork([(0, 2), (1, 2)]) == OOR
    assert g.lens.tolist() == [40, 20, 40, 20, 0, 0]
    assert g.tables[2, :3].tolist() == g.tables[0, :3].tolist()
    # A bad page of the parent is not shared.
    g.tables[1, 0] = 99
    assert g.fork([(1, 4)]) == OOR
    assert g.tables[4].tolist()[:2] == [-1, int(g.tables[1, 1])] and int(g.lens[4]) == 20
    g.lens[5] = -2
    assert g.fork([(0, 5)]) == OOR


@pytest.mark.gpu
def test_last_holder_writes_in_place():
    g = Pool(4, 4, 20, 20)
    assert g.step(None, [20, 0, 0, 0]) == 0
    assert g.fork([(0, 1), (0, 2), (0, 3)]) == 0
    assert g.step(None, [1, 1, 1, 1]) == 0
    # Pages 0, 1 are the prompt's; rows 0 .. 2 copy page 1, row 3 keeps it.
    assert g.pairs.tolist() == [[1, 2], [1, 3], [1, 4], [-1, -1]]
    assert g.tables[:, 1].tolist() == [2, 3, 4, 1] and g.ref[:5].tolist() == [4, 1, 1, 1, 1]
    # A page the caller counts as its own is never written in place.
    g2 = Pool(2, 4, 20, 20)
    assert g2.step(None, [20, 0]) == 0
    g2.ref[1] += 1
    assert g2.step(None, [2, 0]) == 0
    assert g2.pairs.tolist() == [[1, 2], [-1, -1]] and g2.ref[:3].tolist() == [1, 1, 1]


@pytest.mark.gpu
def test_most_rows():
    S, N = 8192, 40000
    m, g = Model(S, 6, N), Pool(S, 6, N, 1 << 17)
    r = np.random.RandomState(9)
    for _ in range(3):
        drop, new = [int(x) for x in r.randint(0, 30, S)], [int(x) for x in r.randint(0, 24, S)]
        m.drop(drop)
        st, q_start, slots, pairs = m.reserve(new, 1 << 17)
        assert g.step(drop, new) == st == 0
        assert g.q_start.tolist() == q_start and np.array_equal(g.slots.cpu().numpy(), slots)
        g.same(m)
    i32 = dict(dtype=torch.int32, device=DEV)
    with pytest.raises(pkv.PkvError) as e:
        pkv.tables_step(torch.zeros(S + 1, **i32), torch.zeros((S + 1, 4), **i32), torch.zeros(8, **i32))
    assert e.value.code == 2


@pytest.mark.gpu
def test_slots_past_32_bits():
    # A pool whose last pages' slots pass 2^31; nothing is allocated for them but the counts.
    N = (1 << 27) + 64
    i32 = dict(dtype=torch.int32, device=DEV)
    ref = torch.ones(N, **i32)
    ref[-8:] = 0
    lens, tables = torch.zeros(2, **i32), torch.full((2, 8), -1, **i32)
    slots, q_start = torch.zeros(70, dtype=torch.int64, device=DEV), torch.zeros(3, **i32)
    pkv.tables_step(lens, tables, ref, new_lens=torch.tensor([20, 40], **i32), q_start=q_start,
                    slot_mapping=slots)
    want = [(N - 8) * 16 + t for t in range(20)] + [(N - 6) * 16 + t for t in range(40)] + [-1] * 10
    assert slots.tolist() == want and int((ref == 0).sum()) == 3


def _dense(pool, cache, s, n):
    """Rows 0 .. n-1 of row s read through the table: [n, Hkv, D]."""
    t = torch.arange(n, device=DEV)
    page = pool.tables[s, (t // 16).long()].long()
    return cache[page, :, :, (t % 16).long()]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_serving_loop(dtype):
    """Prompts in, forks, then decode steps replayed from a graph: tables, copies, cache write,
    whole-prompt and paged attention together, against dense attention over each row's tokens."""
    Hq, Hkv, D, S, N, width = 8, 2, 64, 6, 64, 8
    scale = 1 / math.sqrt(D)
    g = torch.Generator(device=DEV).manual_seed(3)
    pool = Pool(S, width, N, 256)
    kc = torch.full((N, Hkv, D, 16), float("nan"), dtype=dtype, device=DEV)
    vc = kc.clone()
    prompt = [37, 0, 64, 0, 5, 0]
    T = sum(prompt)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv].contiguous(), qkv[:, Hq + Hkv:].contiguous()
    assert pool.step(None, prompt) == 0
    pkv.reshape_and_cache(k, v, pool.slots[:T], kc, vc)
    out = torch.zeros((T, Hq, D), dtype=dtype, device=DEV)
    pkv.prompt_attn(q, k, v, pool.q_start, scale, out, max_q_len=64)
    ref, mass, most = reference(q, k, v, prompt, scale)
    assert bool(((out.double() - ref).abs()
                 <= tolerance(ref, mass, most, prompt, D, scale, dtype, dtype)).all())
    hist = {}
    at = 0
    for s, n in enumerate(prompt):
        hist[s] = (k[at:at + n], v[at:at + n])
        at += n
    assert pool.fork([(0, 1), (0, 3), (2, 5)]) == 0
    for a, b in ((0, 1), (0, 3), (2, 5)):
        hist[b] = hist[a]

    # One decode step, captured once.
    new = torch.ones(S, dtype=torch.int32, device=DEV)
    slots = torch.zeros(S, dtype=torch.int64, device=DEV)
    dq = torch.zeros((S, Hq, D), dtype=dtype, device=DEV)
    dk, dv = (torch.zeros((S, Hkv, D), dtype=dtype, device=DEV) for _ in range(2))
    dout = torch.zeros((S, Hq, D), dtype=torch.float32, device=DEV)
    ws = torch.empty(pkv.workspace_size(S, Hq, Hkv, D, width * 16), dtype=torch.uint8, device=DEV)

    def step():
        pkv.tables_step(pool.lens, pool.tables, pool.ref, new_lens=new, q_start=pool.q_start,
                        slot_mapping=slots, copy_pairs=pool.pairs, status=pool.status)
        pkv.copy_blocks(kc, vc, pool.pairs)
        pkv.reshape_and_cache(dk, dv, slots, kc, vc)
        pkv.paged_attn_decode(dq, kc, vc, pool.tables, pool.lens, scale, dout, workspace=ws)

    graph = None
    for it in range(20):
        dq.copy_(torch.randn(dq.shape, generator=g, device=DEV))
        dk.copy_(torch.randn(dk.shape, generator=g, device=DEV))
        dv.copy_(torch.randn(dv.shape, generator=g, device=DEV))
        if graph is None:
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(pool.status) == 0 and pkv.read_status(ws) == 0
        for s in range(S):
            hist[s] = (torch.cat([hist[s][0], dk[s:s + 1]]), torch.cat([hist[s][1], dv[s:s + 1]]))
            n = hist[s][0].shape[0]
            assert int(pool.lens[s]) == n
            # A dense read through the table gives the row's own tokens, bit for bit.
            assert torch.equal(_dense(pool, kc, s, n), hist[s][0])
            assert torch.equal(_dense(pool, vc, s, n), hist[s][1])
            kk, vv = (x.double().repeat_interleave(Hq // Hkv, 1) for x in hist[s])
            p = torch.softmax(torch.einsum("hd,nhd->hn", dq[s].double(), kk) * scale, -1)
            want = torch.einsum("hn,nhd->hd", p, vv)
            assert float((dout[s].double() - want).abs().max()) <= (1e-5 if dtype == torch.float32 else 4e-3)
    # Retiring every row empties the pool.
    assert pool.step([1 << 30] * S, None) == 0
    assert int(pool.ref.abs().sum()) == 0 and (pool.tables == -1).all()


@pytest.mark.gpu
def test_slots_on_an_8_byte_boundary():
    g = Pool(5, 20, 120, 600)
    buf = torch.full((603,), 77, dtype=torch.int64, device=DEV)
    m = Model(5, 20, 120)
    for new in ([33, 0, 7, 128, 1], [1, 1, 1, 1, 1], [0, 250, 0, 3, 16]):
        st, q_start, slots, pairs = m.reserve(new, 601)
        assert g.step(None, new, slot_mapping=buf[1:602]) == st == 0
        assert np.array_equal(buf[1:602].cpu().numpy(), slots)
        assert int(buf[0]) == 77 and int(buf[602]) == 77
        g.same(m)


@pytest.mark.gpu
def test_two_pools_at_once():
    # Two pools on two streams, the steps captured in two graphs and replayed side by side.
    pools, graphs = [Pool(64, 40, 2000, 4096) for _ in range(2)], []
    new = [torch.full((64,), n, dtype=torch.int32, device=DEV) for n in (3, 7)]
    drop = [torch.full((64,), n, dtype=torch.int32, device=DEV) for n in (1, 2)]
    torch.cuda.synchronize()
    for p, n, d in zip(pools, new, drop):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.tables_step(p.lens, p.tables, p.ref, drop_lens=d, new_lens=n, q_start=p.q_start,
                            slot_mapping=p.slots, copy_pairs=p.pairs, status=p.status)
        graphs.append((graph, torch.cuda.Stream()))
    for _ in range(30):
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for p, n, d in zip(pools, (3, 7), (1, 2)):
        m = Model(64, 40, 2000)
        for _ in range(30):
            m.drop([d] * 64)
            st, q_start, slots, _ = m.reserve([n] * 64, 4096)
            assert st == 0
        assert int(p.status) == 0 and p.q_start.tolist() == q_start
        assert np.array_equal(p.slots.cpu().numpy(), slots)
        p.same(m)
