"""The rotating cache writes (pkv_rope_append, pkv_latent_append): bit for bit
against element-wise f32 arithmetic followed by the plain cache write, and
against the rotation in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_225_gb300 as pkv

from latent_util import ROPE, rope_table, rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16
E4M3, E5M2, INT4 = torch.float8_e4m3fn, torch.float8_e5m2, torch.uint8
CACHES = [F32, BF16, E4M3, E5M2, INT4]
SCALE = 0.0625
MAX_POS = 5000


def raw(t):
    return t.contiguous().view(torch.uint8)


def cache_like(N, H, D, dtype, seed):
    """A cache that holds something everywhere, so that a write too many shows."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (N, H, D, 8 if dtype == INT4 else 16)
    c = torch.randint(0, 100, shape, generator=g, device=DEV)
    return c.to(torch.uint8) if dtype == INT4 else c.float().to(dtype)


def slots_of(pattern, seed):
    """(slots int64, pages): where the tokens of a call go."""
    r = np.random.RandomState(seed)
    if pattern == "one":
        return np.array([37]), 4
    if pattern == "decode":
        N = 150
        return r.permutation(N)[:130].astype(np.int64) * 16 + r.randint(0, 16, 130), N
    if pattern == "order":                     # two pages, tokens in falling order, then pages interleaved
        return np.concatenate([np.arange(31, -1, -1), 32 + np.arange(32).reshape(2, 16).T.reshape(-1)]), 5
    lens = {"pages": [16] * 9, "ragged": [1, 300, 0, 17, 64, 5, 128, 33], "padded": [40, 100, 3],
            "chunk": [70, 81, 9]}[pattern]
    first = [5, 15, 1] if pattern == "chunk" else [0] * len(lens)  # chunks start inside a page
    N = sum(-(-(f + n) // 16) for f, n in zip(first, lens)) + 3
    places, at, got = r.permutation(N), 0, []
    for f, n in zip(first, lens):
        t = np.arange(f, f + n)
        got.append(places[at + t // 16] * 16 + t % 16)
        at += -(-(f + n) // 16)
    got = np.concatenate(got).astype(np.int64)
    if pattern == "padded":                    # padding between and behind, inside pages too
        got[[0, 20, 21, 47, 90]] = -1
        got = np.concatenate([got, np.full(30, -1)])
    return got, N


def case(pattern, Hq, Hkv, D, dtype, seed, fused=True):
    slots, N = slots_of(pattern, seed)
    T = len(slots)
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, MAX_POS, (T,), generator=g, device=DEV, dtype=torch.int32)
    return q, k, v, pos, torch.from_numpy(slots).to(DEV), N


def check(q, k, v, pos, slots, N, rot, cache, interleaved, in_place=False, skip=None):
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    table = rope_table(MAX_POS, rot, DEV)
    kc, vc = cache_like(N, Hkv, D, cache, 1), cache_like(N, Hkv, D, cache, 2)
    want_k, want_v = kc.clone(), vc.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept = torch.full_like(q.contiguous(), 7.0)
    q_in = q.clone()
    out = pkv.rope_append(q, k, v, pos, table, slots, kc, vc, q_out=None if in_place else kept,
                          interleaved=interleaved, k_scale=SCALE, v_scale=2 * SCALE, status=status)
    torch.cuda.synchronize()
    assert out is (q if in_place else kept)
    good = slots >= 0
    if skip is not None:
        good &= ~skip
    assert int(status) == (0 if skip is None else 4)
    k32 = rotate(k, table, torch.where(good, pos, 0), interleaved, F32)
    pkv.reshape_and_cache(k32, v.float().contiguous(), torch.where(good, slots, -1), want_k, want_v, k_scale=SCALE,
                          v_scale=2 * SCALE)
    assert torch.equal(raw(kc), raw(want_k))
    assert torch.equal(raw(vc), raw(want_v))
    turned = rotate(q_in, table, torch.where(good, pos, 0), interleaved, F32).to(q.dtype)
    want = torch.where(good[:, None, None], turned, q_in if in_place else torch.full_like(q_in, 7.0))
    assert torch.equal(raw(out), raw(want))
    # Against 64 bits: two products and a sum, each off by 2^-24, of values up to |a| + |b|; one rounding.
    exact = rotate(q_in, table, torch.where(good, pos, 0), interleaved, torch.float64)[good]
    size = q_in.double()[good].abs().amax(-1, keepdim=True)
    last = 2.0 ** -8 if q.dtype == BF16 else 2.0 ** -24
    assert bool(((out[good].double() - exact).abs() <= 6 * 2.0 ** -24 * size + last * exact.abs()).all())
    return kc, vc


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("pattern", ["one", "decode", "pages", "ragged", "padded", "chunk", "order"])
def test_patterns(pattern, cache, dtype):
    check(*case(pattern, 6, 2, 128, dtype, 3), 128, cache, False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 32), (64, 48), (64, 64), (128, 16), (128, 64), (128, 96), (128, 128)])
def test_rotations(D, rot, interleaved, dtype):
    check(*case("ragged", 5, 3, D, dtype, rot), rot, BF16 if rot % 32 else E4M3, interleaved)
    check(*case("decode", 5, 3, D, dtype, rot), rot, F32, interleaved, in_place=True)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (7, 7), (64, 8), (33, 11), (130, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(Hq, Hkv, D):
    check(*case("ragged", Hq, Hkv, D, BF16, Hq), D, BF16, False)
    check(*case("one", Hq, Hkv, D, BF16, Hq), D, INT4, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_in_place(dtype):
    q, k, v, pos, slots, N = case("ragged", 4, 2, 64, dtype, 5)
    unit = 16 // q.element_size()
    buf = torch.randn(len(pos) * (4 * 64 + 3 * unit) + unit, device=DEV).to(dtype)
    q2 = torch.as_strided(buf, q.shape, (4 * 64 + 3 * unit, 64, 1), unit)
    q2.copy_(q)
    before = buf.clone()
    check(q2, k, v, pos, slots, N, 32, BF16, False, in_place=True)
    gaps = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(gaps, q.shape, q2.stride(), unit).fill_(False)
    assert torch.equal(buf[gaps], before[gaps])
    check(q, k.contiguous(), v, pos, slots, N, 64, E5M2, True, in_place=True)


def test_no_queries_and_no_tokens():
    q, k, v, pos, slots, N = case("ragged", 4, 2, 64, BF16, 8)
    table = rope_table(MAX_POS, 64, DEV)
    a = [cache_like(N, 2, 64, BF16, i) for i in (1, 2)]
    b = [c.clone() for c in a]
    assert pkv.rope_append(None, k, v, pos, table, slots, *a) is None
    pkv.rope_append(q, k, v, pos, table, slots, *b, q_out=torch.empty_like(q))
    assert all(torch.equal(raw(x), raw(y)) for x, y in zip(a, b))
    none = slots[:0]
    before = [c.clone() for c in a]
    pkv.rope_append(q[:0], k[:0], v[:0], pos[:0], table, none, *a)
    pkv.latent_append(torch.empty((0, 256), device=DEV), torch.empty((0, 64), device=DEV), pos[:0], table, none,
                      torch.empty((2, 16, 320), device=DEV))
    torch.cuda.synchronize()
    assert all(torch.equal(raw(x), raw(y)) for x, y in zip(a, before))


@pytest.mark.parametrize("what", ["slot", "huge_slot", "position", "negative_position"])
def test_tokens_out_of_range_are_reported_and_skipped(what):
    q, k, v, pos, slots, N = case("ragged", 4, 2, 64, BF16, 9)
    skip = torch.zeros(len(pos), dtype=torch.bool, device=DEV)
    skip[[3, 100]] = True
    if "slot" in what:
        slots[skip] = N * 16 if what == "slot" else 1 << 62
    else:
        pos[skip] = MAX_POS if what == "position" else -1
    check(q, k, v, pos, slots, N, 64, BF16, False, skip=skip)


def test_slots_past_32_bits():
    # Cells past 2^31 elements and 2^32 bytes.
    H, D, N = 8, 128, 140000
    kc, vc = (torch.zeros((N, H, D, 16), dtype=BF16, device=DEV) for _ in range(2))
    table = rope_table(MAX_POS, D, DEV)
    T = 40
    g = torch.Generator(device=DEV).manual_seed(4)
    k, v = (torch.randn((T, H, D), generator=g, device=DEV).to(BF16) for _ in range(2))
    slots = torch.arange(T, device=DEV) + (N - 3) * 16
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    pkv.rope_append(None, k, v, pos, table, slots, kc, vc)
    got = kc[N - 3:].permute(0, 3, 1, 2).reshape(-1, H, D)[:T]
    assert torch.equal(raw(got), raw(rotate(k, table, pos, False, F32).to(BF16)))
    assert torch.equal(raw(vc[N - 3:].permute(0, 3, 1, 2).reshape(-1, H, D)[:T]), raw(v))
    assert not bool(kc[:N - 3].any())


# ------------------------------------------------------------ latent rows

def latent_case(pattern, R, H, dtype, seed):
    slots, N = slots_of(pattern, seed)
    T = len(slots)
    g = torch.Generator(device=DEV).manual_seed(seed)
    row = torch.randn((T, R + ROPE), generator=g, device=DEV).to(dtype)
    q = torch.randn((T, H, 128 + ROPE), generator=g, device=DEV).to(dtype)
    pos = torch.randint(0, MAX_POS, (T,), generator=g, device=DEV, dtype=torch.int32)
    return row[:, :R], row[:, R:], q[..., 128:], pos, torch.from_numpy(slots).to(DEV), N


@pytest.mark.parametrize("dtype,cache", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("pattern", ["one", "decode", "ragged", "padded", "order"])
@pytest.mark.parametrize("R,H,interleaved", [(512, 16, True), (256, 5, False), (512, 128, False), (256, 0, True)])
def test_latent_rows(R, H, interleaved, pattern, dtype, cache):
    latent, key, q, pos, slots, N = latent_case(pattern, R, max(H, 1), dtype, R + H)
    table = rope_table(MAX_POS, ROPE, DEV)
    c = torch.full((N, 16, R + ROPE), 3.0, dtype=cache, device=DEV)
    want = c.clone()
    q_abs = torch.full((len(pos), max(H, 1), R + ROPE), 5.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = q.clone()
    got = pkv.latent_append(latent, key, pos, table, slots, c, q_rope=q if H else None,
                            q_out=q_abs[..., R:] if H else None, interleaved=interleaved, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    good = slots >= 0
    rows = torch.cat([latent.float(), rotate(key[:, None], table, pos, interleaved, F32)[:, 0]], 1).to(cache)
    want.view(-1, R + ROPE)[slots[good]] = rows[good]
    assert torch.equal(raw(c), raw(want))
    assert bool((q_abs[..., :R] == 5).all())
    if H:
        turned = rotate(before, table, pos, interleaved, F32).to(dtype)
        assert torch.equal(raw(got), raw(torch.where(good[:, None, None], turned, torch.full_like(turned, 5.0))))
        pkv.latent_append(latent, key, pos, table, slots, c, q_rope=q, interleaved=interleaved)  # in place
        assert torch.equal(raw(q), raw(torch.where(good[:, None, None], turned, before)))
    else:
        assert got is None


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_latent_queries_one_head_after_the_other(dtype):
    latent, key, q, pos, slots, N = latent_case("ragged", 256, 6, dtype, 21)
    table = rope_table(MAX_POS, ROPE, DEV)
    c = torch.zeros((N, 16, 320), dtype=dtype, device=DEV)
    q = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = torch.zeros((6, len(pos), ROPE), dtype=dtype, device=DEV).permute(1, 0, 2)
    pkv.latent_append(latent, key, pos, table, slots, c, q_rope=q, q_out=out)
    assert torch.equal(raw(out), raw(rotate(q, table, pos, False, F32).to(dtype)))


def test_latent_rows_out_of_range_and_far():
    R, N = 512, 240000                                # 2.2 * 10^9 numbers
    latent, key, q, pos, slots, _ = latent_case("ragged", R, 4, BF16, 11)
    table = rope_table(MAX_POS, ROPE, DEV)
    c = torch.zeros((N, 16, R + ROPE), dtype=BF16, device=DEV)
    T = len(pos)
    slots = torch.arange(T, device=DEV) + N * 16 - T + 2   # the last two lie past the pool
    pos[5] = MAX_POS
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.zeros((T, 4, ROPE), dtype=BF16, device=DEV)
    pkv.latent_append(latent, key, pos, table, slots, c, q_rope=q, q_out=out, status=status)
    assert int(status) == 4
    good = torch.ones(T, dtype=torch.bool, device=DEV)
    good[[5, T - 2, T - 1]] = False
    flat = c.view(-1, R + ROPE)
    rows = torch.cat([latent, rotate(key[:, None], table, pos.clamp(max=MAX_POS - 1), False, F32)[:, 0].to(BF16)], 1)
    assert torch.equal(raw(flat[slots[good]]), raw(rows[good]))
    assert not bool(flat[slots[5]].any()) and not bool(out[~good].any()) and bool(out[good].any())
    assert not bool(flat[:N * 16 - T + 2].any())


def test_streams_graphs_and_two_calls_at_once():
    q, k, v, pos, slots, N = case("ragged", 8, 2, 128, BF16, 13)
    table = rope_table(MAX_POS, 128, DEV)
    a = [cache_like(N, 2, 128, BF16, i) for i in (1, 2)]
    b, c = [x.clone() for x in a], [x.clone() for x in a]
    oa, ob, oc = (torch.zeros_like(q.contiguous()) for _ in range(3))
    pkv.rope_append(q, k, v, pos, table, slots, *a, q_out=oa)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.rope_append(q, k, v, pos, table, slots, *b, q_out=ob, stream=side)
    pkv.rope_append(q, k, v, pos, table, slots, *c, q_out=oc, stream=other)
    torch.cuda.synchronize()
    for x, y in ((oa, ob), (oa, oc), *zip(a, b), *zip(a, c)):
        assert torch.equal(raw(x), raw(y))
    graph = torch.cuda.CUDAGraph()
    for x in c:
        x.zero_()
    with torch.cuda.graph(graph):
        pkv.rope_append(q, k, v, pos, table, slots, *c, q_out=oc)
    q.mul_(0.5)
    pkv.rope_append(q, k, v, pos, table, slots, *a, q_out=oa)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(raw(oa), raw(oc)) and bool(c[0].any())


def test_queries_in_place_with_other_strides_are_refused():
    q, k, v, pos, slots, N = case("ragged", 4, 2, 64, BF16, 17, fused=False)
    table = rope_table(MAX_POS, 64, DEV)
    caches = [cache_like(N, 2, 64, BF16, i) for i in (1, 2)]
    before = [c.clone() for c in caches]
    T = len(pos)
    wide = torch.zeros((T, 8, 64), dtype=BF16, device=DEV)
    wide[:] = 1.0
    dense = wide.view(-1)[:T * 4 * 64].view(T, 4, 64)     # at wide's address
    for a, b in ((wide[:, :4], dense), (dense, wide[:, :4])):
        with pytest.raises(pkv.PkvError):
            pkv.rope_append(a, k, v, pos, table, slots, *caches, q_out=b)
    row = torch.randn((T, 256 + ROPE), device=DEV).to(BF16)
    cache = torch.zeros((N, 16, 256 + ROPE), dtype=BF16, device=DEV)
    heads = wide.view(-1)[:T * 4 * 64].view(4, T, 64).permute(1, 0, 2)
    for a, b in ((wide[:, :4], dense), (dense, heads), (heads, dense)):
        with pytest.raises(pkv.PkvError):
            pkv.latent_append(row[:, :256], row[:, 256:], pos, table, slots, cache, q_rope=a, q_out=b)
    torch.cuda.synchronize()
    assert bool((wide == 1).all()) and not bool(cache.any())
    assert all(torch.equal(raw(x), raw(y)) for x, y in zip(caches, before))
    # One token has no stride: the same call, which turns it where it lies.
    one = q[:1].clone()
    want = rotate(one, table, pos[:1], False, F32).to(BF16)
    got = pkv.rope_append(wide[:1, :4].copy_(one), k[:1], v[:1], pos[:1], table, slots[:1], *caches, q_out=dense[:1])
    assert torch.equal(raw(got), raw(want))


@pytest.mark.parametrize("cache", CACHES)
def test_a_replayed_graph_writes_what_a_call_writes(cache):
    q, k, v, pos, slots, N = case("padded", 8, 2, 128, BF16, 18)
    table = rope_table(MAX_POS, 128, DEV)
    a = [cache_like(N, 2, 128, cache, i) for i in (1, 2)]
    b = [x.clone() for x in a]
    oa, ob = (torch.zeros_like(q.contiguous()) for _ in range(2))
    scales = dict(k_scale=SCALE, v_scale=2 * SCALE)
    warm = [x.clone() for x in a]
    pkv.rope_append(q, k, v, pos, table, slots, *warm, q_out=ob, **scales)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.rope_append(q, k, v, pos, table, slots, *b, q_out=ob, **scales)
    # Other rows, positions and slots than at the capture.
    k.mul_(0.5)
    v.mul_(-0.5)
    q.mul_(0.25)
    pos.copy_((pos + 7) % MAX_POS)
    slots.copy_(torch.where(slots >= 0, slots ^ 16, slots))
    pkv.rope_append(q, k, v, pos, table, slots, *a, q_out=oa, **scales)
    ob.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(raw(oa), raw(ob))
    good = slots >= 0
    turned = rotate(k, table, pos, False, F32)
    want = [cache_like(N, 2, 128, cache, i) for i in (1, 2)]
    pkv.reshape_and_cache(turned, v.float().contiguous(), slots, *want, **scales)
    for x, y, z in zip(a, b, want):
        assert torch.equal(raw(x), raw(y)) and torch.equal(raw(x), raw(z))
    assert bool(good.any())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_replayed_graph_writes_the_latent_rows_of_a_call(dtype):
    latent, key, q, pos, slots, N = latent_case("padded", 512, 5, dtype, 19)
    table = rope_table(MAX_POS, ROPE, DEV)
    a, b = (torch.full((N, 16, 576), 3.0, dtype=dtype, device=DEV) for _ in range(2))
    oa, ob = (torch.zeros((len(pos), 5, ROPE), dtype=dtype, device=DEV) for _ in range(2))
    pkv.latent_append(latent, key, pos, table, slots, a.clone(), q_rope=q, q_out=ob)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.latent_append(latent, key, pos, table, slots, b, q_rope=q, q_out=ob)
    latent.mul_(0.5)
    key.mul_(-2.0)
    pos.copy_((pos + 7) % MAX_POS)
    slots.copy_(torch.where(slots >= 0, slots ^ 16, slots))
    pkv.latent_append(latent, key, pos, table, slots, a, q_rope=q, q_out=oa)
    ob.zero_()
    graph.replay()
    torch.cuda.synchronize()
    good = slots >= 0
    want = torch.full_like(a, 3.0)
    rows = torch.cat([latent.float(), rotate(key[:, None], table, pos, False, F32)[:, 0]], 1).to(dtype)
    want.view(-1, 576)[slots[good]] = rows[good]
    assert torch.equal(raw(oa), raw(ob)) and torch.equal(raw(a), raw(b)) and torch.equal(raw(b), raw(want))
