"""Latent attention (pkv_latent_attn_decode, pkv_latent_prompt_attn) against the
formulas in 64 bits: lengths, heads, types, strides, what unseen places may hold,
scales, device-side reports, streams and graphs, and a serving run of all of it."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_225_gb300 as pkv

from latent_util import ROPE, decode_reference, pages_for, prompt_reference, rope_table, rotate
from prompt_util import tolerance

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16
NAN, INF = float("nan"), float("inf")


# ----------------------------------------------------------------- decode

def make(lens, H, R, dtype, seed, width=None):
    tables, N = pages_for(lens, seed, width=width)
    g = torch.Generator(device=DEV).manual_seed(seed)
    cache = torch.randn((N, 16, R + ROPE), generator=g, device=DEV).to(dtype)
    q = torch.randn((len(lens), H, R + ROPE), generator=g, device=DEV).to(dtype)
    return q, cache, torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def decode(q, cache, tables, lens, scale, want=0, **kw):
    out = torch.full((q.shape[0], q.shape[1], q.shape[2] - ROPE), NAN, dtype=q.dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.latent_attn_decode(q, cache, tables, lens, scale, out, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == want
    return out


def near(out, ref, mass, most, lens, dims, scale):
    tol = tolerance(ref, mass, most, [max(1, int(n)) for n in lens], dims, scale, out.dtype, out.dtype)
    off = (out.double() - ref).abs()
    assert not torch.isnan(off).any()
    assert bool((off <= tol).all()), f"worst {float((off / tol).max()):.3g} of the tolerance"


def check(q, cache, tables, lens, scale, **kw):
    out = decode(q, cache, tables, lens, scale, **kw)
    n = [int(x) for x in lens]
    ref, mass, most = decode_reference(q, cache, tables, n, scale)
    near(out, ref, mass, most, n, q.shape[2], scale)
    return out


SCALE = 1 / math.sqrt(192)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("lens", [[1], [0], [15], [16], [17], [63], [64], [65], [128], [129], [1000],
                                  [0, 0, 5, 0, 64, 0], [300, 1, 0, 2048, 77, 640, 16], [1] * 200,
                                  [64] * 160, [4097, 3, 5000]])
def test_lengths(lens, R, dtype):
    check(*make(lens, 16, R, dtype, sum(lens) + R), SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("H", [1, 2, 7, 15, 16, 17, 31, 32, 33, 40, 48, 63, 64, 65, 96, 100, 127, 128])
def test_heads(H, R, dtype):
    check(*make([150, 0, 3, 700], H, R, dtype, H + R), SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,n,H", [(1, 30000, 16), (2, 20001, 128), (3, 9999, 64), (300, 70, 32), (40, 513, 20)])
def test_long_and_many(S, n, H, dtype):
    # Ranges that cut one sequence often, and that hold many whole ones.
    check(*make([n] * S, H, 512, dtype, n), SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 3.0])
def test_scales(scale, dtype):
    check(*make([200, 90, 0, 1500], 24, 512, dtype, 7), scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_growing_and_falling_scores(sign, dtype):
    # The running maximum rises by far more than 2^8 again and again, or never after the first token.
    n, R = 3000, 512
    q, cache, tables, lens = make([n, 700], 20, R, dtype, 3)
    q.fill_(0.25)
    for s in range(2):
        ramp = torch.linspace(0, 4, int(lens[s]), device=DEV)
        at = tables[s, :-(-int(lens[s]) // 16)].long()
        rows = cache[at].view(-1, R + ROPE)
        rows[:int(lens[s])] = ((ramp if sign > 0 else ramp.flip(0))[:, None]
                               + 0.01 * rows[:int(lens[s])].float()).to(dtype)
        cache[at] = rows.view(-1, 16, R + ROPE)
    check(q, cache, tables, lens, 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("lens", [[1, 30, 77, 64, 500], [65, 79, 5, 1030]])
def test_unseen_places_may_hold_anything(lens, bad, dtype):
    q, cache, tables, lens_t = make(lens, 40, 512, dtype, 5)
    want = check(q, cache, tables, lens_t, SCALE)
    spoilt = torch.full_like(cache, bad)
    for s, n in enumerate(lens):
        at = tables[s, :-(-n // 16)].long()
        rows = spoilt[at].view(-1, 512 + ROPE)
        rows[:n] = cache[at].view(-1, 512 + ROPE)[:n]
        spoilt[at] = rows.view(-1, 16, 512 + ROPE)
    assert torch.equal(decode(q, spoilt, tables, lens_t, SCALE), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bad_values_reach_the_rows_that_see_them(dtype):
    lens, R = [100, 200, 50], 512
    q, cache, tables, lens_t = make(lens, 16, R, dtype, 6)
    ok = check(q, cache, tables, lens_t, SCALE)
    block = int(tables[1, 3])
    cache[block, 5, 40] = NAN
    out = decode(q, cache, tables, lens_t, SCALE)
    assert torch.isnan(out[1].float()).all()            # a NaN score: the whole row
    assert torch.equal(out[0], ok[0]) and torch.equal(out[2], ok[2])
    cache[block, 5, 40] = 0.0
    q[1, 3, 7] = INF
    out = decode(q, cache, tables, lens_t, SCALE)
    assert torch.isnan(out[1, 3].float()).all() and not torch.isnan(out[1, 4].float()).any()


def test_scores_of_minus_infinity():
    lens, R = [100, 300], 256
    q, cache, tables, lens_t = make(lens, 16, R, BF16, 8)
    q.fill_(1.0)
    cache[..., R] = -INF                                # every score -inf: nothing to weigh
    assert torch.isnan(decode(q, cache, tables, lens_t, SCALE).float()).all()
    cache[..., R] = 0.0
    seen = cache[tables[1].long()].view(-1, R + ROPE)   # a leading run of -inf, then tokens that count
    seen[:200, R] = -INF
    cache[tables[1].long()] = seen.view(-1, 16, R + ROPE)
    out = decode(q, cache, tables, lens_t, SCALE)
    p = torch.softmax(seen[200:300].double() @ q[1].double().T * SCALE, 0)
    ref = p.T @ seen[200:300, :R].double()
    assert float((out[1].double() - ref).abs().max()) < 0.02 * float(ref.abs().max())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bad_lengths_and_blocks_are_reported(dtype):
    lens = [100, 40, 300]
    q, cache, tables, lens_t = make(lens, 16, 512, dtype, 9)
    want = decode(q, cache, tables, lens_t, SCALE)
    wrong = lens_t.clone()
    wrong[1] = -5
    out = decode(q, cache, tables, wrong, SCALE, want=4, max_seq_len=300)
    assert not bool(out[1].any()) and torch.equal(out[0], want[0])
    wrong[1], wrong[2] = 40, 10 ** 9                    # clamped to 300
    out = decode(q, cache, tables, wrong, SCALE, want=4, max_seq_len=300)
    assert torch.equal(out, want)
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        holes = tables.clone()
        holes[0, 2] = bad
        out = decode(q, cache, holes, lens_t, SCALE, want=4)
        zero = torch.cat([cache, torch.zeros_like(cache[:1])])
        holes[0, 2] = cache.shape[0]
        assert torch.equal(out, decode(q, zero, holes, lens_t, SCALE))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bits_do_not_change(dtype):
    a = make([3000, 5, 0, 777, 1200], 32, 512, dtype, 10)
    first = decode(*a, SCALE)
    for _ in range(5):
        assert torch.equal(decode(*a, SCALE), first)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shared_pages_and_queries_of_one_sequence(dtype):
    # Four queries of one sequence: the same table row, a length each.
    q, cache, tables, lens = make([203], 16, 512, dtype, 11)
    n = torch.tensor([200, 201, 202, 203], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    q4 = torch.randn((4, 16, 576), generator=g, device=DEV).to(dtype)
    cache[int(tables[0, 12]), 9:] = cache[int(tables[0, 12]), 9:] * 3
    out = check(q4, cache, tables.expand(4, -1).contiguous(), n, SCALE)
    cache[int(tables[0, 12]), 10] = NAN                 # token 202: only the last query sees it
    again = decode(q4, cache, tables.expand(4, -1).contiguous(), n, SCALE)
    assert torch.equal(again[:3], out[:3]) and torch.isnan(again[3].float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_past_32_bits(dtype):
    R, N = 512, 240000                                  # 2.2 * 10^9 numbers
    cache = torch.zeros((N, 16, R + ROPE), dtype=dtype, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    cache[-40:] = torch.randn((40, 16, R + ROPE), generator=g, device=DEV).to(dtype)
    tables = torch.arange(N - 40, N, dtype=torch.int32, device=DEV).view(1, 40)
    q = torch.randn((1, 16, R + ROPE), generator=g, device=DEV).to(dtype)
    check(q, cache, tables, torch.tensor([635], dtype=torch.int32, device=DEV), SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wide_tables_and_loose_bounds(dtype):
    lens = [70, 0, 900]
    q, cache, tables, lens_t = make(lens, 24, 256, dtype, 12)
    want = decode(q, cache, tables, lens_t, SCALE, max_seq_len=900)
    wide = torch.full((3, 4000), -1, dtype=torch.int32, device=DEV)
    wide[:, :tables.shape[1]] = tables
    ref, mass, most = decode_reference(q, cache, tables, lens, SCALE)
    near(decode(q, cache, wide, lens_t, SCALE), ref, mass, most, lens, 320, SCALE)
    near(want, ref, mass, most, lens, 320, SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_streams_graphs_and_workspaces(dtype):
    a, b = make([900, 31, 2000], 32, 512, dtype, 13), make([400, 1700, 64], 32, 512, dtype, 14)
    want_a, want_b = decode(*a, SCALE), decode(*b, SCALE)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(want_a) for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(3):                                  # two calls at once, workspaces of their own
        pkv.latent_attn_decode(*a, SCALE, outs[0], stream=side)
        pkv.latent_attn_decode(*b, SCALE, outs[1], stream=other)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want_a) and torch.equal(outs[1], want_b)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, args, out in zip(graphs, (a, b), outs[2:]):
        with torch.cuda.graph(graph):
            pkv.latent_attn_decode(*args, SCALE, out)
    for out in outs:
        out.zero_()
    with torch.cuda.stream(side):
        graphs[0].replay()
    with torch.cuda.stream(other):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[2], want_a) and torch.equal(outs[3], want_b)
    a[3][0] = 17                                        # lengths are read at replay
    graphs[0].replay()
    torch.cuda.synchronize()
    n = [17, 31, 2000]
    ref, mass, most = decode_reference(a[0], a[1], a[2], n, SCALE)
    near(outs[2], ref, mass, most, n, 576, SCALE)
    need = pkv.latent_workspace_size(dtype, 3, 32, 512, 2000)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(decode(*b, SCALE, workspace=ws), want_b)
    with pytest.raises(pkv.PkvError):
        decode(*b, SCALE, workspace=ws[:need // 2 // 256 * 256])


@pytest.mark.parametrize("H,R,n", [(16, 512, 50), (64, 512, 900), (128, 256, 3000), (32, 512, 20000)])
def test_bounded_wait_reports_timeout_and_recovers(H, R, n):
    a = make([n, 33], H, R, BF16, 15)
    want = decode(*a, SCALE)
    out = torch.empty_like(want)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.latent_attn_decode(*a, SCALE, out, status=status, flags=pkv.FLAG_TEST_DROP_FIRST_COPY)
    torch.cuda.synchronize()
    assert int(status) == 5
    assert torch.equal(decode(*a, SCALE), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,bound", [(200000, 64), (200000, 4000), (1 << 20, 64)])
def test_many_sequences_most_of_them_empty(S, bound, dtype):
    H, R = 1, 256
    g = torch.Generator(device=DEV).manual_seed(16)
    lens = torch.zeros(S, dtype=torch.int32, device=DEV)
    at = torch.randint(0, S, (50,), generator=g, device=DEV).unique()
    lens[at] = torch.randint(1, 60, (len(at),), generator=g, device=DEV, dtype=torch.int32)
    cache = torch.randn((8, 16, R + ROPE), generator=g, device=DEV).to(dtype)
    tables = torch.randint(0, 8, (S, 4), generator=g, device=DEV, dtype=torch.int32)
    if bound > 64:
        tables = torch.cat([tables, tables.new_full((S, bound // 16 - 4), -1)], 1)
    q = torch.randn((S, H, R + ROPE), generator=g, device=DEV).to(dtype)
    out = decode(q, cache, tables, lens, SCALE, max_seq_len=bound)
    few = torch.ones(S, dtype=torch.bool, device=DEV)
    few[at] = False
    assert not bool(out[few].any())
    n = lens[at].tolist()
    ref, mass, most = decode_reference(q[at], cache, tables[at], n, SCALE)
    near(out[at], ref, mass, most, n, R + ROPE, SCALE)


def test_sizes_past_the_plan_are_refused():
    size = pkv.lib().pkv_latent_attn_workspace_size
    assert size(pkv.BF16, 1 << 20, 16, 512, 64, 16, 1 << 16) == 0
    assert size(pkv.BF16, 1 << 10, 16, 512, 64, 16, 1 << 20) > 0


@pytest.mark.parametrize("R", [256, 512])
@pytest.mark.parametrize("lens", [[4096] * 30, [100, 30000, 1, 64, 6000, 65, 63, 2, 10000], [513] * 152 + [700],
                                  [1] * 100 + [9000] + [1] * 100])
def test_the_same_with_cut_and_whole_sequences(lens, R):
    # A loose bound changes the plan, not the result beyond its rounding.
    q, cache, tables, lens_t = make(lens, 48, R, BF16, 17)
    ref, mass, most = decode_reference(q, cache, tables, lens, SCALE)
    near(decode(q, cache, tables, lens_t, SCALE), ref, mass, most, lens, R + ROPE, SCALE)
    wide = torch.full((len(lens), 20000), -1, dtype=torch.int32, device=DEV)
    wide[:, :tables.shape[1]] = tables
    near(decode(q, cache, wide, lens_t, SCALE), ref, mass, most, lens, R + ROPE, SCALE)


@pytest.mark.parametrize("H", [16, 64, 128])
def test_scattered_scores_of_either_infinity(H):
    # +inf scores make a NaN row, -inf ones weigh nothing; heads do not mix.
    lens, R = [130, 700], 512
    q, cache, tables, lens_t = make(lens, H, R, BF16, 18)
    ok = check(q, cache, tables, lens_t, SCALE)
    cache[int(tables[1, 20]), 3, R] = -INF
    q[1, :, R] = 1.0
    q[1, H // 2, R] = -1.0                              # this head sees +inf
    q[1, H - 1, R] = 0.0                                # and this one 0 * inf
    out = decode(q, cache, tables, lens_t, SCALE).float()
    assert torch.isnan(out[1, H // 2]).all() and torch.isnan(out[1, H - 1]).all()
    rest = [h for h in range(H) if h not in (H // 2, H - 1)]
    assert torch.isfinite(out[1, rest]).all() and torch.equal(out[0], ok[0].float())


# ------------------------------------------------------------ whole prompts

def prompt(lens, H, D, dtype, seed, tail=0):
    T = int(sum(lens)) + tail
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn((T, H, D + ROPE), generator=g, device=DEV).to(dtype)
    kv = torch.randn((T, H, 2 * D), generator=g, device=DEV).to(dtype)
    row = torch.randn((T, 512 + ROPE), generator=g, device=DEV).to(dtype)
    return q, kv[..., :D], row[:, 512:], kv[..., D:]


def starts(lens, first=0):
    return torch.from_numpy(np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)).to(DEV)


def attend(q, k, kr, v, lens, scale, want=0, **kw):
    out = torch.full(v.shape, NAN, dtype=q.dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.latent_prompt_attn(q, k, kr, v, starts(lens), scale, out, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == want
    return out


def check_prompt(q, k, kr, v, lens, scale, **kw):
    out = attend(q, k, kr, v, lens, scale, **kw)
    n = sum(lens)
    ref, mass, most = prompt_reference(q, k, kr, v, lens, scale)
    near(out[:n], ref[:n], mass[:n], most, lens, q.shape[2], scale)
    assert torch.isnan(out[n:].float()).all()           # rows of no sequence are not written
    return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [17], [63], [64], [65], [127, 128, 129], [255, 256, 257], [0, 1, 0, 33, 1, 0],
                                  [300, 5, 0, 256, 1], [1] * 70, [65, 63, 511, 97], [385, 640, 100]])
def test_prompt_lengths(lens, D, dtype):
    check_prompt(*prompt(lens, 4, D, dtype, sum(lens) + D, tail=3), lens, SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [1, 3, 16, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_heads(H, D, dtype):
    check_prompt(*prompt([150, 3, 0, 271], H, D, dtype, H + D), [150, 3, 0, 271], SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,H,D", [(2500, 4, 64), (3001, 8, 128), (4096, 2, 128)])
def test_prompt_long(n, H, D, dtype):
    check_prompt(*prompt([n], H, D, dtype, n), [n], SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_prompt_scales(scale, dtype):
    check_prompt(*prompt([200, 390], 4, 128, dtype, 7), [200, 390], scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_prompt_growing_and_falling_scores(sign, dtype):
    n = 900
    q, k, kr, v = prompt([n], 3, 128, dtype, 3)
    ramp = torch.linspace(0, 6, n, device=DEV)
    q.fill_(1.0)
    k.copy_(((ramp if sign > 0 else ramp.flip(0))[:, None, None] + 0.01 * k.float()).to(dtype))
    check_prompt(q, k, kr, v, [n], 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_strides(D, dtype):
    lens, H = [100, 31, 260], 6
    T, g = sum(lens), torch.Generator(device=DEV).manual_seed(1)
    unit = 16 * 8 // torch.finfo(dtype).bits

    def rows(dims, head_pad, row_pad, first):
        head = dims + head_pad
        buf = torch.randn(T * (H * head + row_pad) + first, generator=g, device=DEV).to(dtype)
        return torch.as_strided(buf, (T, H, dims), (H * head + row_pad, head, 1), first)

    q = rows(D + ROPE, 0, 3 * unit, unit)
    k, v = rows(D, 5 * unit, unit, 0), rows(D, 0, 0, 7 * unit)
    kr = rows(ROPE, unit, 0, unit)[:, 2]
    check_prompt(q, k, kr, v, lens, 0.1)
    check_prompt(q, v, kr.contiguous(), k, lens, 0.1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_one_head_after_the_other(dtype):
    lens, H = [300, 0, 131], 5
    q, k, kr, v = prompt(lens, H, 128, dtype, 33)
    k, v = (x.permute(1, 0, 2).contiguous().permute(1, 0, 2) for x in (k, v))
    assert k.stride(0) == 128 and k.stride(1) == sum(lens) * 128
    check_prompt(q, k, kr, v, lens, SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_prompt_masked_places_may_hold_anything(bad, dtype):
    lens = [70, 400, 45]
    q, k, kr, v = prompt(lens, 4, 128, dtype, 5, tail=9)
    want = check_prompt(q, k, kr, v, lens, SCALE)
    at = 70 + 300                                       # token 300 of the second sequence
    for t in (k, kr, v):
        t[at] = bad
        t[sum(lens):] = bad
    out = attend(q, k, kr, v, lens, SCALE)
    seen = torch.zeros(len(out), dtype=torch.bool, device=DEV)
    seen[at:470] = True
    seen[sum(lens):] = True
    ref, mass, most = prompt_reference(q[:at], k[:at], kr[:at], v[:at], [70, 300], SCALE)
    near(out[:at], ref, mass, most, lens, 192, SCALE)
    near(out[470:515], want[470:515].double(), want[470:515].double().abs() * 0 + 4, 200.0, [45], 192, SCALE)
    assert torch.isnan(out[at:470].float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("what", ["all", "last", "tokens", "sparse", "dims"])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_values_that_are_not_finite(D, what, dtype):
    # NaN among V: dims of rows that see one are NaN, all others are as if it were not there.
    lens = [300, 140, 33]
    q, k, kr, v = prompt(lens, 3, D, dtype, 21)
    g = torch.Generator(device=DEV).manual_seed(2)
    bad = torch.zeros(v.shape, dtype=torch.bool, device=DEV)
    if what == "all":
        bad[:] = True
    elif what == "last":
        bad[[299, 439, 472]] = True
    elif what == "tokens":
        bad[torch.randint(0, sum(lens), (4,), generator=g, device=DEV)] = True
    elif what == "sparse":
        bad = torch.rand(v.shape, generator=g, device=DEV) < 3e-4
    else:
        bad[200, 1, 5] = bad[300, 0] = True
    clean = torch.where(bad, 0.0, v.float()).to(dtype)
    ref, mass, most = prompt_reference(q, k, kr, clean, lens, SCALE)
    out = attend(q, k, kr, torch.where(bad, torch.full_like(clean, NAN), clean), lens, SCALE)
    sees, at = torch.zeros_like(bad), 0
    for n in lens:
        sees[at:at + n] = bad[at:at + n].cumsum(0) > 0
        at += n
    assert torch.equal(torch.isnan(out.float()), sees)
    near(torch.where(sees, torch.zeros_like(out), out), torch.where(sees, 0.0, ref), mass, most, lens, D + ROPE,
         SCALE)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sign", [1, -1])
def test_prompt_infinities(sign, dtype):
    lens = [290]
    q, k, kr, v = prompt(lens, 2, 128, dtype, 22)
    v[100, 0, 3] = sign * INF
    v[200, 0, 3] = -sign * INF
    v[200, 1, 9] = sign * INF
    out = attend(q, k, kr, v, lens, SCALE).float()
    assert torch.isfinite(out[:100]).all()
    assert bool((out[100:200, 0, 3] == sign * INF).all()) and torch.isnan(out[200:, 0, 3]).all()
    assert bool((out[200:, 1, 9] == sign * INF).all()) and torch.isfinite(out[:200, 1]).all()
    rest = out.clone()
    rest[:, 0, 3] = 0
    rest[:, 1, 9] = 0
    assert torch.isfinite(rest).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_invalid_ranges_are_reported_and_not_written(dtype):
    lens = [50, 60, 70]
    q, k, kr, v = prompt(lens, 2, 128, dtype, 23)
    want = attend(q, k, kr, v, lens, SCALE)

    def call(start, **kw):
        out = torch.full(v.shape, NAN, dtype=dtype, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        pkv.latent_prompt_attn(q, k, kr, v, torch.tensor(start, dtype=torch.int32, device=DEV), SCALE, out, status=st,
                               **kw)
        torch.cuda.synchronize()
        return out, int(st)

    out, st = call([0, 50, 110, 999])
    assert st == 4 and torch.equal(out[:110], want[:110]) and torch.isnan(out[110:].float()).all()
    out, st = call([0, 50, 110, 180], max_q_len=60)
    assert st == 4 and torch.equal(out[:110], want[:110]) and torch.isnan(out[110:].float()).all()
    out, st = call([-7, 50])
    assert st == 4 and torch.isnan(out.float()).all()
    out, st = call([0, 50], max_q_len=10 ** 12)
    assert st == 0 and torch.equal(out[:50], want[:50])
    out, st = call([0, 50], max_q_len=0)
    assert st == 4 and torch.isnan(out.float()).all()
    out, st = call([0])
    assert st == 0 and torch.isnan(out.float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_streams_and_graphs(dtype):
    a, b = [300, 40, 900], [500, 77]
    pa, pb = prompt(a, 4, 128, dtype, 24), prompt(b, 4, 128, dtype, 25)
    want_a, want_b = attend(*pa, a, SCALE), attend(*pb, b, SCALE)
    sa, sb = starts(a), starts(b)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.zeros_like(want_a), torch.zeros_like(want_b)
    torch.cuda.synchronize()
    for _ in range(3):
        pkv.latent_prompt_attn(*pa, sa, SCALE, oa, stream=side)
        pkv.latent_prompt_attn(*pb, sb, SCALE, ob, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(oa, want_a) and torch.equal(ob, want_b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.latent_prompt_attn(*pa, sa, SCALE, oa)
    oa.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, want_a)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_bits_do_not_change(dtype):
    lens = [700, 3, 0, 257, 128, 129]
    a = prompt(lens, 6, 128, dtype, 27)
    first = attend(*a, lens, SCALE)
    for _ in range(5):
        assert torch.equal(attend(*a, lens, SCALE), first)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_starts_that_step_back_end(dtype):
    # Not valid, but the call ends, reports it and leaves rows of no sequence alone.
    q, k, kr, v = prompt([400], 2, 64, dtype, 28, tail=5)
    start = torch.tensor([0, 300, 100, 400, 50, 380], dtype=torch.int32, device=DEV)
    out = torch.full(v.shape, NAN, dtype=dtype, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.latent_prompt_attn(q, k, kr, v, start, SCALE, out, status=st)
    torch.cuda.synchronize()
    assert int(st) == 4 and torch.isnan(out[400:].float()).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [40], [200], [300], [3000, 5]])
def test_prompt_timeout_is_reported(lens, D):
    a = prompt(lens, 2, D, BF16, 29)
    want = attend(*a, lens, SCALE)
    attend(*a, lens, SCALE, want=5, flags=pkv.FLAG_TEST_DROP_FIRST_COPY)
    assert torch.equal(attend(*a, lens, SCALE), want)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_output_on_a_16_byte_boundary(D):
    lens, H = [300, 45], 3
    q, k, kr, v = prompt(lens, H, D, BF16, 30)
    want = attend(q, k, kr, v, lens, SCALE)
    buf = torch.full((want.numel() + 16,), NAN, dtype=BF16, device=DEV)
    out = buf[8:8 + want.numel()].view(want.shape)
    assert out.data_ptr() % 32 == 16
    pkv.latent_prompt_attn(q, k, kr, v, starts(lens), SCALE, out)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.isnan(buf[:8]).all() and torch.isnan(buf[-8:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_many_items_with_values_that_are_not_finite(D, dtype):
    # Many short prompts to a CTA, NaN in every third one's V at changing places.
    lens = [129 + (i * 37) % 150 for i in range(600)]
    q, k, kr, v = prompt(lens, 2, D, dtype, 31)
    at, bad = 0, torch.zeros(v.shape, dtype=torch.bool, device=DEV)
    for i, n in enumerate(lens):
        if i % 3 == 0:
            bad[at + (i * 53) % n, i % 2, (i * 7) % D] = True
        at += n
    clean = attend(q, k, kr, torch.where(bad, torch.zeros_like(v), v), lens, SCALE)
    out = attend(q, k, kr, torch.where(bad, torch.full_like(v, NAN), v), lens, SCALE)
    sees, at = torch.zeros_like(bad), 0
    for n in lens:
        sees[at:at + n] = bad[at:at + n].cumsum(0) > 0
        at += n
    assert torch.equal(torch.isnan(out.float()), sees)
    assert torch.equal(torch.where(sees, torch.zeros_like(out), out), torch.where(sees, torch.zeros_like(out), clean))


def test_prompt_as_many_sequences_as_there_may_be():
    S = 1 << 20
    lens = np.zeros(S, np.int64)
    lens[[5, 70000, S - 1]] = [300, 17, 140]
    q, k, kr, v = prompt([300, 17, 140], 2, 128, BF16, 32)
    want = attend(q, k, kr, v, [300, 17, 140], SCALE)
    assert torch.equal(attend(q, k, kr, v, lens, SCALE), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_offsets_past_32_bits(dtype):
    # The last rows of q, k, v and out lie past 2^31 numbers.
    lens, H, D = [150, 40], 16, 128
    T = (2 ** 31) // (H * D) + 300
    q = torch.zeros((T, H, D + ROPE), dtype=dtype, device=DEV)
    kv = torch.zeros((T, H, 2 * D), dtype=dtype, device=DEV)
    kr = torch.zeros((T, ROPE), dtype=dtype, device=DEV)
    small = prompt(lens, H, D, dtype, 26)
    n = sum(lens)
    q[T - n:], kv[T - n:, :, :D], kr[T - n:], kv[T - n:, :, D:] = small
    out = torch.zeros((T, H, D), dtype=dtype, device=DEV)
    pkv.latent_prompt_attn(q, kv[..., :D], kr, kv[..., D:], starts(lens, T - n), SCALE, out, max_q_len=200)
    torch.cuda.synchronize()
    assert torch.equal(out[T - n:], attend(*small, lens, SCALE))
    assert not bool(out[:T - n].any())


# -------------------------------------------------------------- all of it

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_serving_run(dtype):
    """Admission, prompts in the expanded form, their rows into the latent cache, then decode
    steps in the absorbed form over device tables (eager, then a replayed graph), against
    dense attention over every row's tokens in 64 bits."""
    H, D, R, S, N = 8, 128, 512, 3, 64
    g = torch.Generator(device=DEV).manual_seed(31)
    lens = [37, 150, 16]
    T = sum(lens)
    up = torch.randn((H, 2 * D, R), generator=g, device=DEV) / math.sqrt(R)   # keys' and values' up-projections
    table = rope_table(1024, ROPE, DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    seq, tab, ref = torch.zeros(S, **i32), torch.full((S, 20), -1, **i32), torch.zeros(N, **i32)
    q_start, slots = torch.zeros(S + 1, **i32), torch.zeros(T, dtype=torch.int64, device=DEV)
    cache = torch.zeros((N, 16, R + ROPE), dtype=dtype, device=DEV)
    status = torch.zeros(1, **i32)
    pkv.tables_step(seq, tab, ref, new_lens=torch.tensor(lens, **i32), q_start=q_start, slot_mapping=slots,
                    status=status)

    def projections(n):
        row = torch.randn((n, R + ROPE), generator=g, device=DEV).to(dtype)
        return torch.randn((n, H, D + ROPE), generator=g, device=DEV).to(dtype), row

    def expanded(row):
        return torch.einsum("tr,hdr->thd", row[:, :R].float(), up).to(dtype)

    # Prompts.
    q, row = projections(T)
    pos = torch.cat([torch.arange(n, **i32) for n in lens])
    pkv.latent_append(row[:, :R], row[:, R:], pos, table, slots, cache, q_rope=q[..., D:], status=status)
    kr = rotate(row[:, None, R:], table, pos, False, F32)[:, 0].to(dtype)
    kv = expanded(row)
    out = torch.empty((T, H, D), dtype=dtype, device=DEV)
    pkv.latent_prompt_attn(q, kv[..., :D], kr, kv[..., D:], q_start, SCALE, out, status=status)
    want, mass, most = prompt_reference(q, kv[..., :D], kr, kv[..., D:], lens, SCALE)
    near(out, want, mass, most, lens, D + ROPE, SCALE)
    held = [torch.cat([row[s:s + n, :R].float(), kr[s:s + n].float()], 1) for s, n in zip([0, 37, 187], lens)]

    # Decode steps.
    one, pairs = torch.ones(S, **i32), torch.full((S, 2), -1, **i32)
    q_abs = torch.zeros((S, H, R + ROPE), dtype=dtype, device=DEV)
    q_in = torch.zeros((S, H, D + ROPE), dtype=dtype, device=DEV)
    row_in, pos_in = torch.zeros((S, R + ROPE), dtype=dtype, device=DEV), torch.zeros(S, **i32)
    slot, step_out = torch.zeros(S, dtype=torch.int64, device=DEV), torch.zeros((S, H, R), dtype=dtype, device=DEV)

    def step():
        pos_in.copy_(seq)
        pkv.tables_step(seq, tab, ref, new_lens=one, slot_mapping=slot, copy_pairs=pairs, status=status)
        q_abs[..., :R].copy_(torch.einsum("thd,hdr->thr", q_in[..., :D].float(), up[:, :D]))
        pkv.latent_append(row_in[:, :R], row_in[:, R:], pos_in, table, slot, cache, q_rope=q_in[..., D:],
                          q_out=q_abs[..., R:], status=status)
        pkv.latent_attn_decode(q_abs, cache, tab, seq, SCALE, step_out, max_seq_len=320, status=status)

    graph = None
    for i in range(20):
        qi, ri = projections(S)
        q_in.copy_(qi)
        row_in.copy_(ri)
        at = seq.clone()
        if i == 4:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is not None:
            graph.replay()
        else:
            step()
        new_kr = rotate(ri[:, None, R:], table, at, False, F32)[:, 0].to(dtype)
        for s in range(S):
            held[s] = torch.cat([held[s], torch.cat([ri[s, :R].float(), new_kr[s].float()])[None]])
            rows = held[s].double()
            x = q_abs[s].double()
            p = torch.softmax(x @ rows.T * SCALE, -1)
            near(step_out[s], p @ rows[:, :R], p @ rows[:, :R].abs(), float((x.abs() @ rows.abs().T).max()),
                 [len(rows)], R + ROPE, SCALE)
            # The absorbed form is the expanded one: its values multiplied out.
            kvs = torch.einsum("tr,hdr->thd", rows[:, :R], up.double())
            qr = rotate(qi[s:s + 1, :, D:], table, at[s:s + 1], False, torch.float64)[0]
            y = torch.einsum("hd,thd->ht", qi[s, :, :D].double(), kvs[..., :D]) + qr @ rows[:, R:].T
            dense = torch.einsum("ht,thd->hd", torch.softmax(y * SCALE, -1), kvs[..., D:])
            got = torch.einsum("hr,hdr->hd", step_out[s].double(), up[:, D:].double())
            bound = 0.03 if dtype == BF16 else 1e-5     # roundings of q_abs, rows and out to the type
            assert float((got - dense).norm() / dense.norm()) < bound
    assert int(status) == 0 and [int(n) for n in seq] == [n + 20 for n in lens]


@pytest.mark.parametrize("D,seconds", [(64, 3), (128, 2)])
def test_prompt_timeout_waits_for_the_copies_in_flight(D, seconds):
    # A wait gives up after a second.  The first copy of K never comes: the warp that copies K first
    # waits for a slot, then, before it leaves, for block 0, which is not whole.  With heads of 64 it
    # has also asked for the first half of block 3 by then, and that block is not whole either.
    lens = [3000, 5]
    a = prompt(lens, 2, D, BF16, 29)
    want = attend(*a, lens, SCALE)
    out, at = torch.empty_like(want), starts(lens)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    pkv.latent_prompt_attn(*a, at, SCALE, out, status=status, flags=pkv.FLAG_TEST_DROP_FIRST_COPY)
    end.record()
    torch.cuda.synchronize()
    assert int(status) == 5
    assert seconds - 0.1 < begin.elapsed_time(end) / 1e3 < seconds + 0.8
    assert torch.equal(attend(*a, lens, SCALE), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_prompt_rows_that_do_not_see_it_keep_their_bits(bad, D, dtype):
    # One spoilt token and spoilt rows behind the last sequence: every row before the token, and the
    # other sequences whole, are computed from the same numbers in the same order.
    lens = [70, 400, 45]
    q, k, kr, v = prompt(lens, 4, D, dtype, 34, tail=9)
    want = attend(q, k, kr, v, lens, SCALE)
    at = 70 + 300
    for t in (k, kr, v):
        t[at] = bad
        t[sum(lens):] = bad
    out = attend(q, k, kr, v, lens, SCALE)
    assert torch.equal(out[:at], want[:at]) and torch.equal(out[470:515], want[470:515])
    assert torch.isnan(out[at:470].float()).all() and torch.isnan(out[515:].float()).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_bound_of_zero(dtype):
    q, cache, tables, lens = make([5, 0, 70], 16, 256, dtype, 35)
    assert not bool(decode(q, cache, tables, torch.zeros_like(lens), SCALE, max_seq_len=0).any())
    assert not bool(decode(q, cache, tables, lens, SCALE, want=4, max_seq_len=0).any())  # clamped, reported
