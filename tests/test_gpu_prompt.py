"""Whole-prompt attention (pkv_prompt_attn) against the same formula in 64
bits: lengths, groups, types, strides, what masked places may hold, scales,
device-side reports, streams and graphs."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_225_gb300 as pkv

from prompt_util import reference, tolerance

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16


def starts(lens, first=0):
    return torch.from_numpy(np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)).to(DEV)


def make(lens, Hq, Hkv, D, dtype, seed, fused=True, tail=0):
    T = int(sum(lens)) + tail
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def check(q, k, v, lens, scale, out_dtype=None, **kw):
    out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), scale, out, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    ref, mass, most = reference(q, k, v, lens, scale)
    tol = tolerance(ref, mass, most, lens, q.shape[2], scale, q.dtype, out.dtype)
    n = sum(lens)
    off = (out[:n].double() - ref[:n]).abs()
    assert not torch.isnan(off).any()
    assert bool((off <= tol[:n]).all()), f"worst {float((off / tol[:n]).max()):.3g} of the tolerance"
    assert torch.isnan(out[n:].float()).all()      # rows of no sequence are not written
    return out


TYPES = [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)]


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("lens", [[1], [2], [17], [64], [127, 128, 129], [0, 1, 0, 33, 1, 0],
                                  [300, 5, 0, 256, 1], [1] * 70, [65, 63, 511, 97]])
def test_lengths(lens, dtype, out_dtype):
    q, k, v = make(lens, 8, 2, 128, dtype, sum(lens), tail=3)
    check(q, k, v, lens, 1 / math.sqrt(128), out_dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 4), (6, 2), (4, 1), (10, 2), (6, 1), (14, 2), (8, 1),
                                    (9, 1), (10, 1), (11, 1), (24, 2), (13, 1), (14, 1), (15, 1), (16, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_groups(Hq, Hkv, D, dtype):
    lens = [150, 3, 0, 71]
    q, k, v = make(lens, Hq, Hkv, D, dtype, Hq * 100 + D)
    check(q, k, v, lens, 1 / math.sqrt(D))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(2500, 4, 4, 64), (3001, 8, 1, 128), (2047, 12, 4, 128)])
def test_long(n, Hq, Hkv, D, dtype):
    q, k, v = make([n], Hq, Hkv, D, dtype, n)
    check(q, k, v, [n], 1 / math.sqrt(D))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(scale, dtype):
    lens = [200, 90]
    q, k, v = make(lens, 4, 2, 64, dtype, 7)
    check(q, k, v, lens, scale)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("sign", [1, -1])
def test_growing_and_falling_scores(sign, dtype, out_dtype):
    # The running maximum rises by far more than 2^8 again and again (or never
    # after the first key).
    n, D = 700, 64
    q, k, v = make([n], 4, 2, D, dtype, 3, fused=False)
    ramp = torch.linspace(0, 6, n, device=DEV)
    if sign < 0:
        ramp = ramp.flip(0)
    q.fill_(1.0)
    k.copy_((ramp[:, None, None] + 0.01 * k.float()).to(dtype))
    check(q, k, v, [n], 1.0, out_dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_strides(D, dtype):
    # Rows 16-byte multiples apart, each tensor with its own distance, dense rows
    # starting anywhere on a 16-byte boundary.
    lens, Hq, Hkv = [100, 31], 6, 2
    T = sum(lens)
    g = torch.Generator(device=DEV).manual_seed(1)

    def rows(H, pad, first):
        buf = torch.randn(T * (H * D + pad) + first, generator=g, device=DEV).to(dtype)
        return torch.as_strided(buf, (T, H, D), (H * D + pad, D, 1), first)

    unit = 16 * 8 // torch.finfo(dtype).bits
    q, k, v = rows(Hq, unit, 0), rows(Hkv, 3 * unit, unit), rows(Hkv, 0, 5 * unit)
    check(q, k, v, lens, 0.1)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_masked_places_may_hold_anything(bad, dtype, out_dtype):
    # Rows before a bad token, and every other sequence, do not see it.
    lens = [70, 200, 45]
    q, k, v = make(lens, 8, 2, 64, dtype, 9, fused=False, tail=40)
    k2, v2 = k.clone(), v.clone()
    cut = 70 + 90
    k2[cut:70 + 200], v2[cut:70 + 200] = bad, bad
    k2[sum(lens):], v2[sum(lens):] = bad, bad
    a = torch.zeros(q.shape, dtype=out_dtype, device=DEV)
    b = torch.zeros_like(a)
    pkv.prompt_attn(q, k, v, starts(lens), 0.125, a)
    pkv.prompt_attn(q, k2, v2, starts(lens), 0.125, b)
    ref, mass, most = reference(q, k, v, lens, 0.125)
    tol = tolerance(ref, mass, most, lens, 64, 0.125, dtype, out_dtype)
    for rows in (slice(0, cut), slice(270, 315)):
        assert bool(((a[rows].double() - ref[rows]).abs() <= tol[rows]).all())
        assert bool(((b[rows].double() - ref[rows]).abs() <= tol[rows]).all())


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_bad_values_reach_the_rows_that_see_them(dtype, out_dtype):
    lens = [150, 60]
    q, k, v = make(lens, 4, 1, 128, dtype, 10, fused=False)
    v[40, 0, 5] = float("inf")
    v[90, 0, 7] = float("nan")
    k[120, 0, 0] = float("nan")
    out = torch.zeros(q.shape, dtype=out_dtype, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, out)
    o = out.float()
    dims = torch.arange(128, device=DEV)
    assert torch.isfinite(o[:40]).all() and torch.isfinite(o[150:]).all()
    assert bool((o[40:90, :, 5] == math.inf).all()) and torch.isfinite(o[40:90][..., dims != 5]).all()
    assert torch.isnan(o[90:120, :, 7]).all() and bool((o[90:120, :, 5] == math.inf).all())
    assert torch.isfinite(o[90:120][..., (dims != 5) & (dims != 7)]).all()
    assert torch.isnan(o[120:150]).all()


def test_scores_of_minus_infinity():
    # A key whose score is -inf has no weight; a row that sees nothing else is NaN,
    # as in the formula.
    for dtype in (F32, BF16):
        q, k, v = make([140], 2, 1, 64, dtype, 11, fused=False)
        q.copy_(q.abs() + 0.1)
        k[:130, 0, 0] = -float("inf")
        out = torch.zeros(q.shape, dtype=dtype, device=DEV)
        pkv.prompt_attn(q, k, v, starts([140]), 0.1, out)
        assert torch.isnan(out[:130].float()).all()
        ref, mass, _ = reference(q[130:], k[130:], v[130:], [10], 0.1)
        most = float((q[130:].double().abs().amax() * k[130:].double().abs().amax()) * 64)
        tol = tolerance(ref, mass, most, [140], 64, 0.1, dtype, dtype)
        assert bool(((out[130:].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_invalid_ranges_are_reported_and_not_written(dtype):
    q, k, v = make([40, 50, 30], 4, 2, 64, dtype, 12)
    good = torch.zeros(q.shape, dtype=dtype, device=DEV)
    pkv.prompt_attn(q, k, v, starts([40, 50, 30]), 0.1, good)

    def run(qs, **kw):
        out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        pkv.prompt_attn(q, k, v, torch.tensor(qs, dtype=torch.int32, device=DEV), 0.1, out,
                        status=status, **kw)
        return out, int(status)

    out, st = run([0, 40, 90, 121])               # past the rows
    assert st == 4 and torch.equal(out[:90], good[:90]) and bool((out[90:] == 7).all())
    out, st = run([0, 40, 30, 30])                # decreasing
    assert st == 4 and torch.equal(out[:40], good[:40]) and bool((out[40:] == 7).all())
    out, st = run([-1, 40, 90, 120])              # before the rows
    assert st == 4 and bool((out[:40] == 7).all()) and torch.equal(out[40:], good[40:])
    out, st = run([0, 40, 90, 120], max_q_len=45)  # longer than promised
    assert st == 4 and bool((out[40:90] == 7).all())
    assert torch.equal(out[:40], good[:40]) and torch.equal(out[90:], good[90:])
    out, st = run([0, 0, 0, 0])
    assert st == 0 and bool((out == 7).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_starts_that_step_back_end(dtype):
    # Every other range is the whole batch: a thousand times the items that its
    # rows allow.  The call ends, reports it and writes nothing but right rows.
    q, k, v = make([700], 4, 2, 64, dtype, 22)
    good = torch.zeros(q.shape, dtype=dtype, device=DEV)
    pkv.prompt_attn(q, k, v, starts([700]), 0.1, good)
    out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, torch.tensor([0, 700] * 1000, dtype=torch.int32, device=DEV), 0.1, out, status=status)
    assert int(status) == 4
    assert bool(((out == good) | (out == 7)).all())


def test_a_bound_past_the_rows_is_no_bound():
    q, k, v = make([40, 50], 4, 2, 64, BF16, 23)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    pkv.prompt_attn(q, k, v, starts([40, 50]), 0.1, a)
    pkv.prompt_attn(q, k, v, starts([40, 50]), 0.1, b, max_q_len=2 ** 32 + 1)
    assert torch.equal(a, b) and bool((a != 0).any())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_rows(dtype):
    e = torch.empty((0, 4, 64), dtype=dtype, device=DEV)
    out = pkv.prompt_attn(e, e, e, torch.zeros(3, dtype=torch.int32, device=DEV), 0.1, e.clone())
    assert out.shape == (0, 4, 64)
    q, k, v = make([5], 4, 2, 64, dtype, 1)
    out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    pkv.prompt_attn(q, k, v, torch.zeros(1, dtype=torch.int32, device=DEV), 0.1, out)
    assert bool((out == 7).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bits_do_not_change(dtype):
    # Twice, beside other sequences, and with more room in max_q_len: the same bits.
    lens = [200, 333]
    q, k, v = make(lens, 16, 2, 128, dtype, 13)
    a, b, c = (torch.zeros(q.shape, dtype=dtype, device=DEV) for _ in range(3))
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, a)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, b, max_q_len=333)
    pkv.prompt_attn(q, k, v, starts([200]), 0.1, c, max_q_len=200)
    assert torch.equal(a, b) and torch.equal(a[:200], c[:200])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_streams_and_graphs(dtype):
    lens = [90, 200, 1]
    q, k, v = make(lens, 8, 2, 128, dtype, 14, fused=False)
    want = torch.zeros(q.shape, dtype=dtype, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = torch.zeros_like(want)
    qs = starts(lens)
    torch.cuda.synchronize()
    pkv.prompt_attn(q, k, v, qs, 0.1, got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    # One graph, replayed over other lengths and other values in the same buffers; a
    # second graph beside it.
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    o1, o2 = torch.zeros_like(want), torch.zeros_like(want)
    with torch.cuda.graph(g1):
        pkv.prompt_attn(q, k, v, qs, 0.1, o1)
    with torch.cuda.graph(g2):
        pkv.prompt_attn(q, k, v, qs, 0.1, o2)
    side = torch.cuda.Stream()
    for new in ([90, 200, 1], [1, 289, 1], [0, 0, 291]):
        qs.copy_(starts(new))
        k.mul_(0.5)
        pkv.prompt_attn(q, k, v, qs, 0.1, want)
        side.wait_stream(torch.cuda.current_stream())
        g1.replay()
        with torch.cuda.stream(side):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want) and torch.equal(o2, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_past_32_bits(dtype):
    # Rows 2^18 elements apart: the last ones lie past 2^31 elements (2^32 bytes).
    T, Hq, Hkv, D, stride = 8300, 4, 2, 64, 1 << 18
    buf = torch.empty((T, stride), dtype=dtype, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    small = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype)
    n = (Hq + 2 * Hkv) * D
    buf[:, :n] = small.view(T, n)
    rows = buf[:, :n].view(T, Hq + 2 * Hkv, D)
    lens = [8000, 250, 50]
    out = torch.zeros((T, Hq, D), dtype=dtype, device=DEV)
    pkv.prompt_attn(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], starts(lens), 0.125, out)
    want = torch.zeros_like(out)
    c = small.contiguous()
    pkv.prompt_attn(c[:, :Hq], c[:, Hq:Hq + Hkv], c[:, Hq + Hkv:], starts(lens), 0.125, want)
    assert torch.equal(out, want)
    tail = c[8000:]
    check(tail[:, :Hq], tail[:, Hq:Hq + Hkv], tail[:, Hq + Hkv:], [250, 50], 0.125)


def test_many_short_sequences():
    r = np.random.RandomState(5)
    lens = [int(x) for x in r.randint(0, 40, 700)]
    for dtype in (F32, BF16):
        q, k, v = make(lens, 4, 2, 64, dtype, 15)
        check(q, k, v, lens, 0.125)


def test_bounded_wait_reports_timeout_and_recovers():
    lens = [300, 40]
    q, k, v = make(lens, 8, 2, 128, BF16, 16)
    out = torch.zeros(q.shape, dtype=BF16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, out, status=status,
                    flags=pkv.FLAG_TEST_DROP_FIRST_COPY)
    torch.cuda.synchronize()
    assert int(status) == 5  # PKV_ERR_TIMEOUT
    check(q, k, v, lens, 0.1)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_output_on_a_16_byte_boundary(D, dtype, out_dtype):
    # Outputs need 16-byte alignment only.
    lens = [70, 1, 130]
    q, k, v = make(lens, 6, 2, D, dtype, 17)
    unit = 16 * 8 // torch.finfo(out_dtype).bits
    buf = torch.full((q.numel() + 2 * unit,), 7.0, dtype=out_dtype, device=DEV)
    out = buf[unit:unit + q.numel()].view(q.shape)
    assert out.data_ptr() % 32 == 16
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, out)
    want = torch.zeros(q.shape, dtype=out_dtype, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, want)
    assert torch.equal(out, want) and bool((buf[:unit] == 7).all()) and bool((buf[-unit:] == 7).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_calls_at_once(dtype):
    # Two streams, two batches, nothing shared: each as alone.
    runs = []
    for seed, lens in ((20, [500, 40, 300]), (21, [33] * 20)):
        q, k, v = make(lens, 16, 4, 128, dtype, seed)
        want = torch.zeros(q.shape, dtype=dtype, device=DEV)
        pkv.prompt_attn(q, k, v, starts(lens), 0.1, want)
        runs.append((q, k, v, starts(lens), want, torch.zeros_like(want), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for q, k, v, qs, _, got, s in runs:
            pkv.prompt_attn(q, k, v, qs, 0.1, got, stream=s)
    torch.cuda.synchronize()
    for _, _, _, _, want, got, _ in runs:
        assert torch.equal(want, got)


def test_rows_of_a_very_long_prompt_are_computed_again():
    # The last V row is infinite: the rows before it in its block are computed
    # again over half a million keys each, which the waits must allow for.
    n, D, scale = 1 << 19, 64, 0.125
    q, k, v = make([n], 1, 1, D, BF16, 24)
    v[-1] = math.inf
    out = torch.zeros(q.shape, dtype=BF16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, starts([n]), scale, out, status=status)
    assert int(status) == 0
    assert bool((out[-1] == math.inf).all()) and bool(torch.isfinite(out[:-1]).all())
    for i in (0, 1000, n // 2, n - 130, n - 128, n - 77, n - 2):
        qq, kk, vv = q[i, 0].double(), k[:i + 1, 0].double(), v[:i + 1, 0].double()
        p = torch.softmax(kk @ qq * scale, 0)
        ref, mass = p @ vv, p @ vv.abs()
        most = float((kk.abs() @ qq.abs()).max())
        tol = tolerance(ref, mass, most, [i + 1], D, scale, BF16, BF16)
        assert bool(((out[i, 0].double() - ref).abs() <= tol).all()), i


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_calls_without_rows_report_their_ranges(dtype):
    # No rows, or a bound of 0: nothing is computed, a range that is not empty is reported.
    q, k, v = make([5], 4, 2, 64, dtype, 1)

    def run(qs, n, **kw):
        out = torch.full((n,) + tuple(q.shape[1:]), 7.0, dtype=dtype, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        pkv.prompt_attn(q[:n], k[:n], v[:n], torch.tensor(qs, dtype=torch.int32, device=DEV), 0.1, out,
                        status=status, **kw)
        assert bool((out == 7).all())
        return int(status)

    assert run([0, 0, 0], 0) == 0
    assert run([0, 0, 5], 0) == 4
    assert run([0, -1, 0], 0) == 4
    assert run([0] * 700 + [1], 0) == 4
    assert run([0, 5], 5, max_q_len=0) == 4
    assert run([3, 3, 3], 5, max_q_len=0) == 0
    assert run([6, 6], 5, max_q_len=0) == 4


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[2000], [130] * 200, [700, 1, 129, 300, 17, 255, 1100] * 4])
def test_a_late_watcher_of_the_loads(lens, D):
    # The warp that watches the loads looks at each 20 us late, when all that does not wait for it has
    # run ahead: the same bits, and no wait runs out.
    q, k, v = make(lens, 8, 2, D, BF16, 26)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, a)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, b, status=status, flags=pkv.FLAG_TEST_SLOW_GATE)
    assert int(status) == 0 and torch.equal(a, b) and bool((a != 0).any())


def value_reference(q, k, v, lens, scale):
    """reference() with V's NaN and infinities as the values they are: a row that sees one in a
    dim gives it (NaN for both signs), whatever its weight; the others sum what is finite."""
    ref, mass, most = reference(q, k, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), lens, scale)
    G, at = q.shape[1] // k.shape[1], 0
    for n in lens:
        x = v[at:at + n].float().repeat_interleave(G, 1)
        nan, up, down = (torch.cumsum(b, 0) > 0 for b in (torch.isnan(x), x == math.inf, x == -math.inf))
        r = ref[at:at + n]
        r[up], r[down], r[nan | (up & down)] = math.inf, -math.inf, math.nan
        at += n
    return ref, mass, most


def check_values(q, k, v, lens, scale, out_dtype):
    out = torch.zeros(q.shape, dtype=out_dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), scale, out, status=status)
    assert int(status) == 0
    ref, mass, most = value_reference(q, k, v, lens, scale)
    n = sum(lens)
    o, ref = out[:n].double(), ref[:n]
    assert torch.equal(torch.isnan(o), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert torch.equal(o[inf], ref[inf]) and not torch.isinf(o[~inf]).any()
    fine = torch.isfinite(ref)
    tol = tolerance(torch.where(fine, ref, 0), mass[:n], most, lens, q.shape[2], scale, q.dtype, out_dtype)
    off = (o - ref).abs()
    assert bool((off[fine] <= tol[fine]).all()), f"worst {float((off[fine] / tol[fine]).max()):.3g}"
    return out


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (4, 1, 128), (6, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("what", ["all", "last", "tokens", "one_inf", "sparse", "both_signs", "dims"])
def test_values_that_are_not_finite(what, Hq, Hkv, D, dtype, out_dtype):
    lens = [70, 700, 1, 0, 257, 300]
    q, k, v = make(lens, Hq, Hkv, D, dtype, 30, fused=False, tail=9)
    r = np.random.RandomState(31)
    T = v.shape[0]
    inf, nan = math.inf, math.nan
    if what == "all":
        v.fill_(nan)
    elif what == "last":
        for e in np.cumsum(lens)[:-1]:
            v[max(0, int(e) - 1)] = nan
    elif what == "tokens":
        for t, x in zip(r.choice(T, 12, replace=False), [nan, inf, -inf] * 4):
            v[int(t)] = x
    elif what == "one_inf":
        v[72, 0, 5], v[300, Hkv - 1, 7], v[1030, 0, 0] = inf, -inf, inf
    elif what == "sparse":
        u = torch.from_numpy(r.rand(*v.shape)).to(DEV)
        v[u < 1e-3] = nan
        v[(u > 0.5) & (u < 0.5005)] = inf
        v[u > 0.9995] = -inf
    elif what == "both_signs":
        v[100:130, :, ::3] = inf
        v[400:410, :, ::2] = -inf
    elif what == "dims":
        for d in range(D):                         # each dim's first one some rows later
            v[70 + 11 * d % 690, :, d] = [nan, inf, -inf][d % 3]
    check_values(q, k, v, lens, 1 / math.sqrt(D), out_dtype)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_values_and_scores_that_are_not_finite(out_dtype):
    # An infinite V row whose own score is -inf has weight 0: NaN, as in the formula.
    q, k, v = make([400], 2, 1, 64, BF16, 32, fused=False)
    q.copy_(q.abs() + 0.1)
    k[50, 0, 3], v[50, 0, 9] = -math.inf, math.inf
    v[130, 0, 20] = math.nan
    out = torch.zeros(q.shape, dtype=out_dtype, device=DEV)
    pkv.prompt_attn(q, k, v, starts([400]), 0.1, out)
    o = out.float()
    dims = torch.arange(64, device=DEV)
    assert torch.isfinite(o[:50]).all()
    assert torch.isnan(o[50:, :, 9]).all() and torch.isnan(o[130:, :, 20]).all()
    assert torch.isfinite(o[50:130][..., dims != 9]).all()
    assert torch.isfinite(o[130:][..., (dims != 9) & (dims != 20)]).all()
    # A score that is NaN gives a NaN row, whatever V holds after it.
    k[60, 0, 0] = math.nan
    pkv.prompt_attn(q, k, v, starts([400]), 0.1, out)
    o = out.float()
    assert torch.isnan(o[60:]).all() and torch.isfinite(o[:50]).all()


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["all", "last", "one_inf", "sparse"])
def test_what_values_that_are_not_finite_cost(what, out_dtype):
    # At most one slower pass more, 8 times the time in all where it was measured.
    q, k, v = make([8192], 32, 8, 128, BF16, 33, fused=False)
    bad = v.clone()
    if what == "all":
        bad.fill_(math.nan)
    elif what == "last":
        bad[-1] = math.nan
    elif what == "one_inf":
        bad[3, :, 5] = math.inf
    else:
        bad[torch.rand(v.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) < 1e-4] = math.nan
    out = torch.zeros(q.shape, dtype=out_dtype, device=DEV)

    def ms(x):
        best = math.inf
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            pkv.prompt_attn(q, k, x, starts([8192]), 0.1, out)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert ms(bad) <= 20 * ms(v)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_as_many_sequences_as_there_may_be(dtype):
    # 2^20 of them, all but three empty, the longest with many blocks: no wait runs out.
    lens = np.zeros(1 << 20, np.int64)
    lens[[5, 1 << 19, (1 << 20) - 1]] = 3000, 17, 40
    q, k, v = make([3000, 17, 40], 4, 4, 64, dtype, 40)
    out, want = torch.zeros(q.shape, dtype=dtype, device=DEV), torch.zeros(q.shape, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), 0.125, out, status=status)
    pkv.prompt_attn(q, k, v, starts([3000, 17, 40]), 0.125, want)
    assert int(status) == 0 and torch.equal(out, want)
    with pytest.raises(pkv.PkvError) as e:
        pkv.prompt_attn(q, k, v, torch.zeros((1 << 20) + 2, dtype=torch.int32, device=DEV), 0.125, out)
    assert e.value.code == 2


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [40], [200], [3000, 5]])
def test_timeout_with_copies_issued_and_in_flight(lens, D):
    # The copies are all issued (short prompts), or wait for the ring, when the MMA thread gives up.
    q, k, v = make(lens, 8, 2, D, BF16, 41)
    out = torch.zeros(q.shape, dtype=BF16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.prompt_attn(q, k, v, starts(lens), 0.1, out, status=status, flags=pkv.FLAG_TEST_DROP_FIRST_COPY)
    assert int(status) == 5
    check(q, k, v, lens, 0.1)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.7])
@pytest.mark.parametrize("Hq,Hkv", [(7, 1), (10, 2), (13, 1)])
def test_values_that_are_not_finite_in_views(Hq, Hkv, scale, out_dtype):
    # Rows of a fused projection, head groups that leave rows of a tile empty, scales of either sign; twice
    # in a graph, then with other values in the same buffers.
    lens = [300, 33, 0, 150]
    q, k, v = make(lens, Hq, Hkv, 128, BF16, 34)
    clean = v.clone()
    out = torch.zeros(q.shape, dtype=out_dtype, device=DEV)
    qs = starts(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.prompt_attn(q, k, v, qs, scale, out)
    for rows in ((299, 310, 480), (100, 301), ()):
        v.copy_(clean)
        for i, t in enumerate(rows):
            v[t, :, i::3] = [math.nan, math.inf, -math.inf][i % 3]
        want = check_values(q, k, v, lens, scale, out_dtype)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:sum(lens)].nan_to_num(nan=7.0), want[:sum(lens)].nan_to_num(nan=7.0))
