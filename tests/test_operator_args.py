"""Refusals of the whole-prompt attention and of the device block tables, which
need no GPU: nothing is launched."""
import ctypes
import math

import pytest
import torch

import paged_kv_cache_225_gb300 as pkv

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # a plausible, aligned device address; never touched


def prompt(**kw):
    a = dict(q=P, k=P, v=P, dtype=pkv.BF16, qs=32 * 128, ks=8 * 128, vs=8 * 128, start=P, S=2, T=10,
             Hq=32, Hkv=8, D=128, maxq=10, scale=0.1, out=P, out_dtype=pkv.BF16, status=None, flags=0)
    a.update(kw)
    return pkv.lib().pkv_prompt_attn(a["q"], a["k"], a["v"], a["dtype"], a["qs"], a["ks"], a["vs"],
                                     a["start"], a["S"], a["T"], a["Hq"], a["Hkv"], a["D"], a["maxq"],
                                     a["scale"], a["out"], a["out_dtype"], a["status"], a["flags"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(Hq=30), INVALID), (dict(maxq=-1), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(flags=1), INVALID), (dict(flags=0x200), INVALID), (dict(flags=0x100, dtype=pkv.F32), INVALID),
    (dict(dtype=pkv.FP8_E5M2), UNSUPPORTED), (dict(dtype=pkv.INT4), UNSUPPORTED),
    (dict(out_dtype=pkv.FP8_E4M3), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(Hq=136, qs=136 * 128), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(start=None), INVALID),
    (dict(out=None), INVALID), (dict(q=P + 8), INVALID), (dict(k=P + 2), INVALID), (dict(v=P + 4), INVALID),
    (dict(out=P + 8), INVALID), (dict(start=P + 2), INVALID), (dict(status=P + 1), INVALID),
    (dict(qs=32 * 128 - 8), INVALID), (dict(ks=0), INVALID), (dict(vs=-8 * 128), INVALID),
    (dict(qs=32 * 128 + 4), INVALID), (dict(ks=1 << 36), INVALID),
    (dict(dtype=pkv.F32, vs=8 * 128 + 2), INVALID),
    # Nothing to do.
    (dict(S=0, q=None), OK), (dict(T=0, q=None), OK), (dict(maxq=0, q=None), OK),
])
def test_prompt_arguments(kw, want):
    assert prompt(**kw) == want


def step(**kw):
    a = dict(lens=P, tables=P, ref=P, S=4, width=8, block=16, N=64, drop=None, new=P, start=P, slots=P,
             most=10, pairs=P, status=None)
    a.update(kw)
    return pkv.lib().pkv_tables_step(a["lens"], a["tables"], a["ref"], a["S"], a["width"], a["block"],
                                     a["N"], a["drop"], a["new"], a["start"], a["slots"], a["most"],
                                     a["pairs"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), INVALID), (dict(width=0), INVALID), (dict(width=1 << 26), INVALID), (dict(N=0), INVALID),
    (dict(most=-1), INVALID), (dict(block=32), UNSUPPORTED), (dict(S=8193), UNSUPPORTED),
    (dict(lens=None), INVALID), (dict(tables=None), INVALID), (dict(ref=None), INVALID),
    (dict(slots=None), INVALID), (dict(ref=P + 4), INVALID), (dict(slots=P + 4), INVALID),
    (dict(lens=P + 2), INVALID), (dict(tables=P + 1), INVALID), (dict(drop=P + 2), INVALID),
    (dict(new=P + 3), INVALID), (dict(start=P + 2), INVALID), (dict(pairs=P + 2), INVALID),
    (dict(status=P + 2), INVALID), (dict(S=0, most=0, start=None, lens=None), OK),
    (dict(S=0, ref=None), INVALID), (dict(S=0, most=0, ref=None), INVALID),
    (dict(S=0, most=0, start=None, ref=None), OK),
])
def test_step_arguments(kw, want):
    assert step(**kw) == want


def fork(**kw):
    a = dict(pairs=P, n=2, lens=P, tables=P, ref=P, S=4, width=8, block=16, N=64, status=None)
    a.update(kw)
    return pkv.lib().pkv_tables_fork(a["pairs"], a["n"], a["lens"], a["tables"], a["ref"], a["S"],
                                     a["width"], a["block"], a["N"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(S=-1), INVALID), (dict(width=0), INVALID), (dict(N=0), INVALID),
    (dict(block=8), UNSUPPORTED), (dict(pairs=None), INVALID), (dict(lens=None), INVALID),
    (dict(tables=None), INVALID), (dict(ref=None), INVALID), (dict(pairs=P + 2), INVALID),
    (dict(status=P + 2), INVALID), (dict(n=0, pairs=None), OK),
])
def test_fork_arguments(kw, want):
    assert fork(**kw) == want


def test_host_tensors_are_refused():
    q = torch.zeros((4, 2, 64))
    with pytest.raises(ValueError):
        pkv.prompt_attn(q, q, q, torch.zeros(2, dtype=torch.int32), 0.1, q.clone())
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.tables_step(torch.zeros(2, **i32), torch.zeros((2, 4), **i32), torch.zeros(8, **i32))
    with pytest.raises(ValueError):
        pkv.tables_fork(torch.zeros((1, 2), **i32), torch.zeros(2, **i32), torch.zeros((2, 4), **i32),
                        torch.zeros(8, **i32))


@pytest.mark.gpu
def test_tensors_that_do_not_fit():
    d = dict(device="cuda")
    q, k = torch.zeros((6, 4, 64), **d), torch.zeros((6, 2, 64), **d)
    s = torch.tensor([0, 6], dtype=torch.int32, **d)
    ok = pkv.prompt_attn(q, k, k, s, 0.1, torch.ones_like(q))
    assert bool((ok == 0).all())
    for args in ((q, k[:5], k, s), (q, k, k[:, :1], s), (q.transpose(0, 1), k, k, s), (q, k, k[..., ::2], s),
                 (q, k, k, s.view(1, 2)), (q[0], k, k, s)):
        with pytest.raises(ValueError):
            pkv.prompt_attn(*args, 0.1, torch.ones_like(q))
    with pytest.raises(ValueError):
        pkv.prompt_attn(q, k, k, s, 0.1, torch.ones_like(q)[:5])
    for args in ((q, k.bfloat16(), k, s), (q, k, k, s.long()), (q.half(), k.half(), k.half(), s)):
        with pytest.raises(TypeError):
            pkv.prompt_attn(*args, 0.1, torch.ones_like(q))
    with pytest.raises(pkv.PkvError):                        # rows 8 bytes off
        buf = torch.zeros(6 * 258 + 2, **d)
        pkv.prompt_attn(torch.as_strided(buf, (6, 4, 64), (258, 64, 1)), k, k, s, 0.1, torch.ones_like(q))
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, tab, ref = torch.zeros(3, **i32), torch.full((3, 4), -1, **i32), torch.zeros(8, **i32)
    for kw in (dict(drop_lens=torch.zeros(2, **i32)), dict(new_lens=torch.zeros(4, **i32)),
               dict(q_start=torch.zeros(3, **i32)), dict(copy_pairs=torch.zeros((2, 2), **i32)),
               dict(status=torch.zeros(2, **i32)), dict(slot_mapping=torch.zeros((2, 2), dtype=torch.int64, **d))):
        with pytest.raises(ValueError):
            pkv.tables_step(lens, tab, ref, **kw)
    for kw in (dict(new_lens=torch.zeros(3, **d)), dict(slot_mapping=torch.zeros(3, **i32))):
        with pytest.raises(TypeError):
            pkv.tables_step(lens, tab, ref, **kw)
    with pytest.raises(ValueError):
        pkv.tables_step(lens, tab[:2], ref)
    with pytest.raises(ValueError):
        pkv.tables_fork(torch.zeros((1, 3), **i32), lens, tab, ref)


def test_slow_gate_flag_is_for_bf16():
    assert prompt(flags=pkv.FLAG_TEST_SLOW_GATE, dtype=pkv.F32) == INVALID
    assert prompt(flags=pkv.FLAG_TEST_SLOW_GATE, T=0, q=None) == OK


def test_number_of_sequences():
    # More would let the bf16 kernel's waits run out while items are looked up.
    for dtype, qs, kv in ((pkv.BF16, 32 * 128, 8 * 128), (pkv.F32, 32 * 128, 8 * 128)):
        assert prompt(S=(1 << 20) + 1, dtype=dtype, qs=qs, ks=kv, vs=kv) == UNSUPPORTED
        assert prompt(S=1 << 20, dtype=dtype, qs=qs, ks=kv, vs=kv, T=0, q=None) == OK
