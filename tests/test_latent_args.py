"""Refusals of the rotating cache writes and of the latent attention, which need
no GPU: nothing is launched."""
import math

import pytest
import torch

import paged_kv_cache_225_gb300 as pkv

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 6
P = 0x10000  # a plausible, aligned device address; never touched


def append(**kw):
    a = dict(q=P, k=P, v=P, dtype=pkv.BF16, qs=32 * 128, ks=8 * 128, vs=8 * 128, pos=P, table=P, rot=128, most=100,
             slots=P, T=10, Hq=32, Hkv=8, D=128, block=16, N=64, out=P, os=32 * 128, kc=P, vc=P, kv=pkv.BF16,
             ksc=1.0, vsc=1.0, flags=0, status=None)
    a.update(kw)
    return pkv.lib().pkv_rope_append(*(a[n] for n in (
        "q", "k", "v", "dtype", "qs", "ks", "vs", "pos", "table", "rot", "most", "slots", "T", "Hq", "Hkv", "D",
        "block", "N", "out", "os", "kc", "vc", "kv", "ksc", "vsc", "flags", "status")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=0), INVALID), (dict(most=0), INVALID),
    (dict(N=0), INVALID), (dict(rot=0), INVALID), (dict(rot=144), INVALID), (dict(rot=24), UNSUPPORTED),
    (dict(rot=8), UNSUPPORTED), (dict(D=96, rot=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(block=32), UNSUPPORTED), (dict(dtype=pkv.FP8_E4M3), UNSUPPORTED), (dict(kv=9), UNSUPPORTED),
    (dict(flags=1), INVALID), (dict(flags=0x400), INVALID),
    (dict(kv=pkv.FP8_E4M3, ksc=0.0), INVALID), (dict(kv=pkv.INT4, vsc=math.nan), INVALID),
    (dict(kv=pkv.FP8_E5M2, vsc=math.inf), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(pos=None), INVALID), (dict(table=None), INVALID),
    (dict(slots=None), INVALID), (dict(q=P + 8), INVALID), (dict(k=P + 2), INVALID), (dict(v=P + 4), INVALID),
    (dict(out=P + 8), INVALID), (dict(kc=P + 8), INVALID), (dict(vc=P + 1), INVALID), (dict(table=P + 8), INVALID),
    (dict(pos=P + 2), INVALID), (dict(slots=P + 4), INVALID), (dict(status=P + 2), INVALID),
    (dict(qs=32 * 128 - 8), INVALID), (dict(ks=0), INVALID), (dict(vs=-1024), INVALID), (dict(os=32 * 128 + 4), INVALID),
    (dict(ks=1 << 36), INVALID), (dict(dtype=pkv.F32, ks=8 * 128 + 2), INVALID),
    # Nothing to do.
    (dict(T=0, q=None, k=None, slots=None), OK),
])
def test_append_arguments(kw, want):
    assert append(**kw) == want


def latent(**kw):
    a = dict(c=P, kr=P, dtype=pkv.BF16, cs=576, rs=576, q=P, qs=16 * 192, qh=192, pos=P, table=P, most=100, slots=P,
             T=10, H=16, R=512, rope=64, block=16, N=64, out=P, os=16 * 576, oh=576, cache=P, kv=pkv.BF16, flags=0,
             status=None)
    a.update(kw)
    return pkv.lib().pkv_latent_append(*(a[n] for n in (
        "c", "kr", "dtype", "cs", "rs", "q", "qs", "qh", "pos", "table", "most", "slots", "T", "H", "R", "rope",
        "block", "N", "out", "os", "oh", "cache", "kv", "flags", "status")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(most=-1), INVALID), (dict(N=0), INVALID),
    (dict(R=384), UNSUPPORTED), (dict(R=0), UNSUPPORTED), (dict(rope=32), UNSUPPORTED), (dict(block=8), UNSUPPORTED),
    (dict(dtype=pkv.INT4), UNSUPPORTED), (dict(kv=pkv.FP8_E4M3), UNSUPPORTED), (dict(flags=2), INVALID),
    (dict(c=None), INVALID), (dict(kr=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(cache=None), INVALID), (dict(pos=None), INVALID), (dict(table=None), INVALID), (dict(slots=None), INVALID),
    (dict(c=P + 8), INVALID), (dict(kr=P + 2), INVALID), (dict(q=P + 8), INVALID), (dict(out=P + 4), INVALID),
    (dict(cache=P + 8), INVALID), (dict(cs=504), INVALID), (dict(rs=56), INVALID), (dict(qh=56), INVALID),
    (dict(qs=60), INVALID), (dict(qs=56), INVALID), (dict(os=15 * 576 + 56), INVALID),
    (dict(os=64, oh=9 * 64 + 56), INVALID), (dict(oh=63), INVALID),
    (dict(cs=578), INVALID), (dict(status=P + 1), INVALID),
    (dict(T=0, c=None), OK),
])
def test_latent_append_arguments(kw, want):
    assert latent(**kw) == want


def decode(**kw):
    a = dict(q=P, cache=P, dtype=pkv.BF16, tables=P, lens=P, S=4, H=16, R=512, rope=64, block=16, N=64, width=8,
             most=128, scale=0.1, out=P, ws=P, bytes=1 << 40, status=None, flags=0)
    a.update(kw)
    return pkv.lib().pkv_latent_attn_decode(*(a[n] for n in (
        "q", "cache", "dtype", "tables", "lens", "S", "H", "R", "rope", "block", "N", "width", "most", "scale", "out",
        "ws", "bytes", "status", "flags")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), INVALID), (dict(H=0), INVALID), (dict(H=129), UNSUPPORTED), (dict(R=128), UNSUPPORTED),
    (dict(R=576), UNSUPPORTED), (dict(rope=0), UNSUPPORTED), (dict(block=64), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(N=1 << 28), UNSUPPORTED), (dict(width=0), INVALID), (dict(most=-1), INVALID), (dict(most=129), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=-math.inf), INVALID), (dict(dtype=pkv.FP8_E5M2), UNSUPPORTED),
    (dict(S=(1 << 20) + 1), UNSUPPORTED), (dict(flags=1), INVALID), (dict(flags=0x100, dtype=pkv.F32), INVALID),
    (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(tables=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(q=P + 8), INVALID), (dict(cache=P + 8), INVALID), (dict(out=P + 2), INVALID),
    (dict(tables=P + 2), INVALID), (dict(lens=P + 1), INVALID), (dict(status=P + 2), INVALID),
    (dict(ws=None), WORKSPACE), (dict(bytes=100), WORKSPACE), (dict(ws=P + 128), INVALID),
    (dict(width=600, most=9000, bytes=1 << 20), WORKSPACE),
    (dict(S=0, q=None), OK),
])
def test_decode_arguments(kw, want):
    assert decode(**kw) == want


def test_workspace_size():
    size = pkv.lib().pkv_latent_attn_workspace_size
    for dtype in (pkv.F32, pkv.BF16):
        assert size(dtype, 64, 64, 512, 64, 16, 32768) >= size(dtype, 1, 64, 512, 64, 16, 100) >= 256
        for bad in ((-1, 64, 512, 64, 16, 100), (4, 0, 512, 64, 16, 100), (4, 64, 500, 64, 16, 100),
                    (4, 64, 512, 32, 16, 100), (4, 64, 512, 64, 8, 100), (4, 64, 512, 64, 16, -1)):
            assert size(dtype, *bad) == 0
    assert size(pkv.INT4, 4, 64, 512, 64, 16, 100) == 0
    with pytest.raises(ValueError):
        pkv.latent_workspace_size(torch.float16, 4, 64, 512, 100)


def prompt(**kw):
    a = dict(q=P, k=P, kr=P, v=P, dtype=pkv.BF16, qs=16 * 192, ks=16 * 256, kh=256, rs=576, vs=16 * 256, vh=256,
             start=P, S=2, T=10, H=16, D=128, rope=64, most=10, scale=0.1, out=P, status=None, flags=0)
    a.update(kw)
    return pkv.lib().pkv_latent_prompt_attn(*(a[n] for n in (
        "q", "k", "kr", "v", "dtype", "qs", "ks", "kh", "rs", "vs", "vh", "start", "S", "T", "H", "D", "rope", "most",
        "scale", "out", "status", "flags")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(most=-1), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(rope=128), UNSUPPORTED),
    (dict(S=(1 << 20) + 1), UNSUPPORTED), (dict(H=65536), UNSUPPORTED), (dict(dtype=pkv.FP8_E4M3), UNSUPPORTED),
    (dict(scale=math.inf), INVALID), (dict(flags=1), INVALID), (dict(flags=0x100, dtype=pkv.F32), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(kr=None), INVALID), (dict(v=None), INVALID),
    (dict(start=None), INVALID), (dict(out=None), INVALID), (dict(q=P + 8), INVALID), (dict(k=P + 2), INVALID),
    (dict(kr=P + 4), INVALID), (dict(v=P + 8), INVALID), (dict(out=P + 8), INVALID), (dict(start=P + 2), INVALID),
    (dict(status=P + 2), INVALID), (dict(qs=16 * 192 - 8), INVALID), (dict(ks=120), INVALID),
    (dict(kh=120), INVALID), (dict(kh=130), INVALID), (dict(vh=0), INVALID), (dict(vs=1 << 36), INVALID),
    (dict(rs=56), INVALID), (dict(dtype=pkv.F32, rs=66), INVALID),
    # Nothing to do.
    (dict(S=0, q=None), OK), (dict(T=0, q=None), OK), (dict(most=0, q=None), OK),
])
def test_prompt_arguments(kw, want):
    assert prompt(**kw) == want


def test_host_tensors_are_refused():
    x, i = torch.zeros((4, 2, 64)), torch.zeros(4, dtype=torch.int32)
    t, sl = torch.zeros((8, 64)), torch.zeros(4, dtype=torch.int64)
    c = torch.zeros((3, 2, 64, 16))
    with pytest.raises(ValueError):
        pkv.rope_append(x, x, x, i, t, sl, c, c)
    with pytest.raises(ValueError):
        pkv.latent_append(torch.zeros((4, 256)), torch.zeros((4, 64)), i, t, sl, torch.zeros((3, 16, 320)))
    with pytest.raises(ValueError):
        pkv.latent_attn_decode(torch.zeros((1, 2, 320)), torch.zeros((3, 16, 320)), i.view(1, 4), i[:1], 0.1,
                               torch.zeros((1, 2, 256)))
    with pytest.raises(ValueError):
        pkv.latent_prompt_attn(torch.zeros((4, 2, 128)), x, torch.zeros((4, 64)), x, i[:2], 0.1, x.clone())


@pytest.mark.gpu
def test_tensors_that_do_not_fit():
    d = dict(device="cuda")
    x, pos = torch.zeros((4, 2, 64), **d), torch.zeros(4, dtype=torch.int32, **d)
    table, slots = torch.zeros((8, 64), **d), torch.arange(4, **d)
    c = torch.zeros((3, 2, 64, 16), **d)
    good = dict(q=x, k=x.clone(), v=x.clone(), positions=pos, table=table, slot_mapping=slots, k_cache=c,
                v_cache=c.clone())
    pkv.rope_append(**good)
    for kw, err in ((dict(q=x[:3]), ValueError), (dict(v=x[:, :1]), ValueError), (dict(k=x.bfloat16()), TypeError),
                    (dict(q=x.transpose(0, 1)), ValueError), (dict(positions=pos.long()), TypeError),
                    (dict(positions=pos[:3]), ValueError), (dict(slot_mapping=slots[:2]), ValueError),
                    (dict(slot_mapping=slots.int()), TypeError), (dict(table=table.double()), TypeError),
                    (dict(table=table[:, :60].contiguous()), pkv.PkvError), (dict(k_cache=c.bfloat16()), ValueError),
                    (dict(v_cache=c[:2]), ValueError), (dict(k_cache=c[..., :8]), ValueError), (dict(q=None, q_out=x), ValueError),
                    (dict(status=torch.zeros(2, dtype=torch.int32, **d)), ValueError), (dict(table=None), TypeError)):
        with pytest.raises(err):
            pkv.rope_append(**{**good, **kw})
    lat = dict(latent=torch.zeros((4, 256), **d), k_rope=torch.zeros((4, 64), **d), positions=pos, table=table,
               slot_mapping=slots, cache=torch.zeros((3, 16, 320), **d))
    pkv.latent_append(**lat)
    for kw, err in ((dict(k_rope=torch.zeros((4, 32), **d)), ValueError), (dict(latent=torch.zeros((3, 256), **d)), ValueError),
                    (dict(latent=torch.zeros((4, 512), **d)[:, ::2]), ValueError), (dict(q_out=x), ValueError),
                    (dict(q_rope=x[:2]), ValueError), (dict(q_rope=x.bfloat16()), TypeError),
                    (dict(cache=torch.zeros((3, 16, 384), **d)), ValueError),
                    (dict(cache=torch.zeros((3, 16, 320), **d).half()), TypeError),
                    (dict(table=torch.zeros((8, 32), **d)), ValueError)):
        with pytest.raises(err):
            pkv.latent_append(**{**lat, **kw})
    q, cache = torch.zeros((1, 2, 320), **d), torch.zeros((3, 16, 320), **d)
    tab, lens = torch.zeros((1, 2), dtype=torch.int32, **d), torch.ones(1, dtype=torch.int32, **d)
    dec = dict(q=q, cache=cache, block_tables=tab, seq_lens=lens, scale=0.1, out=torch.zeros((1, 2, 256), **d))
    pkv.latent_attn_decode(**dec)
    for kw, err in ((dict(q=q.half()), TypeError), (dict(cache=cache.bfloat16()), TypeError),
                    (dict(out=torch.zeros((1, 2, 320), **d)), ValueError), (dict(seq_lens=lens.long()), TypeError),
                    (dict(block_tables=tab[:, :1].expand(2, 1)), ValueError), (dict(cache=cache[..., :256]), ValueError),
                    (dict(max_seq_len=33), pkv.PkvError), (dict(workspace=torch.zeros(512, **d)[::2]), ValueError)):
        with pytest.raises(err):
            pkv.latent_attn_decode(**{**dec, **kw})
    q, kr = torch.zeros((4, 2, 128), **d), torch.zeros((4, 64), **d)
    st = torch.tensor([0, 4], dtype=torch.int32, **d)
    pr = dict(q=q, k=x, k_rope=kr, v=x, q_start=st, scale=0.1, out=torch.zeros_like(x))
    pkv.latent_prompt_attn(**pr)
    for kw, err in ((dict(k=x[:3]), ValueError), (dict(k_rope=kr[:, :32]), ValueError), (dict(v=x[..., ::2]), ValueError),
                    (dict(q=q.bfloat16()), TypeError), (dict(out=torch.zeros((4, 2, 128), **d)), ValueError),
                    (dict(q_start=st.long()), TypeError), (dict(v=x.transpose(0, 1)), ValueError)):
        with pytest.raises(err):
            pkv.latent_prompt_attn(**{**pr, **kw})


# The largest bound whose lengths the kernels can round up to whole tiles of 64 in 32 bits.
MOST = 2 ** 31 - 65


@pytest.mark.parametrize("dtype", [pkv.F32, pkv.BF16])
def test_bounds_whose_tiles_pass_32_bits_are_refused(dtype):
    size = pkv.lib().pkv_latent_attn_workspace_size
    assert size(dtype, 1, 16, 512, 64, 16, MOST) > 0
    # The width holds the bound, nothing else is wrong: past the plan only the workspace is looked at.
    kw = dict(S=1, dtype=dtype, width=1 << 27, bytes=0)
    assert decode(most=MOST, **kw) == WORKSPACE
    for bound in (MOST + 1, 2 ** 31 - 16, 2 ** 31 - 1):
        assert size(dtype, 1, 16, 512, 64, 16, bound) == 0
        assert decode(most=bound, **kw) == UNSUPPORTED


def test_queries_in_place_need_their_own_strides():
    # q_out at q's address and nothing else wrong: other strides would write rows not yet read.
    for kw in (dict(os=33 * 128), dict(qs=64 * 128), dict(T=2, os=33 * 128)):
        assert append(q=P, out=P, **kw) == INVALID
    for kw in (dict(os=5 * 192, oh=192), dict(os=4 * 192, oh=64), dict(T=1, os=4 * 192, oh=64),
               dict(H=1, os=256, oh=192)):
        assert latent(q=P, out=P, **{**dict(H=4, qs=4 * 192, qh=192), **kw}) == INVALID


@pytest.mark.parametrize("T,H,token,head", [
    (10, (1 << 30) + 1, 1 << 33, 1 << 34),          # 2^64 numbers to a token's heads, 2^36 to a head's tokens
    ((1 << 30) + 1, 10, 1 << 34, 1 << 33),
    (1 << 29, (1 << 29) + 1, 1 << 35, 1 << 35),
])
def test_extents_past_64_bits_are_overlaps(T, H, token, head):
    assert latent(T=T, H=H, qs=token, qh=head, os=token, oh=head) == INVALID
    assert latent(T=T, H=H, qs=token, qh=head, os=token, oh=head, q=P, out=P + 16) == INVALID


def test_workspace_sizes_past_32_bits():
    # The library counts in 32 bits: 2^32 + 100 tokens are not 100.
    assert pkv.latent_workspace_size(torch.bfloat16, 1, 16, 512, 100) > 0
    for far in (2 ** 32, -2 ** 32, 2 ** 40):
        for sizes in ((1 + far, 16, 512, 100), (1, 16 + far, 512, 100), (1, 16, 512 + far, 100),
                      (1, 16, 512, 100 + far)):
            with pytest.raises(ValueError):
                pkv.latent_workspace_size(torch.bfloat16, *sizes)


@pytest.mark.gpu
def test_bounds_past_32_bits():
    d = dict(device="cuda")
    tab, lens = torch.zeros((1, 2), dtype=torch.int32, **d), torch.ones(1, dtype=torch.int32, **d)
    out = torch.full((1, 2, 256), 7.0, **d)
    for bound in (2 ** 32 + 16, -2 ** 32 + 16, -2 ** 31):
        with pytest.raises((ValueError, pkv.PkvError)):
            pkv.latent_attn_decode(torch.zeros((1, 2, 320), **d), torch.zeros((3, 16, 320), **d), tab, lens, 0.1, out,
                                   max_seq_len=bound)
    x, start = torch.zeros((4, 2, 64), **d), torch.tensor([0, 4], dtype=torch.int32, **d)
    rows = torch.full_like(x, 7.0)
    for bound in (-2 ** 32 + 4, -2 ** 31, -1):
        with pytest.raises(pkv.PkvError):
            pkv.latent_prompt_attn(torch.zeros((4, 2, 128), **d), x, torch.zeros((4, 64), **d), x, start, 0.1, rows,
                                   max_q_len=bound)
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((rows == 7).all())
