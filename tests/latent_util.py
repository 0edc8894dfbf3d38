"""The rotation and the latent attention in 64 bits, for the tests."""
import math

import numpy as np
import torch

ROPE = 64


def rope_table(positions, rot, dev, base=10000.0):
    """f32 [positions, rot]: cosines, then sines."""
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(dev)


def rotate(x, table, pos, interleaved, dtype):
    """x [T, H, D] in `dtype` with its first dims turned; every product and sum rounded on its own."""
    rot = table.shape[1]
    cs = table[pos.long()].to(dtype)[:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    y = x.to(dtype).clone()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = y[..., lo].clone(), y[..., hi].clone()
    y[..., lo] = a * c - b * s
    y[..., hi] = b * c + a * s
    return y


def decode_reference(q, cache, tables, lens, scale):
    """(out, sum_t p_t |row_t|, largest sum_d |q_d row_td|) in float64; empty rows are 0."""
    S, H, row = q.shape
    R = row - ROPE
    out = torch.zeros((S, H, R), dtype=torch.float64, device=q.device)
    mass, most = torch.zeros_like(out), 0.0
    for s, n in enumerate(lens):
        if not n:
            continue
        rows = cache[tables[s, :-(-n // 16)].long()].flatten(0, 1)[:n].double()
        x = q[s].double()
        p = torch.softmax(x @ rows.T * scale, -1)
        out[s] = p @ rows[:, :R]
        mass[s] = p @ rows[:, :R].abs()
        most = max(most, float((x.abs() @ rows.abs().T).max()))
    return out, mass, most


def prompt_reference(q, k, k_rope, v, lens, scale):
    """As prompt_util.reference, for the expanded form."""
    T, H, D = v.shape
    out = torch.zeros((T, H, D), dtype=torch.float64, device=q.device)
    mass, most, at = torch.zeros_like(out), 0.0, 0
    for n in lens:
        if n:
            r = slice(at, at + n)
            qq = q[r].double().permute(1, 0, 2)
            kk = torch.cat([k[r].double(), k_rope[r].double()[:, None].expand(n, H, ROPE)], 2).permute(1, 0, 2)
            vv = v[r].double().permute(1, 0, 2)
            seen = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
            p = torch.softmax((qq @ kk.transpose(1, 2) * scale).masked_fill(~seen, -math.inf), -1)
            out[r] = (p @ vv).permute(1, 0, 2)
            mass[r] = (p @ vv.abs()).permute(1, 0, 2)
            most = max(most, float((qq.abs() @ kk.abs().transpose(1, 2)).max()))
        at += n
    return out, mass, most


def pages_for(lens, seed, extra=5, width=None):
    """(tables int32 [S, width], pages of the pool): every row's pages anywhere in the pool."""
    r = np.random.RandomState(seed)
    held = [-(-int(n) // 16) for n in lens]
    N = sum(held) + extra
    places = r.permutation(N)
    tables = np.full((len(lens), width or max(1, max(held, default=1))), -1, np.int32)
    at = 0
    for s, n in enumerate(held):
        tables[s, :n] = places[at:at + n]
        at += n
    return tables, N
