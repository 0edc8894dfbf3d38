"""The whole-prompt attention in 64 bits, and how far a kernel's output may be
from it by its arithmetic."""
import math

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a step of f32, of bf16


def reference(q, k, v, lens, scale):
    """(out, sum_j p_j |v_j|, largest sum_d |q_d k_d|) in float64 on the tensors' device."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    mass = torch.zeros_like(out)
    most = 0.0
    at = 0
    for n in lens:
        if n:
            r = slice(at, at + n)
            qq = q[r].double().permute(1, 0, 2)
            kk = k[r].double().permute(1, 0, 2).repeat_interleave(G, 0)
            vv = v[r].double().permute(1, 0, 2).repeat_interleave(G, 0)
            seen = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
            p = torch.softmax((qq @ kk.transpose(1, 2) * scale).masked_fill(~seen, -math.inf), -1)
            out[r] = (p @ vv).permute(1, 0, 2)
            mass[r] = (p @ vv.abs()).permute(1, 0, 2)
            most = max(most, float((qq.abs() @ kk.abs().transpose(1, 2)).max()))
        at += n
    return out, mass, most


def tolerance(out, mass, most, lens, D, scale, dtype, out_dtype):
    """Element-wise bound.

    A score is a dot product of D terms: off by at most (D + 2) u sum|q_d k_d| |scale| with
    u = 2^-24 (twice that on the tensor cores, whose sums may truncate), its exponential by
    2^-22 more.  A weight is one exponential over a sum of n of them, so it is off by twice
    that plus (n + 2) u, relative; the products with V add n more terms.  bf16 inputs: the
    weights are rounded to bf16 (2^-8) for a bf16 output, split in two parts (2^-16) for an
    f32 one.  The output is rounded once.
    """
    n = max(lens)
    tc = 2 if dtype == torch.bfloat16 else 1
    score = tc * (D + 2) * U32 * most * abs(scale) + 2.0 ** -22 + 4 * U32 * abs(scale) * most
    weight = 2 * (math.exp(score) - 1) + 2 * (n + 2) * U32
    if dtype == torch.bfloat16:
        weight += U16 if out_dtype == torch.bfloat16 else U16 * U16
    weight += tc * (n + 2) * U32
    last = U16 if out_dtype == torch.bfloat16 else U32
    return weight * mass * (1 + last) + last * out.abs() + 1e-37
