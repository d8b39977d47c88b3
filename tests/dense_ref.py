"""64-bit references of the position rotation, the 16-bit paged cache and its
attention, and the bounds their fp32 arithmetic and one rounding allow.

Bounds (u = 2^-24, half a step of fp32; e = torch.finfo(dtype).eps / 2):
  * rotation: a c - fl(b s) in one fma is off by at most u |b s| + u |result|,
    at most 2 u r for a pair of length r; rounding to the result's type adds
    e |result| (and half its smallest step);
  * attention: a score of 128 products is off by at most
    (128 + 2) u scale sum |q_j k_j|, the exponential by 2^-21, weights
    and their sum likewise; with d the largest such score error a weight is
    off by 2 (d + 2^-20) relative, so o by that times A = sum_t p_t |v_t|.
    Rounding a weight to w bits before the product with v adds 2^-w A, and
    rounding the result e |o|.
"""
import math

import torch

D = 128
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rope_table(n, rot, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def rope64(x, pos, table, rot, inter):
    """x [n][heads][128] -> float64, rotated to pos [n] on the fp32 table; also the length r of each coordinate's pair."""
    x = x.double()
    y, r = x.clone(), x.abs()
    c = table[pos, :rot // 2].double()[:, None]
    s = table[pos, rot // 2:].double()[:, None]
    ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    r[..., ia] = r[..., ib] = torch.hypot(a, b)
    return y, r


def check_rotated(got, want, r):
    """got [n][heads][128] of a 16-bit type against rope64's result."""
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    bound = half_step(got.dtype) * want.abs() * (1 + 2 * U) + 4 * U * r + tiny
    bad = (got.double() - want).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} coordinates outside the bound"


def attend64(q, k, v, limits, scale=None):
    """q [H][R][128], k, v [H][T][128], limits [R] -> o, A = sum p |v|, d (the largest score error of a row)."""
    q, k, v = q.double(), k.double(), v.double()
    sc = 1 / math.sqrt(D) if not scale else scale
    T = k.shape[1]
    hide = torch.arange(T, device=q.device)[None] >= limits[:, None].to(q.device)
    s = torch.matmul(q, k.transpose(1, 2)) * sc
    s = s.masked_fill(hide, -math.inf)
    mag = (torch.matmul(q.abs(), k.abs().transpose(1, 2)) * sc).masked_fill(hide, 0.0)
    d = mag.amax(-1, keepdim=True) * (130 * U) if T else torch.zeros(q.shape[:2] + (1,), dtype=torch.float64)
    if T == 0:
        return torch.zeros_like(q), torch.zeros_like(q), d
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    return torch.matmul(p, v), torch.matmul(p, v.abs()), d


def check_attention(got, o, A, d, weight_bits):
    """got of a 16-bit type against attend64's o within the bound above."""
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    bound = half_step(got.dtype) * o.abs() * (1 + 2.0 ** -10) + A * (2.0 ** -weight_bits + 2 * (d + 2.0 ** -20)) * \
        (1 + 2.0 ** -8) + tiny
    err = (got.double() - o).abs()
    assert torch.isfinite(got).all()
    bad = err > bound
    assert not bad.any(), f"{int(bad.sum())} outputs outside the bound, worst ratio {float((err / bound).max()):.2f}"
