"""Plain 64-bit forms of the cache writes and reads and of the tree attention,
on the CPU, with the bounds that the kernels' rounding steps give."""

from __future__ import annotations

import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative
F32 = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def host(x):
    return None if x is None else x.detach().cpu()


def values(cache, scale=None):
    """Cache rows in 64 bits."""
    x = host(cache).double()
    return x if scale is None else x * host(scale).double()[..., None]


def gather(pool, table):
    """A pool's rows in token order: [b, hkv, tokens, ...]."""
    x = host(pool)
    x = x.view(torch.uint8) if x.dtype == E4M3 else x
    x = x[host(table).long()].transpose(1, 2)
    x = x.reshape(x.shape[:2] + (-1,) + x.shape[4:])
    return x.view(E4M3) if pool.dtype == E4M3 else x


def scatter(dense, pool, table):
    """Writes dense [b, hkv, tokens, ...] into the pool's blocks, in place."""
    page = pool.shape[2]
    raw = (lambda x: x.view(torch.uint8) if x.dtype == E4M3 else x)
    for e in range(table.shape[0]):
        for j in range(table.shape[1]):
            raw(pool)[int(table[e, j])] = raw(dense)[e, :, j * page:(j + 1) * page]


def bits_of(sees):
    """[b, t, t] bool -> the int32 mask words."""
    b, t, _ = sees.shape
    words = (t + 31) // 32
    m = torch.zeros((b, t, words * 32), dtype=torch.int64)
    m[:, :, :t] = sees.long()
    m = (m.view(b, t, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(m >= 1 << 31, m - (1 << 32), m).to(torch.int32)


def attention(q, k, v, lens, nodes, sees, scale=None, sloppy=True):
    """(out, bound) in 64 bits: q [b, t, hq, d], k, v [b, hkv, n, d] values,
    lens and nodes lists, sees [b, t, t] bool. Hidden tokens are left out of
    the sums, so what they hold does not matter. The bound is elementwise:

    * a score is a sum of d products in fp32, at most (d + 2) half steps off
      relative to sum |q k|; two such errors (its own and the maximum's, which
      cancels in exact arithmetic but is rounded) move a weight by that times
      the scale;
    * exp2 is 2 units off, the weight's sums are fp32 sums over n tokens;
    * sloppy (bf16 and 8-bit caches): the weight is rounded to bf16, 2^-8.
    """
    q, k, v = host(q).double(), k.double(), v.double()
    b, t, hq, d = q.shape
    g = hq // k.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros_like(q)
    bound = torch.zeros_like(q)
    for e in range(b):
        n, m = lens[e], nodes[e]
        for i in range(m):
            at = torch.cat([torch.arange(n), n + torch.nonzero(sees[e, i, :m]).flatten()])
            if not len(at):
                continue
            for h in range(hq):
                kk, vv = k[e, h // g, at], v[e, h // g, at]
                s = kk @ q[e, i, h] * scale
                p = torch.softmax(s, 0)
                delta = 2 * (d + 4) * F32 * scale * (kk.abs() @ q[e, i, h].abs())
                rel = delta + (len(at) + 64) * F32 + (2.0 ** -8 if sloppy else 0.0)
                out[e, i, h] = p @ vv
                # errors of the weights reach the result through the values and through the sum of weights
                bound[e, i, h] = (p * rel) @ vv.abs() + (p @ (delta + (len(at) + 64) * F32)) * out[e, i, h].abs()
    return out, bound


def check(got, want, bound, what=""):
    got = host(got).double()
    tol = bound * 1.01 + HALF[torch.float32] * want.abs() + 1e-30
    bad = ~((got - want).abs() <= tol) & ~(torch.isnan(got) & torch.isnan(want))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off; worst {float(((got - want).abs() / tol)[bad].max())} x the bound"


def heads(x, w, eps, pos, inv_freq, inter):
    """Norm and rotation in 64 bits: x [b, t, h, d] -> (y, pair norms for the bound)."""
    x = host(x).double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * host(w).double()
    y, norm = x.clone(), x.abs()
    if inv_freq is not None:
        f = host(inv_freq).double()
        a = host(pos).double()[:, :, None, None] * f
        c, s = torch.cos(a), torch.sin(a)
        n = f.numel()
        i0 = torch.arange(n) * 2 if inter else torch.arange(n)
        i1 = i0 + 1 if inter else i0 + n
        y[..., i0] = x[..., i0] * c - x[..., i1] * s
        y[..., i1] = x[..., i1] * c + x[..., i0] * s
        norm[..., i0] = norm[..., i1] = x[..., i0].abs() + x[..., i1].abs()
    return y, norm


# fp32 steps between the input and the stored value: the mean of squares (a sum
# over d / 8 terms a lane and a butterfly: under 24 half steps, halved by the
# root), rsqrt (2 units), two products, the angle (2^-24 of half a turn: 4 half
# steps), sine and cosine (2 units) and the turn's two products and sum
STEPS = 40 * F32
