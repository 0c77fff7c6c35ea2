"""Ragged batches over a paged KV cache: seeded inputs and a plain statement in 64 bits
(CPU torch) of the append and of attention, with the error bounds that the tests apply.

Bounds of attention.  Let w_j be the exact weights, A = sum_j w_j |v_j| (per output
element), u16 = 2^-8 half a bf16 step relative to the value and u32 = 2^-24.
 - A score is a sum of d products in fp32 (each partial sum may be truncated: 2 u32 a step)
   and a few more fp32 operations on it: |ds| <= e = 2 (d + 8) u32 S, S = scale max_j sum_i
   |q_i k_ji|, in natural-log units; every weight moves by at most a factor exp(2 e).
 - The base-2 exponential is off by at most 2^-13 (the degree-3 polynomial's 7.5e-5).
 - A weight is rounded to 16 bits: relative error <= u16 (bf16; fp16's is smaller, but loses
   what lies below 2^-25 of the row's largest weighted row: n 2^-25 max_j w_j max_i |v_ji|).
 - Sums over n keys in fp32, in any order: relative error <= 2 n u32.
 - The output is rounded to bf16: u16 |out|.
So |out - o| <= u16 |o| + (u16 + 2^-13 + 2 n u32 + exp(2 e) - 1) (1 + u16) 2 A + floor; the factor 2 since
numerator and denominator both move.  The rounding of the weights enters the numerator only, so it is
counted once.  |lse - l| <= e + 2^-13 + 2 n u32 + 4 u32 |l| + 2^-20 (the logarithm's own error)."""
import numpy as np
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def batch(ns, ctx, page, seed, slack=2, max_pages=None):
    """cu, seq_lens, page_table (int32 CPU tensors) and the pool's size: pages in random order,
    unused table entries -1."""
    g = torch.Generator().manual_seed(seed)
    lens = [n + c for n, c in zip(ns, ctx)]
    per = [-(-l // page) for l in lens]
    n_pages = sum(per) + slack
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(ns), max(max_pages or 0, max(per), 1)), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(per):
        table[b, :p] = order[at:at + p]
        at += p
    cu = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32)
    return cu, torch.tensor(lens, dtype=torch.int32), table, n_pages


def places(cu, lens, table, page, b):
    """Pages and rows of every cached row of sequence b."""
    r = torch.arange(int(lens[b]))
    return table[b][r // page].long(), r % page


def rotate(x, cos, sin, pos, pair):
    """x [n, heads, d] rotated at pos [n] with fp32 tables, in fp64."""
    x, c, s = x.double(), cos.double()[pos][:, None], sin.double()[pos][:, None]
    if pair == 0:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def attention(q, cu, lens, table, page, kd, vd, scale, max_q=None, fp16_weights=False):
    """q [T, H, d] bf16, kd / vd [n_pages, Hk, page, d] fp64 (dequantised) -> out, lse, and the
    bounds of their errors; tokens behind cu[B] (and past max_q) are NaN in out and lse."""
    T, H, d = q.shape
    Hk = kd.shape[1]
    g = H // Hk
    out = torch.full((T, H, d), float("nan"), dtype=torch.float64)
    lse = torch.full((T, H), float("nan"), dtype=torch.float64)
    ot, lt = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(lens)):
        t0, n = int(cu[b]), int(cu[b + 1] - cu[b])
        L = int(lens[b])
        pg, row = places(cu, lens, table, page, b)
        ok = (pg >= 0) & (pg < kd.shape[0])
        pos = torch.arange(L - n, L)
        seen = (torch.arange(L)[None] <= pos[:, None]) & ok[None]
        take = n if max_q is None else min(n, max_q)
        for h in range(Hk):
            k = torch.where(ok[:, None], kd[pg.clamp(0, kd.shape[0] - 1), h, row], 0.0)
            v = torch.where(ok[:, None], vd[pg.clamp(0, kd.shape[0] - 1), h, row], 0.0)
            for j in range(h * g, h * g + g):
                x = q[t0:t0 + n, j].double()
                s = (x @ k.T * scale).masked_fill(~seen, float("-inf"))
                m = s.amax(-1, keepdim=True) if L else torch.full((n, 1), float("-inf"))
                m = torch.where(m.isfinite(), m, 0.0).double()
                p = torch.exp(s - m)
                z = p.sum(-1, keepdim=True)
                w = p / torch.where(z > 0, z, 1.0)
                o = w @ v
                A = w @ v.abs()
                S = scale * ((x.abs() @ k.abs().T) * seen).amax(-1, keepdim=True) if L else torch.zeros(n, 1)
                cnt = seen.sum(-1, keepdim=True).double()
                e = 2 * (d + 8) * U32 * S
                rel = U16 + 2 * (2.0 ** -13 + 2 * cnt * U32 + torch.expm1(2 * e))
                tol = U16 * o.abs() + rel * (1 + U16) * A + 1e-30
                if fp16_weights and L:
                    tol = tol + cnt * 2.0 ** -25 * (w * v.abs().amax(-1)).amax(-1, keepdim=True)
                l = (m + torch.log(z))[:, 0]
                sl = slice(t0, t0 + take)
                out[sl, j], ot[sl, j] = o[:take], tol[:take]
                lse[sl, j] = l[:take]
                lt[sl, j] = (e + 2.0 ** -13 + 2 * cnt * U32)[:take, 0] + 4 * U32 * l[:take].abs().nan_to_num(0, 0, 0) + 2.0 ** -20
    return out, lse, ot, lt


def check(got, lse, ref, what=""):
    """got / lse against attention()'s answer and bounds; NaN in the reference = not checked."""
    out, l, ot, lt = ref
    have = ~l.isnan()
    got, glse = got.double().cpu(), lse.double().cpu()
    d = (got - out).abs()[have]
    bad = ~(d <= ot[have])
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outputs beyond their bound, worst {float((d / ot[have]).nan_to_num(9e9).max()):.3g} x"
    fin = have & l.isfinite()
    assert torch.equal(glse[have].isfinite(), l[have].isfinite()), f"{what}: lse finiteness"
    assert (glse[have & ~l.isfinite()] == float("-inf")).all()
    dl = (glse - l).abs()[fin]
    assert (dl <= lt[fin]).all(), f"{what}: lse off by {float((dl / lt[fin]).max()):.3g} x its bound"
