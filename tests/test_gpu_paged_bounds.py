"""Attention of chunks against the bounds of the arithmetic that the kernels do (tests/paged_ref.py's are wider:
they allow a polynomial for the exponential, and bf16 weights over an FP8 cache too).

Let w_j be the exact weights of a row that sees c keys, A = sum_j w_j |v_j|, u16 = 2^-8, u32 = 2^-24.
 - Scores: e = 2 (d + 8) u32 S as there, S = scale max_j sum_i |q_i k_ji|.
 - The hardware's base-2 exponential is within 2^-22 of 2^x, relative; a running maximum that moves, or partial
   results that are joined, multiply the values and the sums by such factors, the sums by two of them in a row:
   less than 2^-21 apiece.  A maximum moves once for 32 keys at most, and six joins follow: x = (c / 32 + 8) 2^-21.
   FP8: the logarithm of a value's scale, within 2^-22 max(1, |log2 vs|) and |log2 vs| < 32 here: 2^-17 ln 2 more.
 - A weight is rounded to its type: uw = 2^-8 (bf16), 2^-11 (fp16, over an FP8 cache).  fp16 loses what lies below
   2^-25 of 1: the largest weighted row stands at 2^14 (few query rows) or at 2^3 to 2^15 (many), so a row's weight times
   its scale is off by `floor` = 2^-39 or 2^-28 of the largest.
 - Sums over c keys in fp32, in any order: relative error <= 2 c u32.
 - The output is rounded to bf16: u16 |out|.
|out - o| <= u16 |o| + (uw + 2 (x + 2 c u32 + exp(2 e) - 1)) (1 + u16) A + c floor max_j w_j max_i |v_ji|, and
|lse - l| <= e + x + 2 c u32 + 4 u32 |l| + 2^-20 (the logarithm)."""
import math

import pytest
import torch

from mqa_kv_cache_b200 import workloads as W
from tests import paged_ref as R
from tests.test_gpu_paged import F8, _cache, _chunk, _cuda, _q, _status

pytestmark = pytest.mark.gpu
U16, U32 = R.U16, R.U32


@pytest.fixture(scope="module")
def K():
    from mqa_kv_cache_b200 import kvattn
    return kvattn


def _rows(q, cu, lens, table, page, kd, vd, scale):
    """For each (sequence, head): its slice of tokens, head, scores, unnormalised weights, values, seen keys' S."""
    g = q.shape[1] // kd.shape[1]
    for b in range(len(lens)):
        t0, n, L = int(cu[b]), int(cu[b + 1] - cu[b]), int(lens[b])
        pg, row = R.places(cu, lens, table, page, b)
        seen = torch.arange(L)[None] <= torch.arange(L - n, L)[:, None]
        for h in range(kd.shape[1]):
            k, v = kd[pg, h, row], vd[pg, h, row]
            for j in range(h * g, h * g + g):
                x = q[t0:t0 + n, j].double()
                s = (x @ k.T * scale).masked_fill(~seen, float("-inf"))
                m = s.amax(-1, keepdim=True)
                S = scale * ((x.abs() @ k.abs().T) * seen).amax(-1, keepdim=True)
                yield slice(t0, t0 + n), j, m, torch.exp(s - m), v, S, seen.sum(-1, keepdim=True).double()


def _bounded(q, cu, lens, table, page, kd, vd, scale, fp8, floor, round_weights=None):
    """out, lse and their bounds; with round_weights, out as it is with weights rounded to that type instead."""
    T, H, d = q.shape
    out, ot = torch.zeros(T, H, d, dtype=torch.float64), torch.zeros(T, H, d, dtype=torch.float64)
    lse, lt = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for sl, j, m, p, v, S, c in _rows(q, cu, lens, table, page, kd, vd, scale):
        z = p.sum(-1, keepdim=True)
        w = p / z
        o = w @ v if round_weights is None else (p.to(round_weights).double() / z) @ v
        e = 2 * (d + 8) * U32 * S
        x = (c / 32 + 8) * 2.0 ** -21 + (2.0 ** -17 * math.log(2) if fp8 else 0.0)
        rel = (2.0 ** -11 if fp8 else U16) + 2 * (x + 2 * c * U32 + torch.expm1(2 * e))
        out[sl, j] = o
        ot[sl, j] = U16 * o.abs() + rel * (1 + U16) * (w @ v.abs()) + c * floor * (w * v.abs().amax(-1)).amax(-1, keepdim=True)
        l = (m + torch.log(z))[:, 0]
        lse[sl, j] = l
        lt[sl, j] = (e + x + 2 * c * U32)[:, 0] + 4 * U32 * l.abs() + 2.0 ** -20
    return out, lse, ot, lt


def _floor(n, g, d, fp8):
    """The loss of small weights: up to 8 query rows per KV head, 16 of head_dim 64, go to the kernel of few
    rows, from 33 on to the other one; what may go to either has the wider bound."""
    return 0.0 if not fp8 else 2.0 ** -39 if n * g <= 8 or (n * g <= 16 and d == 64) else 2.0 ** -28


FEW_KEYS = [(3, 2, 64), (3, 2, 128), (3, 16, 64), (3, 16, 128), (3, 64, 64), (3, 64, 128)]  # n, g, d


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,g,d", FEW_KEYS)
def test_weights_are_rounded_once_to_their_type(K, n, g, d, fp8, wide):
    """Three tokens over zero to three cached rows: values of either sign nearly cancel in many columns, where
    a weight's rounding shows.  Small queries, so that the scores' own error does not cover it.  `wide`: page
    tables with room for many more rows."""
    B, page = 60, 16
    ns, ctx = [n] * B, [b % 4 for b in range(B)]
    cu, lens, table, n_pages = R.batch(ns, ctx, page, 400, max_pages=1024 if wide else None)
    tensors, kd, vd = _cache(n_pages, 1, page, d, fp8, 401)
    q, st, scale = _q(int(cu[-1]), g, d, 402, 0.1), _status(), d ** -0.5
    a = (q, cu, lens, table, page, kd, vd, scale, fp8, _floor(n, g, d, fp8))
    ref = _bounded(*a)
    if fp8:  # (bf16 weights, as a statement on the CPU, lie beyond the bounds)
        assert ((_bounded(*a, round_weights=torch.bfloat16)[0] - ref[0]).abs() > ref[2]).any()
    out, lse = _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table), *tensors, scale, max_q=n, dev_status=st)
    assert int(st) == 0
    R.check(out, lse, ref, f"n {n} g {g} d {d}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,ctx,H,Hk,d", [([1, 1], [600, 77], 8, 2, 128), ([2, 1], [5000, 300], 4, 1, 64), ([33, 5], [200, 500], 4, 2, 128),
                                           ([70], [900], 4, 1, 64), ([300], [77], 2, 1, 128), ([1, 40], [40, 4000], 8, 1, 64)])
def test_ordinary_calls_within_the_bounds_of_their_arithmetic(K, ns, ctx, H, Hk, d, fp8):
    page = 32
    cu, lens, table, n_pages = R.batch(ns, ctx, page, 410)
    tensors, kd, vd = _cache(n_pages, Hk, page, d, fp8, 411)
    q, st, scale = _q(int(cu[-1]), H, d, 412), _status(), d ** -0.5
    out, lse = _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table), *tensors, scale, max_q=max(ns), dev_status=st)
    assert int(st) == 0
    R.check(out, lse, _bounded(q, cu, lens, table, page, kd, vd, scale, fp8, _floor(max(ns), H // Hk, d, fp8)), f"{ns} {ctx}")


@pytest.mark.parametrize("n,g,B", [(1, 4, 296), (4, 4, 296), (40, 1, 148), (200, 1, 148)])
def test_many_small_fp8_weights_keep_their_share(K, n, g, B):
    """An early row of large score whose values are zero in half of the columns, and 16K rows behind it whose
    weights are 2^-18 to 2^-27 of its weight: those columns are theirs alone.  As many sequences (of the same pages)
    as CTAs, so that most rows come to the same one, after the large score."""
    page, d, L = 64, 64, 1 << 14
    one = R.batch([n], [L - n], page, 420)
    cu, lens, table, n_pages = torch.arange(B + 1, dtype=torch.int32) * n, one[1].repeat(B), one[2].repeat(B, 1), one[3]
    kc, vc = torch.zeros(2, n_pages, 1, page, d)
    ks, vs = torch.ones(2, n_pages, 1, page)
    pg, row = int(table[0, 0]), 3
    vc[:] = 1.0
    vc[pg, 0, row, : d // 2], vc[pg, 0, row, d // 2:] = -1.0, 0.0
    kc[pg, 0, row], ks[pg, 0, row] = 1.0, 0.25
    scale = 18 * math.log(2) / (d * 0.25)
    mult = torch.linspace(1.0, 1.5, n * g).view(n, g, 1)  # scores of 18 to 27, in log2 units
    q = mult.expand(n, g, d).bfloat16()
    codes = [x.to(F8).view(torch.uint8).cuda() for x in (kc, vc)]
    st = _status()
    out, lse = K.attn_chunk_paged_fp8(q.repeat(B, 1, 1).cuda(), *_cuda(cu, lens, table), codes[0], ks.cuda(), codes[1], vs.cuda(), scale,
                                      max_q=n, dev_status=st)
    assert int(st) == 0
    ref = _bounded(q, *one[:3], page, kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None], scale, True, _floor(n, g, d, True))
    R.check(out, lse, tuple(x.repeat(B, *([1] * (x.dim() - 1))) for x in ref), "small weights")
