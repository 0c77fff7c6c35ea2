"""Attention of chunks where every CTA of the tile kernel walks many short pieces (a server's queue of short
prompts): each sequence's queries have another size, so that anything kept from one piece for another shows.
Against the statement in 64 bits of tests/paged_ref.py."""
import random

import pytest
import torch

from mqa_kv_cache_b200 import workloads as W
from tests import paged_ref as R
from tests.test_gpu_paged import _cache, _chunk, _cuda, _status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from mqa_kv_cache_b200 import kvattn
    return kvattn


def _queries(cu, H, d, seed):
    """N(0, 1) rows, those of each sequence times a power of two of its own, 2^-6 .. 2^5."""
    q = torch.randn(int(cu[-1]), H, d, generator=W.generator(seed))
    for b in range(len(cu) - 1):
        q[int(cu[b]):int(cu[b + 1])] *= 2.0 ** ((5 * b) % 12 - 6)
    return q.bfloat16()


def _run(K, ns, ctx, H, Hk, d, page, fp8, seed):
    cu, lens, table, n_pages = R.batch(ns, ctx, page, seed)
    tensors, kd, vd = _cache(n_pages, Hk, page, d, fp8, seed + 1)
    q, st, scale = _queries(cu, H, d, seed + 2), _status(), d ** -0.5
    b, qg = _cuda(cu, lens, table), q.cuda()
    ws = K.workspace(K.attn_chunk_paged_workspace_bytes(len(ns), int(cu[-1]), max(ns), H, Hk, d))
    calls = [_chunk(K, fp8, qg, *b, *tensors, scale, max_q=max(ns), ws=ws, dev_status=st) for _ in range(4)]
    assert int(st) == 0
    R.check(*calls[0], R.attention(q, cu, lens, table, page, kd, vd, scale, fp16_weights=fp8), f"{H}/{Hk} d{d} fp8={fp8}")
    for out, lse in calls[1:]:
        assert torch.equal(out, calls[0][0]) and torch.equal(lse, calls[0][1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,keys", [(1, 64), (2, 64), (2, 128), (4, 64), (4, 128)])
def test_many_short_prompts(K, g, keys, d, fp8):
    """200 sequences of 17 to 60 tokens, 8 KV heads, 20 to `keys` rows each: about ten units a CTA, most of
    one step; g = 4: blocks of two Q tiles among them."""
    r = random.Random(g * keys)
    ns = [r.randint(17, 60) for _ in range(200)]
    ns[0], ns[1] = 60, 17
    ctx = [max(0, r.randint(max(n, 20), max(n, keys)) - n) for n in ns]
    _run(K, ns, ctx, 8 * g, 8, d, 16, fp8, 300)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,n_hi", [(1, 100), (4, 33), (8, 32), (16, 9)])
def test_many_sequences_of_mixed_lengths(K, g, n_hi, d, fp8):
    """128 sequences, 8 KV heads, chunks of 1 to n_hi tokens over 1 to 64, 65 to 128 or 129 to 300 rows."""
    r = random.Random(g)
    lens = [r.randint(*r.choice([(1, 64), (65, 128), (129, 300)])) for _ in range(128)]
    ns = [min(r.randint(1, n_hi), l) for l in lens]
    ns[-1], lens[-1] = n_hi, n_hi + 40
    _run(K, ns, [l - n for n, l in zip(ns, lens)], 8 * g, 8, d, 32, fp8, 310)
