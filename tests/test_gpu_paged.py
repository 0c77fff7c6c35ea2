"""The paged-cache operators on the GPU: appending a ragged batch (bf16 and FP8), reading an FP8
cache back, and attention of a chunk, each against a plain statement in 64 bits with derived
bounds (tests/paged_ref.py), and runs of them together as a server would make them."""
import numpy as np
import pytest
import torch

import oracle
from mqa_kv_cache_b200 import workloads as W
from tests import paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from mqa_kv_cache_b200 import kvattn
    return kvattn


F8 = torch.float8_e4m3fn


def _cuda(*ts):
    return [t.cuda() for t in ts]


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _tables(K, d, max_pos, pair=0):
    return K.rope_table_build(K.rope_params(d, 10000.0, pair_style=pair), max_pos)


def _quant(x):
    """The rule in fp32: scale = absmax / 448, code = E4M3(x / scale)."""
    s = x.float().abs().amax(-1) / 448.0
    c = (x.float() / torch.where(s > 0, s, 1.0)[..., None]).to(F8)
    return c, s


# ---- append -------------------------------------------------------------------------------------

APPEND = [  # ns, ctx, heads, d, page
    ([1], [0], 1, 64, 16), ([1] * 7, [5, 0, 63, 64, 15, 16, 100], 2, 128, 16), ([3, 0, 17, 64], [13, 9, 0, 128], 2, 64, 32),
    ([130, 1, 65], [0, 511, 30], 8, 128, 64), ([5], [0], 3, 128, 128), ([300, 40], [1, 1023], 1, 64, 1024)]


def _new_tokens(T, heads, d, seed, extra=0):
    """k and v as slices of one projection, so that their token stride is longer than a row."""
    x = W.normal_bf16((T + extra, (2 * heads + 1) * d), W.generator(seed)).cuda()
    return x[:, d:(heads + 1) * d].view(T + extra, heads, d), x[:, (heads + 1) * d:].view(T + extra, heads, d)


@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("ns,ctx,heads,d,page", APPEND)
def test_append_writes_the_rotated_rows_and_nothing_else(K, ns, ctx, heads, d, page, pair):
    cu, lens, table, n_pages = R.batch(ns, ctx, page, 3)
    T = int(cu[-1])
    k, v = _new_tokens(T, heads, d, 11, extra=2)  # two tokens behind the last sequence
    fill = W.normal_bf16((n_pages, heads, page, d), W.generator(5)).cuda()
    kp, vp = fill.clone(), (-fill).clone()
    cos, sin = _tables(K, d, int(lens.max()))
    st = _status()
    K.kv_append_paged_rope(k, v, *_cuda(cu, lens, table), kp, vp, cos, sin, pair_style=pair, dev_status=st)
    # the rotation of the library's in-place operator, bit for bit
    want_k, want_v = fill.clone(), (-fill).clone()
    kr = k[:T].clone()
    pos = torch.cat([torch.arange(l - n, l) for n, l in zip(ns, lens.tolist())]).to(torch.int32)
    K.rope_apply_qk(None, None, kr[None], pos[None].cuda(), cos, sin, k_layout="bthd", pair_style=pair)
    for b, n in enumerate(ns):
        pg, row = R.places(cu, lens, table, page, b)
        pg, row = pg[len(pg) - n:].cuda(), row[len(row) - n:].cuda()
        want_k[pg, :, row] = kr[cu[b]:cu[b] + n]
        want_v[pg, :, row] = v[cu[b]:cu[b] + n]
    assert int(st) == 0
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("ns,ctx,heads,d,page", APPEND)
def test_append_fp8_quantises_the_rotated_rows(K, ns, ctx, heads, d, page, pair):
    """V: the fp32 rule bit for bit (the oracle's quantiser decides the codes).  K: the fp32 rotation is
    off by a few 2^-24 of the row's largest element, so the scale is within 8 * 2^-24 of fp64's and a
    code's value within half a step (2^-4 of it, or 2^-10 absolute) plus that noise."""
    cu, lens, table, n_pages = R.batch(ns, ctx, page, 4)
    T = int(cu[-1])
    k, v = _new_tokens(T, heads, d, 12)
    k[0, 0] = 0  # an all-zero row: scale 0, codes 0
    v[-1, -1] = 0
    kc = torch.full((n_pages, heads, page, d), 0x55, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks = torch.full((n_pages, heads, page), 7.0, device="cuda")
    vs = ks.clone()
    cos, sin = _tables(K, d, int(lens.max()))
    st = _status()
    K.kv_append_paged_rope_fp8(k, v, *_cuda(cu, lens, table), kc, ks, vc, vs, cos, sin, pair_style=pair, dev_status=st)
    assert int(st) == 0
    touched = torch.zeros(n_pages, heads, page, dtype=torch.bool)
    vbits = W.bf16_bits(v.contiguous()).reshape(-1, d)
    oc, osc = oracle.quant_fp8(vbits, group=d)
    oc, osc = torch.from_numpy(np.asarray(oc)).view(T, heads, d), torch.from_numpy(np.asarray(osc)).view(T, heads)
    for b, n in enumerate(ns):
        if n == 0:
            continue
        pg, row = R.places(cu, lens, table, page, b)
        pg, row = pg[len(pg) - n:], row[len(row) - n:]
        touched[pg, :, row] = True
        t = slice(int(cu[b]), int(cu[b]) + n)
        assert torch.equal(vc.cpu()[pg, :, row], oc[t]) and torch.equal(vs.cpu()[pg, :, row], osc[t].float())
        x = R.rotate(k[t].cpu(), cos.cpu(), sin.cpu(), torch.arange(int(lens[b]) - n, int(lens[b])), pair)
        s64 = x.abs().amax(-1) / 448
        s = ks.cpu()[pg, :, row].double()
        assert ((s - s64).abs() <= 8 * R.U32 * s64).all()
        got = kc.cpu()[pg, :, row].view(F8).double()
        y = x / torch.where(s > 0, s, 1.0)[..., None]
        noise = 8 * R.U32 * 448
        assert ((got - y).abs() <= torch.maximum(y.abs() * 2.0 ** -4, torch.full_like(y, 2.0 ** -10)) + noise).all()
    untouched = ~touched.cuda()
    for c in (kc, vc):
        assert (c[untouched] == 0x55).all()
    for s in (ks, vs):
        assert (s[untouched] == 7.0).all()


def test_append_leaves_out_what_has_no_place(K):
    """Bad pages, positions past the table or below zero, lengths past the capacity: skipped and flagged."""
    heads, d, page = 2, 64, 16
    cos, sin = _tables(K, d, 40)
    k, v = _new_tokens(4, heads, d, 13)

    def run(cu, lens, table):
        kp = torch.zeros(3, heads, page, d, dtype=torch.bfloat16, device="cuda")
        vp, st = kp.clone(), _status()
        K.kv_append_paged_rope(k, v, *_cuda(*(torch.tensor(x, dtype=torch.int32) for x in (cu, lens, table))), kp, vp,
                               cos, sin, dev_status=st)
        return int(st), (vp != 0).any(-1).any(1).sum().item()

    assert run([0, 4], [18], [[0, 1]]) == (0, 4)
    assert run([0, 4], [18], [[0, 3]]) == (K.STATUS_BAD_INDEX, 2)        # rows 14, 15 | 16, 17 on a bad page
    assert run([0, 4], [18], [[-1, 1]]) == (K.STATUS_BAD_INDEX, 2)
    assert run([0, 4], [42], [[0, 1, 2]]) == (K.STATUS_BAD_POSITION, 2)  # positions 38 .. 41, tables of 40
    assert run([0, 4], [2], [[0, 1]]) == (K.STATUS_BAD_POSITION, 2)      # positions -2 .. 1
    assert run([0, 4], [99], [[0, 1]])[0] & K.STATUS_BAD_LENGTH
    assert run([0, 9], [18], [[0, 1]])[0] & K.STATUS_BAD_LENGTH
    assert run([3, 1], [18], [[0, 1]]) == (K.STATUS_BAD_LENGTH, 0)
    assert run([0, 2], [18], [[0, 1]]) == (0, 2)                         # tokens 2, 3 belong to nobody


def _rule(x):
    """Codes and scales by the rule in fp32 on the CPU (IEEE divisions)."""
    s = x.float().abs().amax(-1) / 448.0
    c = (x.float() / torch.where(s > 0, s, 1.0)[..., None]).to(F8)
    return c, s


@pytest.mark.parametrize("T", [1, 700])
def test_append_fp8_codes_are_the_divided_quotients(K, T):
    """bf16 values and their row's maximum are small integers times powers of two, so quotients on or next to a
    border between codes are frequent; rows of every size that bf16 has, and rows whose scale's reciprocal is no
    normal number: every code and scale of V is the rule's."""
    heads, d, page = 4, 128, 64
    g = W.generator(77)
    v = torch.randn(T, heads, d, generator=g).bfloat16()
    small = (torch.randint(-128, 129, (T, heads, d), generator=g).float() * 2.0 ** torch.randint(-9, 1, (T, heads, d), generator=g)).bfloat16()
    v[:, 1] = small[:, 1]
    for i, e in enumerate((-133, -126, -118, -100, -92, -40, 40, 100, 109, 120)):  # powers of two of whole rows
        v[i % T, 2] = (small[i % T, 2].float() * 2.0 ** -7 * 2.0 ** max(e, -126) * (2.0 ** (e + 126) if e < -126 else 1.0)).bfloat16()
    v[0, 3] = 0
    lens = [T]
    cu, ln, table, n_pages = R.batch(lens, [0], page, 78)
    cos, sin = torch.ones(T, d // 2, device="cuda"), torch.zeros(T, d // 2, device="cuda")  # no rotation: K by the rule too
    kc, vc = (torch.zeros(n_pages, heads, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages, heads, page, device="cuda") for _ in range(2))
    K.kv_append_paged_rope_fp8(v.cuda(), v.cuda(), *_cuda(cu, ln, table), kc, ks, vc, vs, cos, sin)
    c, s = _rule(v)
    pg, row = R.places(cu, ln, table, page, 0)
    for codes, scales in ((kc, ks), (vc, vs)):
        assert torch.equal(scales.cpu()[pg, :, row], s)
        assert torch.equal(codes.cpu()[pg, :, row].view(F8).float(), c.float())


# ---- read back ----------------------------------------------------------------------------------

@pytest.mark.parametrize("lens,heads,d,page", [([1], 1, 64, 16), ([0, 17, 64, 130], 2, 128, 16), ([300, 5], 8, 64, 128),
                                               ([1000], 2, 128, 1024)])
def test_read_back_is_exact(K, lens, heads, d, page):
    cu, ln, table, n_pages = R.batch([0] * len(lens), lens, page, 6)
    g = W.generator(7)
    codes, s = _quant(torch.randn(2, n_pages, heads, page, d, generator=g) * torch.exp(torch.randn(2, n_pages, heads, page, 1, generator=g)))
    T_max = max(lens) + 3
    kc, vc = codes.view(torch.uint8).cuda()
    ks, vs = s.cuda()
    ko = torch.full((len(lens), heads, T_max, d), 3.0, dtype=torch.bfloat16, device="cuda")
    vo, st = ko.clone(), _status()
    K.kv_read_paged_fp8(kc, ks, vc, vs, *_cuda(table, ln), ko, vo, dev_status=st)
    assert int(st) == 0
    for x, o in ((0, ko), (1, vo)):
        want = torch.full(o.shape, 3.0).bfloat16()
        for b, l in enumerate(lens):
            pg, row = R.places(cu, ln, table, page, b)
            want[b, :, :l] = (codes[x].float()[pg, :, row] * s[x][pg, :, row][..., None]).bfloat16().transpose(0, 1)
        assert torch.equal(o.cpu(), want)


def test_read_back_flags_bad_pages_and_lengths(K):
    codes = torch.full((2, 1, 16, 64), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    s = torch.ones(2, 1, 16, device="cuda")
    ko = torch.zeros(1, 1, 40, 64, dtype=torch.bfloat16, device="cuda")

    def run(table, length):
        k, v, st = ko.clone(), ko.clone(), _status()
        K.kv_read_paged_fp8(codes, s, codes, s, *_cuda(torch.tensor([table], dtype=torch.int32), torch.tensor([length], dtype=torch.int32)), k, v, dev_status=st)
        return int(st), int((k[0, 0, :, 0] == 1).sum()), int((v[0, 0, :, 63] == 1).sum())

    assert run([1, 0], 20) == (0, 20, 20)
    assert run([1, 2], 20) == (K.STATUS_BAD_INDEX, 16, 16)
    assert run([-1, 0], 20) == (K.STATUS_BAD_INDEX, 4, 4)
    assert run([1, 0], 99) == (K.STATUS_BAD_LENGTH, 32, 32)
    assert run([1, 0], -1) == (K.STATUS_BAD_LENGTH, 0, 0)


# ---- attention ----------------------------------------------------------------------------------

def _cache(n_pages, Hk, page, d, fp8, seed, spread=1.0):
    """Pages on the GPU and what they stand for in fp64."""
    g = W.generator(seed)
    out = []
    for _ in range(2):
        x = torch.randn(n_pages, Hk, page, d, generator=g)
        if fp8:
            c, s = _quant(x * torch.exp(spread * torch.randn(n_pages, Hk, page, 1, generator=g)))
            out.append(((c.view(torch.uint8).cuda(), s.cuda()), c.double() * s.double()[..., None]))
        else:
            out.append(((x.bfloat16().cuda(),), x.bfloat16().double()))
    (kt, kd), (vt, vd) = out
    return kt + vt, kd, vd


def _chunk(K, fp8, *a, **kw):
    return (K.attn_chunk_paged_fp8 if fp8 else K.attn_chunk_paged)(*a, **kw)


def _q(T, H, d, seed, std=1.0):
    x = (torch.randn(T, (H + 3) * d, generator=W.generator(seed)) * std).bfloat16()
    return x[:, d:(H + 1) * d].view(T, H, d)


def _case(K, ns, ctx, H, Hk, d, page, fp8, seed=1, scale=None, max_q=None, extra=0, std=1.0, spread=1.0, poison=True):
    cu, lens, table, n_pages = R.batch(ns, ctx, page, seed)
    T = int(cu[-1])
    tensors, kd, vd = _cache(n_pages, Hk, page, d, fp8, seed + 1, spread)
    if poison:  # what lies behind the last row of a sequence (and in free pages) is never used
        used = torch.zeros(n_pages, page, dtype=torch.bool)
        for b in range(len(ns)):
            pg, row = R.places(cu, lens, table, page, b)
            used[pg, row] = True
        free = (~used)[:, None].expand(n_pages, Hk, page).cuda()
        for t in tensors:
            t[free] = 0x7F if t.dtype == torch.uint8 else float("nan")
    q = _q(T + extra, H, d, seed + 2, std)
    scale = d ** -0.5 if scale is None else scale
    out = torch.full((T + extra, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + extra, H), 5.0, device="cuda")
    st = _status()
    _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table), *tensors, scale, max_q=max_q, out=out, lse=lse, dev_status=st)
    ref = R.attention(q, cu, lens, table, page, kd, vd, scale, max_q=max_q, fp16_weights=fp8)
    R.check(out, lse, ref, f"{ns} {ctx} H{H} Hk{Hk} d{d} page{page} fp8={fp8}")
    unwritten = ref[1].isnan().any(-1)
    assert (out.cpu()[unwritten] == 5.0).all() and (lse.cpu()[unwritten] == 5.0).all()
    return int(st)


SHAPES = [  # ns, ctx, H, Hk, d, page
    ([1], [0], 1, 1, 64, 16),
    ([1], [0], 8, 2, 128, 16),
    ([1] * 5, [1, 15, 16, 63, 127], 8, 2, 64, 16),
    ([1] * 4, [700, 0, 64, 129], 4, 4, 128, 32),
    ([1, 1], [2000, 333], 16, 1, 128, 64),
    ([1, 1, 1], [300, 5, 128], 32, 1, 64, 32),
    ([1, 1], [300, 129], 64, 1, 128, 16),
    ([4, 5], [230, 236], 8, 2, 64, 16),
    ([7, 1, 3, 0, 8], [120, 64, 0, 40, 57], 4, 2, 128, 64),
    ([33], [0], 4, 1, 128, 32),
    ([128], [0], 2, 2, 128, 128),
    ([129, 127], [1, 128], 2, 1, 64, 16),
    ([300], [77], 4, 1, 128, 16),
    ([65, 1, 513], [1000, 900, 0], 8, 2, 128, 64),
    ([260], [515], 8, 8, 64, 64),
    ([40, 0, 9], [500, 10, 250], 64, 1, 64, 32),
    ([70], [333], 64, 1, 128, 1024),
    ([1, 1, 200, 1], [600, 20, 300, 0], 32, 8, 128, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,ctx,H,Hk,d,page", SHAPES, ids=str)
def test_attention(K, ns, ctx, H, Hk, d, page, fp8):
    assert _case(K, ns, ctx, H, Hk, d, page, fp8, max_q=max(ns)) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("n", [1, 2, 19])
def test_group_sizes(K, g, n, fp8):
    assert _case(K, [n, 1], [150, 66], 2 * g if g < 64 else g, 2 if g < 64 else 1, 128, 32, fp8, seed=g, max_q=n) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 3, 90])
def test_large_scores(K, n, fp8):
    """Scores of hundreds: the running maximum moves by far more than a rounding step between tiles."""
    assert _case(K, [n], [600], 4, 1, 128, 16, fp8, std=6.0, scale=1.0, seed=9, max_q=n) == 0


@pytest.mark.parametrize("n", [1, 90])
def test_fp8_rows_of_very_different_size(K, n):
    assert _case(K, [n], [500], 4, 1, 128, 16, True, spread=4.0, seed=10, max_q=n) == 0


@pytest.mark.parametrize("n,H,Hk,d", [(1, 8, 2, 128), (3, 8, 1, 64), (1, 32, 2, 128), (50, 4, 1, 128), (300, 2, 1, 64)])
def test_every_fp8_code(K, n, H, Hk, d):
    """Pages that hold all finite codes, subnormal ones and both zeros among them, under scales of 2^-12 .. 2^12."""
    page, ctx = 32, 400
    cu, lens, table, n_pages = R.batch([n], [ctx], page, 210)
    g = W.generator(211)
    finite = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    tensors, deq = [], []
    for _ in range(2):
        codes = finite[torch.randint(0, len(finite), (n_pages, Hk, page, d), generator=g)]
        codes[:, :, ::3] &= 0x8F  # rows of subnormal codes and the smallest normal ones
        sc = 2.0 ** torch.randint(-12, 1, (n_pages, Hk, page), generator=g).float() * (1 + torch.rand(n_pages, Hk, page, generator=g)) / 448
        tensors += [codes.cuda(), sc.cuda()]
        deq.append(codes.view(F8).double() * sc.double()[..., None])
    q, st = _q(n, H, d, 212), _status()
    out, lse = K.attn_chunk_paged_fp8(q.cuda(), *_cuda(cu, lens, table), *tensors, 0.5, max_q=n, dev_status=st)
    assert int(st) == 0
    R.check(out, lse, R.attention(q, cu, lens, table, page, *deq, 0.5, fp16_weights=True), "all codes")


@pytest.mark.parametrize("e", [-60, 0, 60])
@pytest.mark.parametrize("n", [1, 40])
def test_fp8_queries_of_any_size(K, n, e):
    """Query rows around 2^e, elements of a row up to 2^12 apart, one row zero: FP8 attention takes them through fp16."""
    page, d, H, Hk, ctx = 16, 128, 4, 2, 200
    cu, lens, table, n_pages = R.batch([n], [ctx], page, 220)
    tensors, kd, vd = _cache(n_pages, Hk, page, d, True, 221)
    g = W.generator(222)
    q = (torch.randn(n, H, d, generator=g) * 2.0 ** torch.randint(-12, 1, (n, H, d), generator=g) * 2.0 ** e).bfloat16()
    q[0, 1] = 0
    scale = 2.0 ** -e
    out, lse = K.attn_chunk_paged_fp8(q.cuda(), *_cuda(cu, lens, table), *tensors, scale, max_q=n)
    R.check(out, lse, R.attention(q, cu, lens, table, page, kd, vd, scale, fp16_weights=True), f"2^{e}")


@pytest.mark.parametrize("e", [-80, 0, 80])
@pytest.mark.parametrize("n", [1, 40, 90])
def test_fp8_values_of_any_size(K, n, e):
    """Value rows around 2^e, e^3 apart (one standard deviation), every seventh zero: their scales enter the
    running reference as logarithms, and a zero row still takes its share of the sum."""
    page, d, H, Hk, ctx = 32, 128, 4, 2, 400
    cu, lens, table, n_pages = R.batch([n], [ctx], page, 230)
    (kc, ks, vc, vs), kd, vd = _cache(n_pages, Hk, page, d, True, 231, spread=3.0)
    vs *= 2.0 ** e
    vd = vd * 2.0 ** e
    vc[:, :, ::7], vs[:, :, ::7], vd[:, :, ::7] = 0, 0.0, 0.0
    q = _q(n, H, d, 232, 0.3)
    out, lse = K.attn_chunk_paged_fp8(q.cuda(), *_cuda(cu, lens, table), kc, ks, vc, vs, d ** -0.5, max_q=n)
    R.check(out, lse, R.attention(q, cu, lens, table, page, kd, vd, d ** -0.5, fp16_weights=True), f"2^{e}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,ctx,H,Hk,d", [([300, 1, 70], [200, 900, 0], 8, 2, 128), ([260, 40], [130, 1], 8, 1, 64)])
def test_page_tables_far_wider_than_the_sequences(K, ns, ctx, H, Hk, d, fp8):
    """Room for 256K rows a sequence; the entries past a sequence's last row are no pages."""
    page = 64
    cu, lens, table, n_pages = R.batch(ns, ctx, page, 240)
    table = torch.cat([table, torch.full((len(ns), 4096 - table.shape[1]), -7, dtype=torch.int32)], 1).contiguous()
    tensors, kd, vd = _cache(n_pages, Hk, page, d, fp8, 241)
    q, st = _q(int(cu[-1]), H, d, 242), _status()
    out, lse = _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table), *tensors, d ** -0.5, max_q=max(ns), dev_status=st)
    assert int(st) == 0
    R.check(out, lse, R.attention(q, cu, lens, table, page, kd, vd, d ** -0.5, fp16_weights=fp8), "wide tables")


@pytest.mark.parametrize("e", [-80, 0, 80])
def test_fp8_values_of_any_size_in_long_room(K, e):
    """test_fp8_values_of_any_size where the sequences have room for far more rows."""
    page, d, H, Hk, n, ctx = 64, 128, 8, 2, 150, 700
    cu, lens, table, n_pages = R.batch([n], [ctx], page, 250)
    table = torch.cat([table, torch.full((1, 4096 - table.shape[1]), -1, dtype=torch.int32)], 1).contiguous()
    (kc, ks, vc, vs), kd, vd = _cache(n_pages, Hk, page, d, True, 251, spread=3.0)
    vs *= 2.0 ** e
    vd = vd * 2.0 ** e
    vc[:, :, ::7], vs[:, :, ::7], vd[:, :, ::7] = 0, 0.0, 0.0
    q = _q(n, H, d, 252, 0.3)
    out, lse = K.attn_chunk_paged_fp8(q.cuda(), *_cuda(cu, lens, table), kc, ks, vc, vs, d ** -0.5, max_q=n)
    R.check(out, lse, R.attention(q, cu, lens, table, page, kd, vd, d ** -0.5, fp16_weights=True), f"2^{e}")


@pytest.mark.parametrize("fp8", [False, True])
def test_without_a_bound_on_the_chunks(K, fp8):
    assert _case(K, [1, 1, 1], [100, 30, 0], 8, 2, 128, 16, fp8, max_q=None) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,heads", [(1, (4, 4)), (5, (8, 1)), (100, (4, 2))])
def test_tokens_behind_the_last_sequence_stay_as_they_were(K, n, heads, fp8):
    assert _case(K, [n, n], [60, 200], *heads, 128, 16, fp8, extra=7, max_q=n) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hk", [(4, 1), (64, 1)])
def test_a_chunk_longer_than_its_bound(K, H, Hk, fp8):
    """The tokens past max_q are left unwritten, the others are right, and the call says so."""
    assert _case(K, [6, 40, 3], [100, 70, 8], H, Hk, 64, 16, fp8, max_q=6) == K.STATUS_BAD_LENGTH


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [2, 60])
def test_sequences_shorter_than_their_chunk_and_empty_ones(K, n, fp8):
    """seq_lens < n: the first tokens stand before row 0 and see nothing: zeros and -inf."""
    assert _case(K, [n, n, 0, n], [10, -n // 2, 4, -n], 8, 2, 128, 16, fp8, max_q=n) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,H,Hk", [(1, 8, 2), (3, 4, 2), (70, 4, 1)])
def test_bad_pages_are_skipped(K, n, H, Hk, fp8):
    page, d = 16, 128
    ns, ctx = [n, n], [200, 40]
    cu, lens, table, n_pages = R.batch(ns, ctx, page, 21)
    table[0, 0], table[0, 3], table[0, 9] = -1, n_pages, 1 << 30
    table[1, :] = -5  # a sequence with no page at all
    tensors, kd, vd = _cache(n_pages, Hk, page, d, fp8, 22)
    q, st = _q(2 * n, H, d, 23), _status()
    out, lse = _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table), *tensors, 0.1, max_q=n, dev_status=st)
    assert int(st) == K.STATUS_BAD_INDEX
    R.check(out, lse, R.attention(q, cu, lens, table, page, kd, vd, 0.1, fp16_weights=fp8), "bad pages")
    assert (out[n:] == 0).all() and (lse[n:] == float("-inf")).all()


@pytest.mark.parametrize("n", [1, 80])
def test_batch_data_out_of_range_is_forced_into_it(K, n):
    """Lengths and offsets that no host check sees: flagged, and nothing stray is read or written."""
    page, d, H, Hk = 16, 64, 4, 2
    cu, lens, table, n_pages = R.batch([n, n], [40, 90], page, 31)
    tensors, kd, vd = _cache(n_pages, Hk, page, d, False, 32)
    q = _q(2 * n, H, d, 33).cuda()
    for c, l in (([0, n, 5 * n], [40 + n, 90 + n]), ([-3, n, 2 * n], [40 + n, 90 + n]), ([0, n, 2 * n], [-7, 1 << 30]),
                 ([2 * n, n, 0], [9, 9])):
        st = _status()
        K.attn_chunk_paged(q, *_cuda(torch.tensor(c, dtype=torch.int32), torch.tensor(l, dtype=torch.int32),
                                     table.clamp(min=0)), *tensors, 0.1, max_q=n, dev_status=st)
        assert int(st) & K.STATUS_BAD_LENGTH


def test_long_cache_few_heads(K):
    """Work split over a long axis: one sequence, one KV head, 20000 rows, one to three tokens."""
    for fp8 in (False, True):
        for n in (1, 3):
            assert _case(K, [n], [20000 - n], 8, 1, 128, 64, fp8, seed=41, max_q=n, poison=False) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,ctx,H,Hk,d", [([40], [19960], 4, 1, 128), ([1, 33, 1], [9000, 6000, 5], 8, 1, 64),
                                           ([260], [9000], 1, 1, 128), ([9], [20000], 64, 1, 128)])
def test_blocks_shared_by_many_ctas(K, ns, ctx, H, Hk, d, fp8):
    """Few blocks of query rows over long caches: one block's keys are spread over most of the card."""
    assert _case(K, ns, ctx, H, Hk, d, 64, fp8, seed=45, max_q=max(ns), poison=False) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,ctx,H,Hk,d", [([2, 2, 1], [1500, 700, 40], 64, 8, 128), ([2, 1], [5000, 900], 16, 2, 64)])
def test_sixteen_rows_a_head_shared_by_ctas(K, ns, ctx, H, Hk, d, fp8):
    assert _case(K, ns, ctx, H, Hk, d, 64, fp8, seed=260, max_q=2) == 0


def test_many_sequences(K):
    ns = [1 + (b % 3) for b in range(300)]
    ctx = [(b * 37) % 150 for b in range(300)]
    for fp8 in (False, True):
        assert _case(K, ns, ctx, 4, 2, 64, 16, fp8, seed=43, max_q=3) == 0
        assert _case(K, ns, ctx, 32, 1, 64, 16, fp8, seed=44, max_q=3) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(K, fp8):
    """A pool of more than 2^31 elements whose last pages are the ones in use."""
    page, d, Hk, H = 64, 128, 2, 8
    n_pages = (1 << 31) // (page * d * Hk) + 40
    pool = [torch.empty(n_pages, Hk, page, d, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2)]
    scales = [torch.empty(n_pages, Hk, page, device="cuda") for _ in range(2)] if fp8 else []
    ns, ctx = [2, 130], [300, 500]
    cu, lens, table, small = R.batch(ns, ctx, page, 51)
    assert small <= 40
    tensors, kd, vd = _cache(small, Hk, page, d, fp8, 52)
    big = n_pages - 40
    tens = list(tensors)
    if fp8:
        for dst, src in zip((pool[0], scales[0], pool[1], scales[1]), tens):
            dst[big:big + small] = src
        args = (pool[0], scales[0], pool[1], scales[1])
    else:
        for dst, src in zip(pool, tens):
            dst[big:big + small] = src
        args = tuple(pool)
    q, st = _q(132, H, d, 53), _status()
    out, lse = _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table + big), *args, 0.1, dev_status=st)
    assert int(st) == 0
    R.check(out, lse, R.attention(q, cu, lens, table, page, kd, vd, 0.1, fp16_weights=fp8), "big pool")
    if fp8:
        ko = torch.zeros(2, Hk, 640, d, dtype=torch.bfloat16, device="cuda")
        vo = ko.clone()
        K.kv_read_paged_fp8(*args, *_cuda(table + big, lens), ko, vo)
        pg, row = R.places(cu, lens, table, page, 1)
        assert torch.equal(vo[1, :, :630].cpu().double(), vd[pg, :, row].transpose(0, 1).float().bfloat16().double())
    # the append's addresses, on the last page
    k = W.normal_bf16((3, Hk, d), W.generator(54)).cuda()
    cos, sin = _tables(K, d, 64)
    c3, l3, t3 = _cuda(*(torch.tensor(x, dtype=torch.int32) for x in ([0, 3], [3], [[n_pages - 1]])))
    if fp8:
        K.kv_append_paged_rope_fp8(k, k, c3, l3, t3, *args, cos, sin)
        got = args[2][-1, :, :3].view(F8).float() * args[3][-1, :, :3][..., None]
        assert (got - k.transpose(0, 1).float()).abs().max() <= 2.0 ** -4 * k.abs().max()
    else:
        K.kv_append_paged_rope(k, k, c3, l3, t3, *args, cos, sin)
        assert torch.equal(args[1][-1, :, :3], k.transpose(0, 1))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,ctx", [(1, 9000), (6, 3000), (400, 700)])
def test_repeated_calls_give_the_same_bits(K, fp8, n, ctx):
    page, d, H, Hk = 64, 128, 8, 2
    cu, lens, table, n_pages = R.batch([n, n], [ctx, ctx // 3], page, 61)
    tensors, _, _ = _cache(n_pages, Hk, page, d, fp8, 62)
    q = _q(2 * n, H, d, 63).cuda()
    b = _cuda(cu, lens, table)
    ws = K.workspace(K.attn_chunk_paged_workspace_bytes(2, 2 * n, n, H, Hk, d))
    first = _chunk(K, fp8, q, *b, *tensors, 0.1, max_q=n, ws=ws)
    assert not ws[:65536].any()
    for _ in range(3):
        again = _chunk(K, fp8, q, *b, *tensors, 0.1, max_q=n, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 70])
def test_one_workspace_for_calls_of_other_shapes(K, fp8, n):
    """A workspace left behind by a call of another shape serves the next one."""
    ws = K.workspace(max(K.attn_chunk_paged_workspace_bytes(4, 300, m, 64, 1, 128) for m in (1, 5, 70)))
    for ns, ctx, H, Hk in (([n, n], [4000, 30], 8, 2), ([n], [900], 64, 1), ([n] * 3, [10, 3000, 0], 4, 4)):
        cu, lens, table, n_pages = R.batch(ns, ctx, 32, 71)
        tensors, kd, vd = _cache(n_pages, Hk, 32, 128, fp8, 72)
        q = _q(int(cu[-1]), H, 128, 73)
        out, lse = _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table), *tensors, 0.09, max_q=n, ws=ws)
        R.check(out, lse, R.attention(q, cu, lens, table, 32, kd, vd, 0.09, fp16_weights=fp8), f"{ns} {ctx}")


@pytest.mark.parametrize("fp8", [False, True])
def test_one_workspace_for_both_kinds_of_call(K, fp8):
    """Single tokens, chunks, then single tokens again on one workspace; its counters are zero after each."""
    ws = K.workspace(max(K.attn_chunk_paged_workspace_bytes(3, 400, m, 8, 1, 128) for m in (1, 4, 130)))
    for turn, (ns, ctx) in enumerate((([1, 1], [9000, 30]), ([130, 1], [900, 3000]), ([4, 1, 2], [5000, 0, 77]), ([1], [12000]))):
        cu, lens, table, n_pages = R.batch(ns, ctx, 64, 75)
        tensors, kd, vd = _cache(n_pages, 1, 64, 128, fp8, 76)
        q = _q(int(cu[-1]), 8, 128, 77)
        out, lse = _chunk(K, fp8, q.cuda(), *_cuda(cu, lens, table), *tensors, 0.09, max_q=max(ns), ws=ws)
        R.check(out, lse, R.attention(q, cu, lens, table, 64, kd, vd, 0.09, fp16_weights=fp8), f"turn {turn}")
        assert not ws[:65536].any()


def test_small_workspaces_and_foreign_tensors_are_refused(K):
    cu, lens, table, n_pages = R.batch([1], [30], 16, 81)
    tensors, _, _ = _cache(n_pages, 2, 16, 64, False, 82)
    q = _q(1, 8, 64, 83).cuda()
    b = _cuda(cu, lens, table)
    need = K.attn_chunk_paged_workspace_bytes(1, 1, 1, 8, 2, 64)
    with pytest.raises(K.KvattnError) as e:
        K.attn_chunk_paged(q, *b, *tensors, 0.1, ws=torch.zeros(need - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -6
    with pytest.raises(TypeError):
        K.attn_chunk_paged(q, b[0].cpu(), *b[1:], *tensors, 0.1)
    with pytest.raises(TypeError):
        K.attn_chunk_paged(q.float(), *b, *tensors, 0.1)
    with pytest.raises(ValueError):
        K.attn_chunk_paged(q, b[0][:1], *b[1:], *tensors, 0.1)
    with pytest.raises(ValueError):
        K.attn_chunk_paged(q[:, ::2], *b, *tensors, 0.1)
    with pytest.raises(ValueError):
        K.attn_chunk_paged(q, *b, tensors[0], tensors[1][:1], 0.1)
    assert K.attn_chunk_paged(q[:0], *b, *tensors, 0.1)[0].shape == (0, 8, 64)


# ---- runs of them together ----------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,H,Hk", [(128, 8, 2), (64, 4, 1)])
def test_serving_steps_against_one_causal_pass(K, fp8, d, H, Hk):
    """Two sequences served in steps (a prompt in two chunks, guessed tokens, single tokens; the other
    sequence joins later): every step's append and attention against the fp64 statement over the whole
    of each sequence, from the rows that the cache holds."""
    page, scale = 16, d ** -0.5
    steps = [([70, 0], 0), ([61, 9], 1), ([4, 3], 2), ([1, 1], 3), ([1, 1], 4), ([0, 130], 5)]
    cos, sin = _tables(K, d, 256)
    n_pages = 24
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(2, 12).cuda()
    rows = torch.uint8 if fp8 else torch.bfloat16
    kp, vp = (torch.zeros(n_pages, Hk, page, d, dtype=rows, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages, Hk, page, device="cuda") for _ in range(2))
    have = [0, 0]
    st = _status()
    for ns, i in steps:
        T = sum(ns)
        qkv = W.normal_bf16((T, (H + 2 * Hk) * d), W.generator(100 + i)).cuda()
        q, k, v = (x.view(T, -1, d) for x in qkv.split([H * d, Hk * d, Hk * d], -1))
        have = [a + b for a, b in zip(have, ns)]
        cu = torch.tensor([0, ns[0], T], dtype=torch.int32)
        lens = torch.tensor(have, dtype=torch.int32)
        b = _cuda(cu, lens) + [table]
        pos = torch.cat([torch.arange(l - n, l) for n, l in zip(ns, have)]).to(torch.int32).cuda()
        K.rope_apply_qk(q[None], pos[None], None, None, cos, sin, q_layout="bthd", dev_status=st)
        if fp8:
            K.kv_append_paged_rope_fp8(k, v, *b, kp, ks, vp, vs, cos, sin, dev_status=st)
            out, lse = K.attn_chunk_paged_fp8(q, *b, kp, ks, vp, vs, scale, max_q=max(ns), dev_status=st)
            kd, vd = (c.cpu().view(F8).double() * s.cpu().double()[..., None] for c, s in ((kp, ks), (vp, vs)))
        else:
            K.kv_append_paged_rope(k, v, *b, kp, vp, cos, sin, dev_status=st)
            out, lse = K.attn_chunk_paged(q, *b, kp, vp, scale, max_q=max(ns), dev_status=st)
            kd, vd = kp.cpu().double(), vp.cpu().double()
        R.check(out, lse, R.attention(q.cpu(), cu, lens, table.cpu(), page, kd, vd, scale, fp16_weights=fp8), f"step {i}")
    assert int(st) == 0


def test_a_prompt_in_chunks_agrees_with_the_prefill(K):
    """A prompt appended and attended in three chunks, against attn_prefill_causal on the same rows: both are
    within the bf16 bound of the exact result, so they differ by at most twice that."""
    d, H, Hk, page, scale = 128, 8, 2, 64, 128 ** -0.5
    T, cuts = 520, [0, 200, 201, 520]
    g = W.generator(5)
    q, k, v = W.normal_bf16((T, H, d), g), W.normal_bf16((T, Hk, d), g), W.normal_bf16((T, Hk, d), g)
    want, wlse = K.attn_prefill_causal(q[None].cuda(), *(x.transpose(0, 1)[None].contiguous().cuda() for x in (k, v)), scale)
    table = torch.randperm(9, generator=torch.Generator().manual_seed(2)).to(torch.int32)[None].cuda()
    kp, vp = (torch.zeros(9, Hk, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cos, sin = torch.ones(T, d // 2, device="cuda"), torch.zeros(T, d // 2, device="cuda")  # no rotation
    got, glse = [], []
    for a, b in zip(cuts, cuts[1:]):
        cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, b - a], [b]))
        K.kv_append_paged_rope(k[a:b].cuda(), v[a:b].cuda(), cu, lens, table, kp, vp, cos, sin)
        o, l = K.attn_chunk_paged(q[a:b].cuda(), cu, lens, table, kp, vp, scale)
        got.append(o)
        glse.append(l)
    cu, lens = torch.tensor([0, T], dtype=torch.int32), torch.tensor([T], dtype=torch.int32)
    _, _, ot, lt = R.attention(q, cu, lens, table.cpu(), page, kp.cpu().double(), vp.cpu().double(), scale)
    assert ((torch.cat(got).double() - want[0].double()).abs().cpu() <= 2 * ot).all()
    assert ((torch.cat(glse).double() - wlse[0].T.double()).abs().cpu() <= 2 * lt).all()


def test_an_fp8_cache_read_back_serves_the_contiguous_decode(K):
    """Append in FP8, attend from the pages; read the cache back and decode from it.  The read rows are
    bf16-rounded, the pages are not: a score moves by at most u16 S, a value by u16 |v|."""
    d, H, Hk, page, scale, L = 128, 8, 2, 32, 128 ** -0.5, 333
    g = W.generator(6)
    q, k, v = W.normal_bf16((1, H, d), g), W.normal_bf16((L, Hk, d), g), W.normal_bf16((L, Hk, d), g)
    cos, sin = _tables(K, d, L)
    table = torch.randperm(11, generator=torch.Generator().manual_seed(3)).to(torch.int32)[None]
    kc, vc = (torch.zeros(11, Hk, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(11, Hk, page, device="cuda") for _ in range(2))
    lens, cu = torch.tensor([L], dtype=torch.int32), torch.tensor([0, L], dtype=torch.int32)
    K.kv_append_paged_rope_fp8(k.cuda(), v.cuda(), *_cuda(cu, lens, table), kc, ks, vc, vs, cos, sin)
    one = torch.tensor([0, 1], dtype=torch.int32)
    a, al = K.attn_chunk_paged_fp8(q.cuda(), *_cuda(one, lens, table), kc, ks, vc, vs, scale)
    ko, vo = (torch.zeros(1, Hk, L, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K.kv_read_paged_fp8(kc, ks, vc, vs, *_cuda(table, lens), ko, vo)
    b, bl = K.attn_decode_gqa(q.cuda(), ko, vo, lens.cuda(), scale)
    kd, vd = (c.cpu().view(F8).double() * s.cpu().double()[..., None] for c, s in ((kc, ks), (vc, vs)))
    ref = R.attention(q, one, lens, table, page, kd, vd, scale, fp16_weights=True)
    R.check(a, al, ref, "pages")
    pg, row = R.places(one, lens, table, page, 0)
    S = max(float((q[0, j].double().abs() @ kd[pg, j // 4, row].abs().T).max()) for j in range(H)) * scale
    move = R.U16 * S
    A = vd[pg, :, row].abs().amax(0).repeat_interleave(4, 0)  # [H, d]: an average of |v| is at most its largest
    assert ((b.cpu().double()[0] - ref[0][0]).abs() <= ref[2][0] + (2 * np.expm1(2 * move) + R.U16) * A).all()
    assert ((bl.cpu().double()[0] - ref[1][0]).abs() <= ref[3][0] + move).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 40])
def test_captured_and_replayed_on_another_stream(K, fp8, n):
    """An append and an attention captured into a graph on a side stream, replayed after the batch's
    lengths and tokens changed in place: the replay follows the device data."""
    page, d, H, Hk, scale = 16, 128, 8, 2, 0.1
    cu, lens, table, n_pages = R.batch([n, n], [50, 200], page, 91, max_pages=40)
    table = torch.arange(2 * 40, dtype=torch.int32).view(2, 40)
    n_pages = 80
    tensors, _, _ = _cache(n_pages, Hk, page, d, fp8, 92)
    q = _q(2 * n, H, d, 93).contiguous().cuda()
    k, v = (W.normal_bf16((2 * n, Hk, d), W.generator(94 + i)).cuda() for i in range(2))
    cos, sin = _tables(K, d, 640)
    b = _cuda(cu, lens, table)
    out, lse, st = torch.zeros_like(q), torch.zeros(2 * n, H, device="cuda"), _status()
    ws = K.workspace(K.attn_chunk_paged_workspace_bytes(2, 2 * n, n, H, Hk, d))

    def step():
        (K.kv_append_paged_rope_fp8 if fp8 else K.kv_append_paged_rope)(k, v, *b, *tensors, cos, sin, dev_status=st)
        _chunk(K, fp8, q, *b, *tensors, scale, max_q=n, out=out, lse=lse, ws=ws, dev_status=st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warm-up before the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for turn in range(2):
        lens2 = torch.tensor([300 + turn * 7 + n, 64 + n], dtype=torch.int32)
        b[1].copy_(lens2)
        q.copy_(_q(2 * n, H, d, 95 + turn))
        k.copy_(W.normal_bf16((2 * n, Hk, d), W.generator(97 + turn)))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        side.synchronize()
        assert int(st) == 0
        if fp8:
            kd, vd = (c.cpu().view(F8).double() * s.cpu().double()[..., None] for c, s in ((tensors[0], tensors[1]), (tensors[2], tensors[3])))
        else:
            kd, vd = (t.cpu().double() for t in tensors)
        R.check(out, lse, R.attention(q.cpu(), cu, lens2, table, page, kd, vd, scale, fp16_weights=fp8), f"replay {turn}")


@pytest.mark.parametrize("fp8", [False, True])
def test_two_streams_with_a_workspace_each(K, fp8):
    """Two calls in flight at once, each with its own workspace."""
    page, d, H, Hk = 32, 128, 8, 2
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for i, (n, ctx) in enumerate(((1, 5000), (130, 2000))):
        cu, lens, table, n_pages = R.batch([n, n], [ctx, 40], page, 101 + i)
        tensors, kd, vd = _cache(n_pages, Hk, page, d, fp8, 103 + i)
        q = _q(2 * n, H, d, 105 + i)
        calls.append((q, cu, lens, table, kd, vd, q.cuda(), _cuda(cu, lens, table), tensors, n,
                      K.workspace(K.attn_chunk_paged_workspace_bytes(2, 2 * n, n, H, Hk, d))))
    torch.cuda.synchronize()
    outs = []
    for turn in range(3):
        outs = []
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                outs.append(_chunk(K, fp8, c[6], *c[7], *c[8], 0.1, max_q=c[9], ws=c[10]))
    torch.cuda.synchronize()
    for o, c in zip(outs, calls):
        R.check(*o, R.attention(c[0], c[1], c[2], c[3], page, c[4], c[5], 0.1, fp16_weights=fp8), "two streams")
