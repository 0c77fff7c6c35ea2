"""The paged-cache operators refuse bad arguments on the host, before any launch.  CPU only:
the pointers are never dereferenced."""
import ctypes

import pytest

from mqa_kv_cache_b200 import build as kbuild

vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
FAKE = vp(1 << 20)
OFF = vp((1 << 20) + 8)  # not 16-byte aligned
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = -1, -3, -2, -4, -6


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(kbuild.build())
    head = [vp, i64, vp, i64, vp, vp, vp] + [i32] * 7
    lib.kv_append_paged_rope.argtypes = head + [vp, vp, vp, vp, i32, i32, vp, vp]
    lib.kv_append_paged_rope_fp8.argtypes = head + [vp, vp, vp, vp, vp, vp, i32, i32, vp, vp]
    lib.kv_read_paged_fp8.argtypes = [vp] * 6 + [i32] * 7 + [vp, vp, vp, vp]
    chunk = [vp, i64, vp, vp, vp] + [i32] * 9
    lib.attn_chunk_paged.argtypes = chunk + [vp, vp, f32, vp, vp, vp, sz, vp, vp]
    lib.attn_chunk_paged_fp8.argtypes = chunk + [vp, vp, vp, vp, f32, vp, vp, vp, sz, vp, vp]
    lib.attn_chunk_paged_workspace_bytes.argtypes = [i32] * 6
    lib.attn_chunk_paged_workspace_bytes.restype = sz
    lib.kvattn_last_error_string.restype = ctypes.c_char_p
    return lib


SIZES = dict(B=2, n_tokens=5, heads=2, d=64, page=16, max_pages=4, n_pages=9)

# (what is changed, the code expected), for every call that takes a batch
BATCH = [(dict(B=0), SHAPE), (dict(B=1025), SHAPE), (dict(n_tokens=-1), SHAPE), (dict(heads=0), SHAPE),
         (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
         (dict(page=2048), UNSUPPORTED), (dict(max_pages=0), SHAPE), (dict(max_pages=(1 << 26) + 1), SHAPE),
         (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 30), SHAPE), (dict(n_tokens=1 << 30), SHAPE),
         (dict(B=1024, heads=32, n_pages=9), UNSUPPORTED)]


def _append(lib, fp8=False, k=FAKE, v=FAKE, cu=FAKE, lens=FAKE, table=FAKE, stride=None, out=FAKE, scales=FAKE,
            cos=FAKE, max_pos=64, pair=0, **change):
    s = {**SIZES, **change}
    stride = s["heads"] * s["d"] if stride is None else stride
    head = (k, stride, v, stride, cu, lens, table, s["B"], s["n_tokens"], s["heads"], s["d"], s["page"],
            s["max_pages"], s["n_pages"])
    if fp8:
        return lib.kv_append_paged_rope_fp8(*head, out, scales, out, scales, cos, FAKE, max_pos, pair, None, None)
    return lib.kv_append_paged_rope(*head, out, out, cos, FAKE, max_pos, pair, None, None)


def _read(lib, codes=FAKE, scales=FAKE, table=FAKE, lens=FAKE, T_max=64, out=FAKE, **change):
    s = {**SIZES, **change}
    return lib.kv_read_paged_fp8(codes, scales, codes, scales, table, lens, s["B"], s["heads"], s["d"], s["page"],
                                 s["max_pages"], s["n_pages"], T_max, out, out, None, None)


def _chunk(lib, fp8=False, q=FAKE, cu=FAKE, lens=FAKE, table=FAKE, stride=None, pages=FAKE, scales=FAKE, scale=0.1,
           out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, g=2, max_q=0, **change):
    s = {**SIZES, **change}
    H = s["heads"] * g
    stride = H * s["d"] if stride is None else stride
    head = (q, stride, cu, lens, table, s["B"], s["n_tokens"], max_q, H, s["heads"], s["d"], s["page"],
            s["max_pages"], s["n_pages"])
    if fp8:
        return lib.attn_chunk_paged_fp8(*head, pages, scales, pages, scales, scale, out, lse, ws, ws_bytes, None, None)
    return lib.attn_chunk_paged(*head, pages, pages, scale, out, lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize("change,code", BATCH, ids=lambda x: str(x))
def test_sizes_are_refused_by_every_call(lib, change, code):
    for fp8 in (False, True):
        assert _append(lib, fp8, **change) == code
        assert _chunk(lib, fp8, **change) == code
    if "n_tokens" not in change:
        assert _read(lib, **change) == code
    assert lib.kvattn_last_error_string()


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(lib, fp8):
    for name in ("k", "v", "cu", "lens", "table", "out", "cos"):
        assert _append(lib, fp8, **{name: None}) == NULL, name
    for name in ("k", "v", "out", "cos"):
        assert _append(lib, fp8, **{name: OFF}) == ALIGN, name
    assert _append(lib, fp8, stride=132) == ALIGN
    assert _append(lib, fp8, stride=64) == SHAPE
    assert _append(lib, fp8, pair=2) == UNSUPPORTED
    assert _append(lib, fp8, max_pos=0) == SHAPE
    if fp8:
        assert _append(lib, fp8, scales=None) == NULL
        assert _append(lib, fp8, scales=OFF) == ALIGN


def test_read_refusals(lib):
    for name in ("codes", "scales", "table", "lens", "out"):
        assert _read(lib, **{name: None}) == NULL, name
    for name in ("codes", "scales", "out"):
        assert _read(lib, **{name: OFF}) == ALIGN, name
    assert _read(lib, T_max=0) == SHAPE


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_refusals(lib, fp8):
    for name in ("q", "cu", "lens", "table", "pages", "out"):
        assert _chunk(lib, fp8, **{name: None}) == NULL, name
    for name in ("q", "pages", "out"):
        assert _chunk(lib, fp8, **{name: OFF}) == ALIGN, name
    assert _chunk(lib, fp8, lse=vp((1 << 20) + 2)) == ALIGN
    for g in (3, 5, 128):
        assert _chunk(lib, fp8, g=g) == UNSUPPORTED
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _chunk(lib, fp8, scale=scale) == SHAPE
    assert _chunk(lib, fp8, stride=260) == ALIGN
    assert _chunk(lib, fp8, stride=128) == SHAPE
    if fp8:
        assert _chunk(lib, fp8, scales=None) == NULL
        assert _chunk(lib, fp8, scales=OFF) == ALIGN


def test_empty_calls_do_nothing(lib):
    assert _append(lib, n_tokens=0, k=None, v=None) == 0
    assert _append(lib, True, n_tokens=0, k=None, v=None) == 0
    assert _chunk(lib, n_tokens=0, q=None, out=None, ws=None, ws_bytes=0) == 0
    assert _chunk(lib, True, n_tokens=0, q=None, out=None, ws=None, ws_bytes=0) == 0


def test_workspace_query_rejects_bad_heads(lib):
    q = lib.attn_chunk_paged_workspace_bytes
    assert q(0, 1, 1, 8, 2, 64) == 0 and q(1, 1, 1, 8, 3, 64) == 0 and q(1, 1, 1, 0, 1, 64) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    from mqa_kv_cache_b200 import kvattn as K
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        K.attn_chunk_paged(q, i, i[:1], i[None], pages, pages, 0.1)
    with pytest.raises(TypeError):
        K.kv_append_paged_rope(q, q, i, i[:1], i[None], pages, pages, i, i)
    with pytest.raises(TypeError):
        K.kv_read_paged_fp8(pages, i, pages, i, i[None], i, pages, pages)
