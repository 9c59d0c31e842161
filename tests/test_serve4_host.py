"""The rotated append and the 4-bit calls without a GPU: refusals on the host
before any launch."""
import ctypes

import pytest
import torch

import serve4_util
from causal_streaming_softmax_gb300 import api, build

P = 0x10000
PAGE = 16 * 36  # bytes of a page of one head


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def paged(four, **kw):
    base = dict(batch=3, tokens=10, heads=4, kv_heads=2, head_dim=64, page_size=16, num_pages=50,
                table_width=8, max_new=4, dtype=1, scale=0.125, q_token=256, q_head=64,
                o_token=256, o_head=64, k_token=128, k_head=64, v_token=128, v_head=64,
                kc_page=2048, kc_head=1024, kc_row=64, vc_page=2048, vc_head=1024, vc_row=64)
    if four:
        base.update(kc_page=2 * PAGE, kc_head=PAGE, kc_row=-3, vc_page=2 * PAGE, vc_head=PAGE,
                    vc_row=0)
    base.update(kw)
    return api.AttnPagedShape(**base)


def append(lib, four, s, q=P, k=2 * P, v=3 * P, cos=P, sin=P, angles=100, slots=P, cu=P, lens=P,
           out=4 * P, kc=5 * P, vc=6 * P):
    f = lib.attn_paged_append4 if four else lib.attn_paged_append
    return f(None if s is None else ctypes.byref(s), q, k, v, cos, sin, angles, slots, cu, lens,
             out, kc, vc, None)


def load(lib, s, slots=P, kc=P, vc=P, k=P, v=2 * P):
    return lib.attn_paged_load4(None if s is None else ctypes.byref(s), slots, kc, vc, k, v, None)


def fwd4(lib, s, q=P, k=P, v=P, table=P, cu=P, lens=P, ws=P, n=1 << 40, o=P, lse=None):
    return lib.attn_paged_fwd4(None if s is None else ctypes.byref(s), q, k, v, table, cu, lens,
                               ws, n, o, lse, None)


COMMON = [dict(batch=0), dict(batch=4097), dict(tokens=-1), dict(page_size=4), dict(page_size=24),
          dict(page_size=2048), dict(num_pages=0), dict(num_pages=1 << 27), dict(table_width=0),
          dict(kv_heads=0), dict(head_dim=32), dict(dtype=7)]
ROWS = [dict(q_token=8), dict(q_head=60), dict(k_token=-128), dict(k_head=68), dict(v_head=0),
        dict(o_token=64), dict(o_head=1 << 38), dict(heads=5), dict(heads=258)]
POOL16 = [dict(kc_page=0), dict(kc_row=65), dict(vc_head=-1024), dict(vc_row=32),
          dict(kc_page=1024)]
POOL4 = [dict(kc_page=PAGE), dict(kc_head=PAGE - 16), dict(vc_page=2 * PAGE + 8),
         dict(vc_head=-PAGE), dict(vc_page=1 << 40), dict(kc_page=PAGE, kc_head=49 * PAGE)]


@pytest.mark.parametrize("kw", COMMON + ROWS + POOL16)
def test_append_shape_refused(lib, kw):
    assert append(lib, False, paged(False, **kw)) == api.ATTN_ERR_SHAPE


@pytest.mark.parametrize("kw", COMMON + ROWS + POOL4)
def test_append4_shape_refused(lib, kw):
    assert append(lib, True, paged(True, **kw)) == api.ATTN_ERR_SHAPE
    if not set(kw) & {"q_token", "q_head", "o_token", "o_head", "heads"}:
        assert append(lib, True, paged(True, **kw), q=None, cos=None, sin=None, cu=None, lens=None,
                      out=None) == api.ATTN_ERR_SHAPE


@pytest.mark.parametrize("four", [False, True])
def test_append_pointers_refused(lib, four):
    s = paged(four)
    assert append(lib, four, None) == api.ATTN_ERR_NULL
    for name in ("q", "k", "v", "cos", "sin", "slots", "cu", "lens", "out", "kc", "vc"):
        assert append(lib, four, s, **{name: None}) == api.ATTN_ERR_NULL, name
        assert append(lib, four, s, **{name: P + 2}) == api.ATTN_ERR_ALIGN, name
    for name in ("q", "k", "v", "cos", "sin", "out", "kc", "vc"):
        assert append(lib, four, s, **{name: P + 8}) == api.ATTN_ERR_ALIGN, name
    for n in (0, -1):
        assert append(lib, four, s, angles=n) == api.ATTN_ERR_SHAPE
    # in place with other strides
    wide = paged(four, o_token=512)
    assert append(lib, four, wide, out=P) == api.ATTN_ERR_SHAPE
    # nothing to do: no pointer is looked at
    none = dict(q=None, k=None, v=None, slots=None, cu=None, lens=None, out=None, kc=None, vc=None)
    assert append(lib, four, paged(four, tokens=0), **none) == api.ATTN_OK


def test_append4_without_rotation_reads_no_q(lib):
    s = paged(True, heads=-7, q_token=3, o_head=5)
    none = dict(q=None, cos=None, sin=None, cu=None, lens=None, out=None, angles=-1)
    for name in ("k", "v", "slots", "kc", "vc"):
        assert append(lib, True, s, **{**none, name: None}) == api.ATTN_ERR_NULL, name
    assert append(lib, True, paged(True, tokens=0, heads=-7), **none) == api.ATTN_OK
    # the 16-bit append always turns
    assert append(lib, False, paged(False), cos=None, sin=None) == api.ATTN_ERR_NULL


@pytest.mark.parametrize("kw", COMMON + POOL4 + [dict(k_token=-128), dict(k_head=68),
                                                 dict(v_token=64), dict(k_token=64)])
def test_load4_shape_refused(lib, kw):
    assert load(lib, paged(True, **kw)) == api.ATTN_ERR_SHAPE


def test_load4_pointers_refused(lib):
    assert load(lib, None) == api.ATTN_ERR_NULL
    s = paged(True)
    for name in ("slots", "kc", "vc", "k", "v"):
        assert load(lib, s, **{name: None}) == api.ATTN_ERR_NULL, name
        assert load(lib, s, **{name: P + 2}) == api.ATTN_ERR_ALIGN, name
    assert load(lib, paged(True, tokens=0), *[None] * 5) == api.ATTN_OK


@pytest.mark.parametrize("kw", COMMON + POOL4 + [dict(heads=5), dict(scale=0.0), dict(max_new=0),
                                                 dict(heads=258), dict(q_token=8),
                                                 dict(o_token=64)])
def test_fwd4_shape_refused(lib, kw):
    assert fwd4(lib, paged(True, **kw)) == api.ATTN_ERR_SHAPE


def test_fwd4_pointers_refused(lib):
    assert fwd4(lib, None) == api.ATTN_ERR_NULL
    s = paged(True)
    for name in ("q", "k", "v", "table", "cu", "lens", "ws", "o"):
        assert fwd4(lib, s, **{name: None}) == api.ATTN_ERR_NULL, name
        assert fwd4(lib, s, **{name: P + 2}) == api.ATTN_ERR_ALIGN, name
    assert fwd4(lib, s, lse=P + 4) == api.ATTN_ERR_ALIGN
    need = lib.attn_paged_workspace_bytes(ctypes.byref(s))
    assert fwd4(lib, s, n=need - 1) == api.ATTN_ERR_WORKSPACE
    assert fwd4(lib, paged(True, tokens=0), *[None] * 7, 0, None) == api.ATTN_OK


@pytest.mark.parametrize("kw,size", [(dict(), 2708480), (dict(max_new=1), 2708480),
                                     (dict(max_new=9), 2708480 + 32442880),
                                     (dict(heads=32, kv_heads=1), 32442880)])
def test_the_workspace_is_that_of_the_16_bit_call(lib, kw, size):
    """A workspace of the size that attn_paged_fwd had before the 4-bit cache came serves
    both calls: two parts of 16 rows (264 bytes and a description of 16 a block) for 320
    blocks, and of 384 rows for 160 where requests may be chunks."""
    assert 320 * (16 + 2 * 16 * 264) == 2708480 and 160 * (16 + 2 * 384 * 264) == 32442880
    for four in (False, True):
        s = paged(four, q_token=2048, o_token=2048, **kw)
        assert lib.attn_paged_workspace_bytes(ctypes.byref(s)) == size


def test_python_binding_refuses_host_tensors():
    s = api.PagedShape(1, 2, 2, 1, 16, 3, 1)
    q, k = torch.zeros((2, 2, 64), dtype=torch.float16), torch.zeros((2, 1, 64),
                                                                     dtype=torch.float16)
    pool = api.alloc_paged_pool4(s, "cpu")
    assert pool.shape == (3, 1, 2, 288)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)
    cos = torch.ones((4, 32))
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_paged_append4(s, q, k, k, cos, cos, i(0, 1), i(0, 2), i(2), q, pool, pool)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_paged_load4(s, i(0, 1), pool, pool, k, k)
    with pytest.raises(ValueError, match="CUDA"):
        api.attn_paged_fwd4(s, q, pool, pool, i(0)[None], i(0, 2), i(2),
                            torch.zeros(8, dtype=torch.uint8), q)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_host_form_of_the_quantiser(dtype):
    """Known values of the form that the GPU tests compare with."""
    x = torch.zeros((1, 1, 8, 64))
    x[0, 0, 0, :4] = torch.tensor([-8.0, 7.0, 3.4, 0.5])
    x[0, 0, 0, 32:36] = torch.tensor([16.0, -16.0, 3.0, 5.0])
    x[0, 0, 1, 0] = 4.0
    pool = serve4_util.pool_of(x.to(dtype), dtype)
    v, s = serve4_util.values(pool, dtype)
    assert v[0, 0, 0, :4].tolist() == [-8.0, 7.0, 3.0, 0.0] and s[0, 0, 0, 0] == 1
    # the extremum of a tie is the negative one; 3 / 2 = 1.5 goes to 2, 5 / 2 = 2.5 to 2
    assert v[0, 0, 0, 32:36].tolist() == [14.0, -16.0, 4.0, 4.0]
    assert v[0, 0, 1, 0] == 4.0 and s[0, 0, 1, 0] == 0.5
    assert (v[0, 0, 2:] == 0).all()
    # code * scale is exact in the type
    y = torch.randn((4, 2, 16, 64)) * 10
    v, _ = serve4_util.values(serve4_util.pool_of(y.to(dtype), dtype), dtype)
    assert torch.equal(v, v.to(dtype).double())
