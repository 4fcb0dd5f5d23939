"""Refusals of the paged-cache entry points, on the CPU: status codes of the C
functions for arguments they must not accept (fake pointers, never followed:
every call fails validation or stops at the device query), and the binding's
own checks of types, shapes and devices."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def va():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer ABI checks run only where no GPU is visible")
    from packed_variable_length_varlen_gb300 import build
    build.build()
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


def _cache(va, **kw):
    c = va.VarlenKvCache()
    kind = kw.pop("type", 0)
    page, heads, dim = kw.get("page_size", 16), kw.get("num_kv_heads", 2), kw.get("head_dim", 64)
    c.k, c.v, c.block_table, c.seqlens = 0x10000, 0x20000, 0x30000, 0x40000
    if kind == 1:
        c.k_scale, c.v_scale = 0x50000, 0x60000
    c.sk = va.VarlenPageStride(page * heads * dim, heads * dim, dim)
    c.sv = va.VarlenPageStride(page * heads * dim, heads * dim, dim)
    c.table_stride, c.type, c.num_pages, c.page_size, c.max_pages = 8, kind, 10, page, 8
    c.num_kv_heads, c.head_dim = heads, dim
    for n, x in kw.items():
        setattr(c, n, x)
    return c


def _calls(va, c, total=10, batch=1, cu=0x2000, k=0x1000, stride=None):
    st = va.VarlenStride(*(stride or (c.num_kv_heads * c.head_dim, c.head_dim)))
    r = ctypes.byref(c)
    yield va.LIB.varlen_attn_cache_write(k, st, k, st, cu, batch, total, r, None)
    yield va.LIB.varlen_attn_cache_read(r, cu, batch, total, k, st, k, st, None)
    yield va.LIB.varlen_attn_fwd_paged(k, st, cu, batch, total, c.num_kv_heads, 0, r, 0.125, -1, -1, k, st, 0x3000,
                                       0x100000, 1 << 40, None)


@pytest.mark.parametrize("kind", [0, 1])
def test_valid_arguments_reach_the_device_query(va, kind):
    for dim in (64, 96, 128):
        for page in (16, 32, 64, 128, 256, 512, 1024):
            for st in _calls(va, _cache(va, type=kind, head_dim=dim, page_size=page)):
                assert st in (va.VARLEN_ERR_CUDA, va.VARLEN_ERR_ARCH), st


@pytest.mark.parametrize("change,code", [
    ({"num_pages": 0}, "SHAPE"), ({"num_pages": -1}, "SHAPE"), ({"max_pages": -1}, "SHAPE"),
    ({"table_stride": -1}, "SHAPE"), ({"num_kv_heads": 0}, "SHAPE"), ({"type": 2}, "SHAPE"), ({"type": -1}, "SHAPE"),
    ({"page_size": 0}, "SHAPE"), ({"page_size": 8}, "SHAPE"), ({"page_size": 48}, "SHAPE"),
    ({"page_size": 2048}, "SHAPE"), ({"page_size": -16}, "SHAPE"), ({"max_pages": 1 << 27}, "SHAPE"),
    ({"head_dim": 80}, "HEAD_DIM"), ({"head_dim": 256}, "HEAD_DIM"),
    ({"k": None}, "NULL"), ({"v": None}, "NULL"), ({"seqlens": None}, "NULL"), ({"block_table": None}, "NULL"),
    ({"k": 0x10008}, "ALIGN"), ({"v": 0x20008}, "ALIGN"),
])
def test_cache_refusals(va, change, code):
    c = _cache(va)
    for n, x in change.items():
        setattr(c, n, x)
    for st in _calls(va, c):
        assert st == getattr(va, "VARLEN_ERR_" + code), (change, st)


def test_scale_refusals(va):
    for change, code in (({"k_scale": None}, va.VARLEN_ERR_NULL), ({"v_scale": None}, va.VARLEN_ERR_NULL),
                         ({"k_scale": 0x50008}, va.VARLEN_ERR_ALIGN)):
        c = _cache(va, type=1)
        for n, x in change.items():
            setattr(c, n, x)
        assert set(_calls(va, c)) == {code}


@pytest.mark.parametrize("stride", [(2048, 128, 60), (2048, 100, 64), (-2048, 128, 64), (1 << 39, 128, 64),
                                    (2000, 128, 64), (2048, 64, 64), (2048, 128, 32), (1024, 128, 64), (0, 128, 64),
                                    (2048, 0, 64), (2048, 128, 0)])
def test_page_stride_refusals(va, stride):
    for which in ("sk", "sv"):
        c = _cache(va)
        setattr(c, which, va.VarlenPageStride(*stride))
        for st in _calls(va, c):
            assert st == va.VARLEN_ERR_STRIDE, (stride, st)


def test_head_major_and_single_extents_are_accepted(va):
    c = _cache(va)
    c.sk = va.VarlenPageStride(2048, 64, 1024)  # [page, head, row, dim]
    for st in _calls(va, c):
        assert st in (va.VARLEN_ERR_CUDA, va.VARLEN_ERR_ARCH)
    c = _cache(va, num_pages=1, num_kv_heads=1)
    c.sk = c.sv = va.VarlenPageStride(0, 64, 0)  # strides over one element do not matter
    for st in _calls(va, c):
        assert st in (va.VARLEN_ERR_CUDA, va.VARLEN_ERR_ARCH)


def test_call_refusals(va):
    c = _cache(va)
    assert set(_calls(va, c, batch=0)) == {va.VARLEN_ERR_SHAPE}
    assert set(_calls(va, c, batch=(1 << 30) + 1)) == {va.VARLEN_ERR_SHAPE}
    assert set(_calls(va, c, total=-1)) == {va.VARLEN_ERR_SHAPE}
    assert set(_calls(va, c, cu=None)) == {va.VARLEN_ERR_NULL}
    assert set(_calls(va, c, k=None)) == {va.VARLEN_ERR_NULL}
    assert set(_calls(va, c, k=0x1008)) == {va.VARLEN_ERR_ALIGN}
    assert set(_calls(va, c, stride=(130, 64))) == {va.VARLEN_ERR_STRIDE}
    st = va.VarlenStride(128, 64)
    assert va.LIB.varlen_attn_cache_write(0x1000, st, 0x1000, st, 0x2000, 1, 10, None, None) == va.VARLEN_ERR_NULL
    # an output that overlaps itself
    assert va.LIB.varlen_attn_cache_read(ctypes.byref(c), 0x2000, 1, 10, 0x1000, va.VarlenStride(64, 64), 0x1000, st,
                                         None) == va.VARLEN_ERR_STRIDE


def test_attention_refusals(va):
    c = _cache(va)
    r = ctypes.byref(c)

    def call(heads=4, scale=0.125, sq=(256, 64), so=(256, 64), lse=0x3000, ws=0x100000, nb=1 << 40, total=10):
        return va.LIB.varlen_attn_fwd_paged(0x1000, va.VarlenStride(*sq), 0x2000, 1, total, heads, 0, r, scale, -1, -1,
                                            0x1000, va.VarlenStride(*so), lse, ws, nb, None)

    assert call() in (va.VARLEN_ERR_CUDA, va.VARLEN_ERR_ARCH)
    for heads in (0, -2, 3, 258):
        assert call(heads=heads, sq=(20000, 64), so=(20000, 64)) == va.VARLEN_ERR_SHAPE
    assert call(total=2 ** 29) == va.VARLEN_ERR_SHAPE  # 2^31 rows of four heads
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == va.VARLEN_ERR_SHAPE
    assert call(lse=None) == va.VARLEN_ERR_NULL
    assert call(sq=(0, 64)) == va.VARLEN_ERR_STRIDE
    assert call(sq=(256, 0)) == va.VARLEN_ERR_STRIDE
    assert call(so=(256, 0)) == va.VARLEN_ERR_STRIDE
    need = va.varlen_attn_fwd_paged_workspace_size(1, 10, 4, 2, 64)
    assert need > 0
    for ws, nb in ((None, need), (0x100010, need), (0x100000, need - 1)):
        assert call(ws=ws, nb=nb) == va.VARLEN_ERR_WORKSPACE
    assert call(nb=need) in (va.VARLEN_ERR_CUDA, va.VARLEN_ERR_ARCH)
    assert va.varlen_attn_fwd_paged_workspace_size(-1, 10, 4, 2, 64) == 0
    assert va.varlen_attn_fwd_paged_workspace_size(1, 10, 4, 0, 64) == 0


# ------------------------------------------------------------------ the binding

def _tensors(kind="bf16", pages=6, page=16, heads=2, dim=64, batch=3):
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    t = {"k_pages": torch.zeros(pages, page, heads, dim, dtype=dt), "v_pages": torch.zeros(pages, page, heads, dim, dtype=dt),
         "block_table": torch.zeros(batch, 2, dtype=torch.int32), "seqlens": torch.zeros(batch, dtype=torch.int32)}
    if kind == "e4m3":
        t["k_scale"] = torch.ones(pages, heads, page, dtype=torch.bfloat16)
        t["v_scale"] = torch.ones(pages, heads, page, dtype=torch.bfloat16)
    return t


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_binding_describes_the_tensors(va, kind):
    t = _tensors(kind)
    c = va.PagedCache(**t).struct
    assert (c.k, c.v) == (t["k_pages"].data_ptr(), t["v_pages"].data_ptr())
    assert (c.num_pages, c.page_size, c.num_kv_heads, c.head_dim, c.max_pages) == (6, 16, 2, 64, 2)
    assert (c.sk.page, c.sk.row, c.sk.head) == (2048, 128, 64)
    assert c.type == (va.VARLEN_CACHE_BF16 if kind == "bf16" else va.VARLEN_CACHE_E4M3)
    assert (c.k_scale is None) == (kind == "bf16")


@pytest.mark.parametrize("kind,change", [
    ("bf16", {"k_pages": torch.zeros(6, 16, 2, 64)}),
    ("bf16", {"v_pages": torch.zeros(6, 16, 2, 32, dtype=torch.bfloat16)}),
    ("bf16", {"k_pages": torch.zeros(6, 16, 64, 2, dtype=torch.bfloat16).transpose(2, 3)}),
    ("bf16", {"block_table": torch.zeros(3, 2, dtype=torch.int64)}),
    ("bf16", {"block_table": torch.zeros(2, 3, dtype=torch.int32).T}),
    ("bf16", {"seqlens": torch.zeros(2, dtype=torch.int32)}),
    ("bf16", {"seqlens": torch.zeros(3, dtype=torch.int64)}),
    ("bf16", {"k_scale": torch.ones(6, 2, 16, dtype=torch.bfloat16)}),
    ("e4m3", {"k_scale": None}),
    ("e4m3", {"v_scale": torch.ones(6, 16, 2, dtype=torch.bfloat16)}),
    ("e4m3", {"v_scale": torch.ones(6, 2, 16)}),
])
def test_the_binding_refuses_tensors(va, kind, change):
    with pytest.raises(ValueError):
        va.PagedCache(**{**_tensors(kind), **change})


def test_the_binding_refuses_calls(va):
    c = va.PagedCache(**_tensors())
    cu = torch.tensor([0, 1, 2, 4], dtype=torch.int32)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for bad in ((k.float(), k, cu), (k, k[:3], cu), (k[:, :1], k[:, :1], cu), (k[..., :32], k, cu), (k, k, cu.long()),
                (k, k, cu[:3]), (k, k.transpose(1, 2), cu)):
        with pytest.raises(ValueError):
            va.cache_write(c, *bad)
    with pytest.raises(ValueError, match="CUDA"):
        va.cache_write(c, k, k, cu)
    with pytest.raises(ValueError, match="CUDA"):
        va.cache_read(c, cu, 4)
    with pytest.raises(ValueError):
        va.cache_read(c, cu, 5, k, k)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        va.attention_fwd_paged(q, c, cu)
    for kw in ({"out": q[:3]}, {"out": q.float()}, {"lse": torch.zeros(4, 3)}, {"lse": torch.zeros(4, 4).double()}):
        with pytest.raises(ValueError):
            va.attention_fwd_paged(q, c, cu, **kw)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_handle_refuses_other_tensors(va, kind):
    """Calls use what the handle was made with: another tensor in its place would be without effect and is refused;
    writing into the ones it has (`+=` among the ways) is not."""
    t = _tensors(kind)
    c = va.PagedCache(**t)
    for name in ("k_pages", "v_pages", "block_table", "seqlens", "k_scale", "v_scale"):
        old = getattr(c, name)
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, torch.zeros(1) if old is None else old.clone())
        assert getattr(c, name) is old
    for name in ("batch", "num_kv_heads", "head_dim", "device", "struct"):
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, 1)
    c.seqlens += 3
    c.block_table[0, 1] = 5
    assert t["seqlens"].tolist() == [3, 3, 3] and int(t["block_table"][0, 1]) == 5
    assert c.struct.seqlens == t["seqlens"].data_ptr()


def test_the_binding_refuses_a_workspace_with_gaps(va):
    """The kernels use the workspace's bytes one after another: an expanded or strided tensor does not have as many as
    its element count says."""
    c = va.PagedCache(**_tensors())
    cu = torch.tensor([0, 1, 2, 4], dtype=torch.int32)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    need = va.varlen_attn_fwd_paged_workspace_size(3, 4, 4, 2, 64)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            va.attention_fwd_paged(q, c, cu, workspace=ws)
