"""Refusals of the packed and paged entry points: every one before any launch, on the CPU."""
import ctypes
import os
import re

import pytest
import torch

from block_sparse_attention_stats_b200 import _lib as L
from block_sparse_attention_stats_b200 import packed as K
from block_sparse_attention_stats_b200.build import build

OK, INVALID, UNSUPPORTED, WORKSPACE = (L.PISA_OK, L.PISA_ERR_INVALID_ARG, L.PISA_ERR_UNSUPPORTED,
                                       L.PISA_ERR_WORKSPACE)
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pisa.h")


@pytest.fixture(scope="module")
def lib():
    build()
    return L.load()


def R(ptr, h=6400, r=64):
    return L.PisaRows(ptr, h, r)


def G(ptr, p=2048, h=1024, r=64):
    return L.PisaPages(ptr, p, h, r)


A = [0x100000 * (i + 1) for i in range(40)]      # pointers that are only compared


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(L.PisaRows) == 24 and ctypes.sizeof(L.PisaPages) == 32
    text = open(HEADER).read()
    body = re.search(r"typedef struct \{([^}]*)\} pisa_page_step;", re.sub(r"/\*.*?\*/", "", text, flags=re.S)).group(1)
    names = [n for line in body.split(";") for n in re.findall(r"\*?(\w+)\s*(?:,|$)", line.strip())]
    assert names == [n for n, _ in L.PisaPageStep._fields_]


def varlen(lib, q=None, k=None, v=None, dtype=L.PISA_BF16, cu=A[5], B=2, T=100, Hq=4, Hkv=2, d=64, scale=0.0,
           flags=1, out=None, lse=None, o32=None, ws=A[6], ws_bytes=None):
    need = lib.pisa_varlen_attention_workspace_bytes(4, 2, 64)
    return lib.pisa_varlen_attention(q or R(A[0]), k or R(A[1]), v or R(A[2]), dtype, cu, B, T, Hq, Hkv, d, scale,
                                     flags, out or R(A[3]), lse, o32, ws, need if ws_bytes is None else ws_bytes, None)


COMMON = [
    (dict(dtype=7), INVALID), (dict(dtype=L.PISA_F32), UNSUPPORTED),
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(Hq=5), INVALID), (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(B=(1 << 16) + 1), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(cu=None), INVALID), (dict(cu=A[5] + 2), INVALID),
    (dict(q=R(None)), INVALID), (dict(q=R(A[0] + 8)), INVALID), (dict(q=R(A[0], r=60)), INVALID),
    (dict(q=R(A[0], r=68)), INVALID), (dict(q=R(A[0], h=0)), INVALID), (dict(q=R(A[0], h=-6400)), INVALID),
    (dict(q=R(A[0], r=0)), INVALID), (dict(out=R(A[3], h=64, r=64)), INVALID), (dict(out=R(A[0])), INVALID),
    (dict(ws=None), INVALID), (dict(ws=A[6] + 4), INVALID), (dict(ws_bytes=100), WORKSPACE),
    (dict(lse=A[7] + 1), INVALID), (dict(out=R(A[3], h=64, r=136)), INVALID),
]


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(k=R(A[1] + 2)), INVALID), (dict(v=R(A[2], r=32)), INVALID), (dict(o32=A[8] + 4), INVALID),
    (dict(o32=A[3]), INVALID), (dict(out=R(A[1])), INVALID), (dict(out=R(A[2])), INVALID), (dict(flags=4), INVALID)])
def test_varlen_refuses(lib, change, status):
    assert varlen(lib, **change) == status


def test_nothing_is_launched_for_no_tokens(lib):
    """T = 0 needs no pointer: an empty tensor has none."""
    none = R(None)
    assert varlen(lib, q=none, k=none, v=none, out=none, T=0, ws=None) == OK
    assert bwd(lib, q=none, T=0, ws=None) == OK
    assert paged(lib, q=none, out=none, T=0, ws=None) == OK
    assert write(lib, k=none, v=none, slots=None, T=0) == OK


def test_strides_of_an_extent_of_one_are_not_used(lib):
    """One head, or one token: whatever the stride says (here the call goes on to the workspace check)."""
    one = R(A[0], h=1, r=64)
    assert varlen(lib, q=one, k=R(A[1], h=0), v=R(A[2], h=3), out=R(A[3], h=-1), Hq=1, Hkv=1, ws_bytes=0) == WORKSPACE
    row = dict(q=R(A[0], r=1), k=R(A[1], r=0), v=R(A[2], r=7), out=R(A[3], r=3))
    assert varlen(lib, T=1, ws_bytes=0, **row) == WORKSPACE


def bwd(lib, q=None, dout=None, dtype=L.PISA_BF16, lse=A[7], o32=A[8], cu=A[5], B=2, T=100, Hq=4, Hkv=2, d=64,
        scale=0.0, flags=1, dq=None, dk=None, dv=None, ws=A[6], ws_bytes=None):
    need = lib.pisa_varlen_attention_bwd_workspace_bytes(100, 4, 2, 64)
    return lib.pisa_varlen_attention_bwd(
        q or R(A[0]), R(A[1]), R(A[2]), dout or R(A[3]), dtype, lse, o32, cu, B, T, Hq, Hkv, d, scale, flags,
        dq or R(A[9]), dk or R(A[10]), dv or R(A[11]), ws, need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=L.PISA_F16), UNSUPPORTED), (dict(dtype=L.PISA_F32), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(B=0), INVALID), (dict(Hq=5), INVALID), (dict(Hq=400), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
    (dict(scale=-0.5), INVALID), (dict(flags=8), INVALID), (dict(cu=None), INVALID), (dict(lse=None), INVALID),
    (dict(B=(1 << 16) + 1), UNSUPPORTED), (dict(T=1 << 24, Hq=128, Hkv=1), UNSUPPORTED),
    (dict(lse=A[7] + 2), INVALID), (dict(o32=None), INVALID), (dict(o32=A[8] + 4), INVALID),
    (dict(dout=R(A[3], r=8)), INVALID), (dict(dq=R(A[0])), INVALID), (dict(dk=R(A[9])), INVALID),
    (dict(dv=R(A[10])), INVALID), (dict(dq=R(A[8])), INVALID), (dict(dv=R(A[7])), INVALID),
    (dict(dk=R(A[10], h=64)), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=4096), WORKSPACE)])
def test_backward_refuses(lib, change, status):
    assert bwd(lib, **change) == status


def paged(lib, q=None, k=None, v=None, dtype=L.PISA_BF16, pages=10, ps=16, table=A[12], width=4, cu=A[5], kv=A[13],
          B=2, T=100, Hq=4, Hkv=2, d=64, scale=0.0, out=None, lse=None, ws=A[6], ws_bytes=None):
    need = lib.pisa_paged_attention_workspace_bytes(4, 2, 64)
    return lib.pisa_paged_attention(q or R(A[0]), k or G(A[1]), v or G(A[2]), dtype, pages, ps, table, width, cu, kv,
                                    B, T, Hq, Hkv, d, scale, out or R(A[3]), lse, ws,
                                    need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(pages=0), INVALID), (dict(ps=0), INVALID), (dict(ps=8), UNSUPPORTED), (dict(ps=48), UNSUPPORTED),
    (dict(ps=512), UNSUPPORTED), (dict(width=0), INVALID), (dict(table=None), INVALID), (dict(kv=None), INVALID),
    (dict(k=G(A[1] + 2)), INVALID), (dict(k=G(None)), INVALID), (dict(v=G(A[2], p=0)), INVALID),
    (dict(v=G(A[2], r=65)), INVALID), (dict(v=G(A[2], h=32)), INVALID), (dict(out=R(A[1])), INVALID),
    (dict(out=R(A[2])), INVALID)])
def test_paged_refuses(lib, change, status):
    assert paged(lib, **change) == status


def step(**change):
    s = dict(past_lens=A[20], new_lens=A[21], B=2, T=10, block_table=A[22], width=4, page_size=16, free_pages=A[23],
             free_cap=5, num_free=A[24], slots=A[25], cu_seqlens=A[26], kv_lens=A[27], num_free_out=A[28])
    s.update(change)
    return L.PisaPageStep(*[s[n] for n, _ in L.PisaPageStep._fields_])


STEP = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(width=0), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(B=16385), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED),
    (dict(width=1 << 27), UNSUPPORTED), (dict(free_cap=-1), INVALID), (dict(past_lens=None), INVALID),
    (dict(new_lens=A[21] + 1), INVALID), (dict(block_table=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(num_free=None), INVALID), (dict(slots=None), INVALID), (dict(slots=A[25] + 4), INVALID),
    (dict(cu_seqlens=None), INVALID), (dict(kv_lens=None), INVALID), (dict(num_free_out=None), INVALID),
    (dict(kv_lens=A[20]), INVALID), (dict(num_free_out=A[24]), INVALID), (dict(kv_lens=A[26]), INVALID),
    (dict(slots=A[22]), INVALID), (dict(block_table=A[23]), INVALID),
]


@pytest.mark.parametrize("change,status", STEP)
def test_plan_refuses(lib, change, status):
    assert lib.pisa_page_plan(ctypes.byref(step(**change)), None) == status


def test_plan_refuses_no_struct(lib):
    assert lib.pisa_page_plan(None, None) == INVALID


def write(lib, k=None, v=None, dtype=L.PISA_BF16, slots=A[25], T=10, Hkv=2, d=64, kc=None, vc=None, pages=10, ps=16):
    return lib.pisa_page_write(k or R(A[1]), v or R(A[2]), dtype, slots, T, Hkv, d, kc or G(A[3]), vc or G(A[4]),
                               pages, ps, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=L.PISA_F32), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(T=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(d=80), UNSUPPORTED), (dict(pages=0), INVALID), (dict(ps=20), UNSUPPORTED), (dict(slots=None), INVALID),
    (dict(slots=A[25] + 4), INVALID), (dict(k=R(A[1] + 2)), INVALID), (dict(v=R(A[2], r=0)), INVALID),
    (dict(kc=G(A[3], r=63)), INVALID), (dict(vc=G(A[3])), INVALID), (dict(kc=G(A[1])), INVALID),
    (dict(vc=G(A[1])), INVALID)])
def test_write_refuses(lib, change, status):
    assert write(lib, **change) == status


def whole(lib, s=None, q=None, k=None, kc=None, vc=None, dtype=L.PISA_BF16, pages=10, Hq=4, Hkv=2, d=64, scale=0.0,
          out=None, lse=None, ws=A[6], ws_bytes=1 << 30):
    return lib.pisa_paged_step(ctypes.byref(step(**(s or {}))), q or R(A[0]), k or R(A[1]), R(A[2]), kc or G(A[3]),
                               vc or G(A[4]), dtype, pages, Hq, Hkv, d, scale, out or R(A[9]), lse, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [(dict(s=c), st) for c, st in STEP] + [
    (dict(dtype=L.PISA_F32), UNSUPPORTED), (dict(pages=0), INVALID), (dict(Hq=3), INVALID), (dict(d=16), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(q=R(A[0], r=4)), INVALID), (dict(k=R(None)), INVALID),
    (dict(kc=G(A[3], p=8)), INVALID), (dict(vc=G(A[3])), INVALID), (dict(out=R(A[3])), INVALID),
    (dict(out=R(A[0])), INVALID), (dict(lse=A[7] + 1), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=0), WORKSPACE)])
def test_whole_step_refuses_before_the_plan(lib, change, status):
    assert whole(lib, **change) == status


def test_f16_stays_out_of_the_sparse_path(lib):
    assert lib.pisa_dense_attention(A[0], A[1], A[2], A[3], L.PISA_F16, 1, 1, 128, 64, 0.0, A[6], 1 << 30,
                                    None) == INVALID


def test_workspace_sizes(lib):
    w = lib.pisa_varlen_attention_workspace_bytes
    assert w(8, 2, 128) > w(8, 2, 64) > 0 and w(8, 2, 96) == 0 and w(7, 2, 64) == 0 and w(0, 0, 64) == 0
    b = lib.pisa_varlen_attention_bwd_workspace_bytes
    assert b(1000, 8, 2, 128) > b(10, 8, 2, 128) > 0 and b(0, 8, 2, 128) == 0 and b(10, 8, 3, 128) == 0
    assert lib.pisa_paged_attention_workspace_bytes(256, 1, 64) == 0


# ---- the binding's own checks: on CPU tensors, before a pointer is taken -------------------------

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_checks():
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for q, k, v in ((t(4, 4, 64), t(3, 4, 64), t(3, 4, 64)), (t(4, 4, 64), t(2, 5, 64), t(2, 5, 64)),
                    (t(4, 4, 64), t(2, 4, 64), t(1, 4, 64)), (t(4, 4), t(2, 4), t(2, 4)),
                    (t(4, 4, 64, dtype=torch.float32),) + (t(2, 4, 64, dtype=torch.float32),) * 2):
        with pytest.raises(ValueError):
            K.pisa_varlen_attention(q, k, v, cu)
    q, k = t(4, 4, 64), t(2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        K.pisa_varlen_attention(q, k, k, cu)
    with pytest.raises(ValueError):
        K.pisa_varlen_attention_bwd(q, k, k, k, None, None, cu)
    with pytest.raises(ValueError, match="lse and out_f32"):
        K.pisa_varlen_attention_bwd(q, k, k, q, None, None, cu)
    with pytest.raises(ValueError, match="bf16"):
        h = [x.half().requires_grad_() for x in (q, k, k)]
        K.varlen_attention(*h, cu)
    c = t(3, 2, 16, 64)
    for bad in (t(3, 2, 16), t(3, 2, 8, 64)):
        with pytest.raises(ValueError):
            K.pisa_paged_attention(q, c, bad, t(1, 4, dtype=torch.int32), cu, cu[:1])
    with pytest.raises(ValueError):
        K.pisa_paged_attention(t(4, 4, 128), c, c, t(1, 4, dtype=torch.int32), cu, cu[:1])
    with pytest.raises(ValueError):
        K.pisa_page_write(t(1, 4, 64), t(1, 4, 64), t(4, dtype=torch.int64), c, c)


def test_layouts_that_are_taken_in_place():
    x = t(5, 3, 64)
    assert K._strides_ok(x) and K._strides_ok(x.transpose(0, 1)) and K._strides_ok(t(5, 9, 64)[:, 2:4])
    assert not K._strides_ok(x[:1, :, :32].expand(3, -1, -1)) and not K._strides_ok(x.transpose(1, 2))
    assert not K._strides_ok(t(5, 3, 68)[..., :64]) and K._strides_ok(t(5, 3, 72)[..., :64])
    assert K._laid_out(x) is x
    y = K._laid_out(x[:1].expand(3, -1, -1))
    assert y.is_contiguous()
