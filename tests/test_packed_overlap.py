"""Operands that share memory are refused, layouts that lie between one another are not (CPU: a call that
is not refused here goes on to the check of the workspace's size)."""
import ctypes

import pytest

from block_sparse_attention_stats_b200 import _lib as L
from block_sparse_attention_stats_b200.build import build

INVALID, WORKSPACE = L.PISA_ERR_INVALID_ARG, L.PISA_ERR_WORKSPACE
MB = 1 << 20
A = [(i + 1) * 64 * MB for i in range(40)]     # only compared
T, HQ, HKV, D, B = 100, 4, 2, 64, 2
ROW = 2 * D                                    # bytes


@pytest.fixture(scope="module")
def lib():
    build()
    return L.load()


def heads(ptr, h=T * D, r=D):                  # [H, T, d]
    return L.PisaRows(ptr, h, r)


def tokens(ptr, n, r=None):                    # [T, H, d] of a row of n heads
    return L.PisaRows(ptr, D, n * D if r is None else r)


def pages(ptr, p=HKV * 16 * D, h=16 * D, r=D):
    return L.PisaPages(ptr, p, h, r)


def varlen(lib, q=heads(A[0]), k=heads(A[1]), v=heads(A[2]), cu=A[3], out=heads(A[4]), lse=A[5], o32=A[6], ws=A[7],
           ws_bytes=0):
    return lib.pisa_varlen_attention(q, k, v, L.PISA_BF16, cu, B, T, HQ, HKV, D, 0.0, 1, out, lse, o32, ws, ws_bytes,
                                     None)


ALL = 1 << 34
FUSED = A[20]                                  # [T, HQ + 2 HKV, d]
N = HQ + 2 * HKV


@pytest.mark.parametrize("change", [
    dict(out=heads(A[0] + ROW)), dict(out=heads(A[0] - ROW)), dict(out=heads(A[1] + T * ROW)),
    dict(out=heads(A[2] - 3 * T * ROW)), dict(out=tokens(A[0] + ROW, HQ)), dict(out=heads(A[0] + (HQ * T - 1) * ROW)),
    dict(out=heads(A[3] - 16)), dict(lse=A[0] + 64), dict(lse=A[4] + 4), dict(lse=A[3] - 4), dict(o32=A[4] + 32),
    dict(o32=A[1] - 16), dict(o32=A[5] - 16), dict(lse=A[5], o32=A[5] + 16),
    # slices of one tensor: out over a head of k, out a row on
    dict(q=tokens(FUSED, N), k=tokens(FUSED + HQ * ROW, N), v=tokens(FUSED + (HQ + HKV) * ROW, N),
         out=tokens(FUSED + ROW, N)),
    dict(q=tokens(FUSED, 2 * HQ), out=tokens(FUSED + (HQ - 1) * ROW, 2 * HQ)),
    dict(q=tokens(FUSED, 2 * HQ), out=tokens(FUSED + (3 * HQ) * ROW - ROW, 2 * HQ)),
    dict(q=heads(FUSED, 2 * T * D), out=heads(FUSED + T * ROW - ROW, 2 * T * D)),
    # a dense tensor against rows that are far apart
    dict(q=heads(FUSED, r=8 * D, h=8 * T * D), out=heads(FUSED + 8 * ROW)),
    dict(ws=A[4] - 1024, ws_bytes=ALL), dict(ws=A[1] + 128, ws_bytes=ALL), dict(ws=A[5] + 16, ws_bytes=ALL),
    dict(ws=A[3] - 1024, ws_bytes=ALL)])
def test_packed_operands_that_meet(lib, change):
    assert varlen(lib, **change) == INVALID


@pytest.mark.parametrize("change", [
    {}, dict(lse=None, o32=None),
    # one allocation, end to end
    dict(q=heads(A[0]), out=heads(A[0] + HQ * T * ROW), lse=A[0] + 2 * HQ * T * ROW),
    # slices of one tensor by heads, by tokens, out among them
    dict(q=tokens(FUSED, N), k=tokens(FUSED + HQ * ROW, N), v=tokens(FUSED + (HQ + HKV) * ROW, N)),
    dict(q=tokens(FUSED, 2 * HQ), out=tokens(FUSED + HQ * ROW, 2 * HQ)),
    dict(q=tokens(FUSED + HQ * ROW, 2 * HQ), out=tokens(FUSED, 2 * HQ)),
    dict(q=heads(FUSED, 2 * T * D), out=heads(FUSED + T * ROW, 2 * T * D)),
    dict(q=heads(FUSED, 2 * T * D), out=heads(FUSED - T * ROW, 2 * T * D)),
    # dense rows in the gaps of others
    dict(q=heads(FUSED, h=64 * T * D), lse=FUSED + T * ROW, out=heads(FUSED + (T * ROW * 64 * 4))),
    # inputs may share memory with one another
    dict(k=heads(A[0]), v=heads(A[0] + ROW))])
def test_packed_operands_that_do_not(lib, change):
    assert varlen(lib, **change) == WORKSPACE


def bwd(lib, q=heads(A[0]), dout=heads(A[3]), lse=A[4], o32=A[5], cu=A[6], dq=heads(A[7]), dk=heads(A[8]),
        dv=heads(A[9]), ws=A[10], ws_bytes=0):
    return lib.pisa_varlen_attention_bwd(q, heads(A[1]), heads(A[2]), dout, L.PISA_BF16, lse, o32, cu, B, T, HQ, HKV,
                                         D, 0.0, 1, dq, dk, dv, ws, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(dq=heads(A[0] + ROW)), dict(dk=heads(A[1] - ROW)), dict(dv=heads(A[2] + ROW)), dict(dq=heads(A[3] + ROW)),
    dict(dk=heads(A[4] + 16)), dict(dv=heads(A[5] - 16)), dict(dq=heads(A[6] - 16)), dict(dk=heads(A[7] + ROW)),
    dict(dv=heads(A[8] + T * ROW)), dict(dk=tokens(FUSED, N), dv=tokens(FUSED + ROW, N)),
    dict(ws=A[7] + 256, ws_bytes=ALL), dict(ws=A[3] - 1024, ws_bytes=ALL)])
def test_gradients_that_meet(lib, change):
    assert bwd(lib, **change) == INVALID


def test_gradients_that_do_not(lib):
    assert bwd(lib) == WORKSPACE
    assert bwd(lib, dq=tokens(FUSED, N), dk=tokens(FUSED + HQ * ROW, N),
               dv=tokens(FUSED + (HQ + HKV) * ROW, N)) == WORKSPACE
    assert bwd(lib, dq=heads(A[7]), dk=heads(A[7] + HQ * T * ROW), dv=heads(A[7] + (HQ + HKV) * T * ROW)) == WORKSPACE


P, PS, W = 10, 16, 4


def paged(lib, q=heads(A[0]), kc=pages(A[1]), vc=pages(A[2]), table=A[3], cu=A[4], kv=A[5], out=heads(A[6]), lse=A[7],
          ws=A[8], ws_bytes=0):
    return lib.pisa_paged_attention(q, kc, vc, L.PISA_BF16, P, PS, table, W, cu, kv, B, T, HQ, HKV, D, 0.0, out, lse,
                                    ws, ws_bytes, None)


PAGE = HKV * PS * ROW


@pytest.mark.parametrize("change", [
    dict(out=heads(A[0] + ROW)), dict(out=heads(A[1] + P * PAGE - ROW)), dict(out=heads(A[2] - ROW)),
    dict(out=heads(A[3] - 16)), dict(out=heads(A[4] - 16)), dict(out=heads(A[5] - 16)), dict(lse=A[6] + 4),
    dict(lse=A[1] + 4), dict(lse=A[3] + 4 * B * W - 4), dict(ws=A[1] - 1024, ws_bytes=ALL),
    dict(ws=A[3] - 1024, ws_bytes=ALL)])
def test_paged_operands_that_meet(lib, change):
    assert paged(lib, **change) == INVALID


def test_paged_operands_that_do_not(lib):
    assert paged(lib) == WORKSPACE
    # two layers' caches, keys and values in one tensor, and keys that are the values
    assert paged(lib, kc=pages(FUSED, p=4 * HKV * PS * D), vc=pages(FUSED + PAGE, p=4 * HKV * PS * D)) == WORKSPACE
    assert paged(lib, kc=pages(FUSED), vc=pages(FUSED)) == WORKSPACE


@pytest.mark.parametrize("kc,vc,k,slots", [
    (A[3], A[3] + PAGE, A[0], A[5]), (A[3], A[4], A[3] + P * PAGE - ROW, A[5]), (A[3], A[4], A[4] - ROW, A[5]),
    (A[3], A[4], A[0], A[3] + 8), (A[3], A[4], A[0], A[4] + P * PAGE - 8)])
def test_writes_that_meet(lib, kc, vc, k, slots):
    assert lib.pisa_page_write(heads(k), heads(A[1]), L.PISA_BF16, slots, T, HKV, D, pages(kc), pages(vc), P, PS,
                               None) == INVALID


def step(**change):
    s = dict(past_lens=A[20], new_lens=A[21], B=B, T=T, block_table=A[22], width=W, page_size=PS, free_pages=A[23],
             free_cap=5, num_free=A[24], slots=A[25], cu_seqlens=A[26], kv_lens=A[27], num_free_out=A[28])
    s.update(change)
    return L.PisaPageStep(*[s[n] for n, _ in L.PisaPageStep._fields_])


MEET = [dict(kv_lens=A[20] + 4), dict(cu_seqlens=A[21] - 8), dict(num_free_out=A[23] + 16), dict(slots=A[23] - 8),
        dict(block_table=A[24] - 4 * B * W + 4), dict(kv_lens=A[26] + 4 * B), dict(cu_seqlens=A[25] + 8 * T - 4),
        dict(num_free_out=A[22] + 4), dict(kv_lens=A[25] + 8), dict(num_free_out=A[21] + 4)]


@pytest.mark.parametrize("change", MEET)
def test_plans_that_meet(lib, change):
    assert lib.pisa_page_plan(ctypes.byref(step(**change)), None) == INVALID


def whole(lib, s=None, q=heads(A[0]), k=heads(A[1]), v=heads(A[2]), kc=pages(A[3]), vc=pages(A[4]), out=heads(A[5]),
          lse=A[6], ws=A[7], ws_bytes=0):
    return lib.pisa_paged_step(ctypes.byref(step(**(s or {}))), q, k, v, kc, vc, L.PISA_BF16, P, HQ, HKV, D, 0.0, out,
                               lse, ws, ws_bytes, None)


@pytest.mark.parametrize("change", [dict(s=c) for c in MEET] + [
    dict(out=heads(A[0] + ROW)), dict(out=heads(A[22] - 16)), dict(out=heads(A[3] + ROW)), dict(kc=pages(A[4] + PAGE)),
    dict(kc=pages(A[1] + ROW)), dict(vc=pages(A[20] - 16)), dict(lse=A[26] + 4), dict(lse=A[5] + 4),
    dict(lse=A[24]), dict(ws=A[25] - 1024, ws_bytes=ALL), dict(ws=A[3] - 1024, ws_bytes=ALL)])
def test_steps_that_meet(lib, change):
    assert whole(lib, **change) == INVALID


def test_steps_that_do_not(lib):
    assert whole(lib) == WORKSPACE
    # the plan's small results in one allocation
    assert whole(lib, s=dict(cu_seqlens=A[26], kv_lens=A[26] + 4 * (B + 1), num_free_out=A[26] + 4 * (2 * B + 1))) \
        == WORKSPACE
    # q, k, v of one projection; keys and values in one cache tensor
    assert whole(lib, q=tokens(FUSED - 512 * MB, N), k=tokens(FUSED - 512 * MB + HQ * ROW, N),
                 v=tokens(FUSED - 512 * MB + (HQ + HKV) * ROW, N), kc=pages(A[3], p=2 * HKV * PS * D),
                 vc=pages(A[3] + PAGE, p=2 * HKV * PS * D)) == WORKSPACE


# caches whose heads, pages or rows reach into one another: [pages, heads, page size] strides
SELF = [dict(p=PS * D, h=PS * D), dict(h=PS * D - 8), dict(p=HKV * PS * D - 8), dict(p=D, h=P * D, r=2 * D),
        dict(r=2 * D), dict(p=2 * HKV * PS * D, h=2 * HKV * PS * D, r=D)]
APART = [dict(), dict(p=HKV * PS * D, h=D, r=HKV * D), dict(p=4 * HKV * PS * D), dict(p=D, h=P * D, r=P * HKV * D),
         dict(p=2 * HKV * PS * D, h=2 * PS * D, r=2 * D), dict(p=PS * D, h=P * PS * D)]


@pytest.mark.parametrize("strides", SELF)
def test_a_cache_that_meets_itself_is_not_written(lib, strides):
    for kc, vc in ((pages(A[3], **strides), pages(A[4])), (pages(A[3]), pages(A[4], **strides))):
        assert lib.pisa_page_write(heads(A[0]), heads(A[1]), L.PISA_BF16, A[5], T, HKV, D, kc, vc, P, PS,
                                   None) == INVALID
        assert whole(lib, kc=kc, vc=vc) == INVALID
    # reading it does no harm
    assert paged(lib, kc=pages(A[1], **strides)) == WORKSPACE


@pytest.mark.parametrize("strides", APART)
def test_a_cache_that_does_not_is(lib, strides):
    assert whole(lib, kc=pages(A[3], **strides), vc=pages(A[4], **strides)) == WORKSPACE
