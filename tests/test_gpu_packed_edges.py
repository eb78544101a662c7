"""Edges of packed and paged attention: scores and weights of any size, rows of no sequence,
non-finite queries, padded batches, callers with a context of their own, and the backward's
whole contract.  Bounds as in packed_util."""
import math

import pytest
import torch

import packed_util as U

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def P():
    from block_sparse_attention_stats_b200.build import build
    build()
    import block_sparse_attention_stats_b200 as P
    return P


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def pages_of(x, ps):
    """[H, n, d] rows as a cache [pages, H, ps, d], page i holding positions i ps .. (i + 1) ps - 1."""
    h, n, d = x.shape
    need = -(-n // ps)
    c = torch.full((h, need * ps, d), math.nan, dtype=x.dtype)
    c[:, :n] = x
    return c.view(h, need, ps, d).transpose(0, 1).contiguous()


# ---- scores of any size --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [HF, BF])
def test_scores_past_every_range(P, dtype):
    """Scores so large that their float32 spacing is whole powers of two: weights stay finite."""
    d, n = 64, 600
    q, k = torch.full((1, n, d), 6000.0).to(dtype), torch.full((1, n, d), 9000.0).to(dtype)
    k[0, ::7] = 8000.0
    v = rows(3, 1, n, d, dtype=dtype)
    for scale in (1e-3, 1.0):
        a = P.pisa_varlen_attention(q.cuda(), k.cuda(), v.cuda(), i32([0, n]), scale=scale)
        kc, vc = (pages_of(x, 16).cuda() for x in (k, v))
        b = P.pisa_paged_attention(q[:, :1].cuda(), kc, vc, i32([list(range(kc.shape[0]))]), i32([0, 1]), i32([n]),
                                   scale=scale)
        P.pisa_device_status()
        assert torch.isfinite(a.float()).all() and torch.isfinite(b.float()).all()


# ---- f16 weights far below the largest ------------------------------------------------------------

def sink(n, d, gap, spread):
    """A query, n keys and values of one head: key 0 scores 2^gap times the weight of the others (which
    vary by `spread`), and its value is zero, so the output is the tail's alone."""
    q = torch.zeros(1, d)
    q[0, 0] = 4
    k = rows(1, n, d, dtype=torch.float32) * spread
    k[:, 0] = k[:, 0] if spread else 0
    k[0] = 0
    k[0, 0] = 4
    v = (0.5 + torch.rand(n, d, generator=torch.Generator().manual_seed(2))) if spread else \
        (0.5 + torch.rand(1, d, generator=torch.Generator().manual_seed(2))).expand(n, d).clone()
    v[0] = 0
    return q.half(), k.half(), v.half(), gap * math.log(2) / 16


GAPS = [(18.3, 0.0), (23.7, 0.0), (25.6, 0.0), (26.7, 0.0), (23.7, 0.05)]


@pytest.mark.parametrize("gap,spread", GAPS)
@pytest.mark.parametrize("new,hq,kv,d,ps", [(1, 2, [131072], 64, 64), (1, 1, [90001], 128, 16),
                                            (5, 4, [20000], 64, 128), (1, 2, [3000] * 40, 64, 16),
                                            (70, 2, [131072], 64, 64), (300, 1, [50001], 128, 16),
                                            (40, 4, [3000] * 20, 128, 32)])
def test_f16_tails_of_long_caches(P, new, hq, kv, d, ps, gap, spread):
    """One key far above a long tail: the tail is in the output with its whole weight."""
    m = kv[0]
    q, k, v, scale = sink(m, d, gap, spread)
    q = q.expand(new, d)
    pages = -(-m // ps)
    kc, vc = (pages_of(x[None], ps).cuda() for x in (k, v))
    table = i32([list(range(pages))] * len(kv))                 # every request reads the same pages
    T = new * len(kv)
    qs = q.repeat(len(kv), 1)[None].expand(hq, T, d).contiguous().cuda()
    lse = torch.zeros(hq, T, device="cuda")
    out = P.pisa_paged_attention(qs, kc, vc, table, i32([new * b for b in range(len(kv) + 1)]), i32(kv), scale=scale,
                                 lse=lse)
    P.pisa_device_status()
    _, want, bound, ln, ln_bound, _ = U.attend(q.double(), k.double(), v.double(), torch.arange(m - new, m), scale,
                                               U.half_step(HF))
    for b in range(len(kv)):
        r = slice(b * new, (b + 1) * new)
        for h in range(hq):
            U.check(out[h, r], want, bound, f"request {b} head {h}")
            U.check(lse[h, r], ln, ln_bound, f"lse of request {b} head {h}")


@pytest.mark.parametrize("gap,spread", GAPS)
@pytest.mark.parametrize("lens,d", [([20000], 64), ([9000, 300, 4000], 128)])
def test_f16_tails_of_long_prompts(P, lens, d, gap, spread):
    n = max(lens)
    q, k, v, scale = sink(n, d, gap, spread)
    T = sum(lens)
    qs = q.expand(T, d)[None].contiguous().cuda()
    ks, vs = (torch.cat([x[:m] for m in lens])[None].cuda() for x in (k, v))
    cu = i32(U.offsets(lens))
    for f32 in (None, torch.zeros(1, T, d, device="cuda")):
        lse = torch.zeros(1, T, device="cuda")
        out = P.pisa_varlen_attention(qs, ks, vs, cu, scale=scale, lse=lse, out_f32=f32)
        P.pisa_device_status()
        for a, m in zip(U.offsets(lens), lens):
            at = torch.tensor(sorted({0, 1, 130, 299, m // 2, m - 2, m - 1}))
            at = at[at < m]
            _, want, bound, ln, ln_bound, _ = U.attend(q.expand(len(at), d).double(), k[:m].double(), v[:m].double(),
                                                       at, scale, U.half_step(HF))
            U.check(out[0, a + at], want, bound, f"out of {m}")
            U.check(lse[0, a + at], ln, ln_bound, f"lse of {m}")
            if f32 is not None:
                U.check(f32[0, a + at].half(), want, bound, f"out_f32 of {m}")



# ---- rows of no sequence ---------------------------------------------------------------------------

def stale(*like):
    """Memory of the allocator that holds NaN: what an uninitialised result would show."""
    held = [torch.full_like(x, math.nan) for x in like for _ in range(4)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("cu,T", [([5, 40, 100], 130), ([7, 7, 9], 9), ([130, 130], 130), ([3, 500], 500)])
def test_rows_before_the_first_sequence_are_zero(P, cu, T):
    hq, hkv, d = 4, 2, 64
    q, k, v, g = (rows(i, h, T, d).cuda() for i, h in ((1, hq), (2, hkv), (3, hkv), (4, hq)))
    a, b = cu[0], cu[-1]
    stale(q, k, v)
    plain = P.varlen_attention(q, k, v, i32(cu))
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    stale(q, k, v)
    out = P.varlen_attention(*leaves, i32(cu))
    stale(q, k, v)
    grads = torch.autograd.grad(out, leaves, g)
    P.pisa_device_status()
    for x in (plain, out, *grads):
        assert (x[:, :a] == 0).all() and (x[:, b:] == 0).all()
    # the sequences themselves: as where they begin at row 0
    if b > a:
        cut = [x[:, a:b].detach().contiguous().requires_grad_() for x in (q, k, v)]
        ref = P.varlen_attention(*cut, i32([c - a for c in cu]))
        assert torch.equal(out[:, a:b], ref)
        with torch.no_grad():
            assert torch.equal(plain[:, a:b], P.varlen_attention(*cut, i32([c - a for c in cu])))
        for x, y in zip(grads, torch.autograd.grad(ref, cut, g[:, a:b].contiguous())):
            assert torch.equal(x[:, a:b], y)
    # without zero_tail they keep what they held
    kept = torch.full_like(q, 7.0)
    P.pisa_varlen_attention(q, k, v, i32(cu), out=kept)
    assert (kept[:, :a] == 7).all() and (kept[:, b:] == 7).all() and torch.equal(kept[:, a:b], plain[:, a:b])


# ---- non-finite queries -------------------------------------------------------------------------------

@pytest.mark.parametrize("new,kv,ps,d", [([1, 1], [50000, 300], 64, 128), ([40, 1], [50000, 300], 64, 128),
                                         ([1, 1], [50, 30], 16, 64), ([40, 3], [50, 30], 16, 128)])
def test_a_query_of_nan_gives_nan_and_touches_no_other_row(P, new, kv, ps, d):
    """Also where the request's keys are shared out over many blocks, whose parts are joined."""
    hq, hkv = 4, 2
    need = [-(-m // ps) for m in kv]
    kc, vc = (rows(i, sum(need), hkv, ps, d).cuda() for i in (2, 3))
    table = torch.full((2, max(need)), -1)
    table[0, :need[0]], table[1, :need[1]] = torch.arange(need[0]), torch.arange(need[0], sum(need))
    q = rows(1, hq, sum(new), d).cuda()
    dirty = q.clone()
    bad = new[0] // 2
    dirty[1, bad] = math.nan

    def call(x):
        lse = torch.zeros(hq, sum(new), device="cuda")
        return P.pisa_paged_attention(x, kc, vc, i32(table.tolist()), i32(U.offsets(new)), i32(kv), lse=lse), lse

    a, b = call(q), call(dirty)
    P.pisa_device_status()
    for x, y in zip(a, b):
        assert torch.isnan(y[1, bad]).all()
        keep = torch.ones(x.shape[:2], dtype=torch.bool)
        keep[1, bad] = False
        assert torch.equal(x[keep], y[keep])


@pytest.mark.parametrize("lens,row", [([6000], 5990), ([300, 20], 311)])
def test_a_query_of_nan_in_a_prompt(P, lens, row):
    T, d = sum(lens), 64
    q, k, v = (rows(i, h, T, d).cuda() for i, h in ((1, 2), (2, 1), (3, 1)))
    dirty = q.clone()
    dirty[0, row] = math.nan

    def call(x, f32):
        lse = torch.zeros(2, T, device="cuda")
        return P.pisa_varlen_attention(x, k, v, i32(U.offsets(lens)), lse=lse, out_f32=f32), lse

    for f32 in (None, torch.zeros(2, T, d, device="cuda")):
        a, b = call(q, f32), call(dirty, f32)
        P.pisa_device_status()
        for x, y in zip(a, b):
            assert torch.isnan(y[0, row]).all()
            keep = torch.ones(x.shape[:2], dtype=torch.bool)
            keep[0, row] = False
            assert torch.equal(x[keep], y[keep])


# ---- padded batches -----------------------------------------------------------------------------------

@pytest.mark.parametrize("new,hq,hkv,d,ps", [([1] * 40 + [380], 4, 2, 128, 64), ([1] * 30 + [400], 8, 4, 64, 16)])
def test_padding_rows_change_no_bits(P, new, hq, hkv, d, ps):
    """A chunk beside single tokens: rows behind the batch, as many as make the number of requests divide
    the number of rows or not, are not a reason to work otherwise."""
    kv = [n + 50 * (i % 7) for i, n in enumerate(new)]
    need = [-(-m // ps) for m in kv]
    at = U.offsets(need)
    table = i32([list(range(a, a + n)) + [-1] * (max(need) - n) for a, n in zip(at, need)])
    kc, vc = (rows(i, sum(need), hkv, ps, d).cuda() for i in (2, 3))
    n, B = sum(new), len(new)
    up = -(-n // B) * B
    q = rows(1, hq, up + 2, d).cuda()
    got = [P.pisa_paged_attention(q[:, :T], kc, vc, table, i32(U.offsets(new)), i32(kv))[:, :n]
           for T in (up - 1 if up > n else up + 1, up, up + 1, up + 2)]
    P.pisa_device_status()
    assert all(torch.equal(x, got[0]) for x in got)


# ---- a caller's own context ---------------------------------------------------------------------------

def test_a_callers_context_stays_current(P):
    """A host thread with a context of its own has it after the call too, and the call works there."""
    import ctypes
    import threading
    from block_sparse_attention_stats_b200 import _lib as L

    torch.zeros(1, device="cuda")
    cuda, lib = ctypes.CDLL("libcuda.so.1"), L.load()
    seen, failed = {}, []

    def ok(code):
        assert code == 0, f"CUresult {code}"

    def current():
        c = ctypes.c_void_p()
        ok(cuda.cuCtxGetCurrent(ctypes.byref(c)))
        return c.value

    def body():
        mine = ctypes.c_void_p()
        ok(cuda.cuCtxCreate_v2(ctypes.byref(mine), 0, 0))
        try:
            # tensor maps are encoded, and refused (a group's stride past 2^40 bytes): nothing is launched
            far = L.PisaRows(1 << 20, (1 << 38) - 8, 64)
            near = L.PisaRows(2 << 20, 6400, 64)
            seen["status"] = lib.pisa_varlen_attention(
                far, near, near, L.PISA_BF16, 3 << 20, 1, 100, 8, 2, 64, 0.0, 1, L.PisaRows(4 << 20, 6400, 64), None,
                None, 5 << 20, 1 << 30, None)
            seen["kept"] = current() == mine.value
            if not seen["kept"]:
                return
            # one token attends to itself: out = v
            d, need = 64, lib.pisa_varlen_attention_workspace_bytes(1, 1, 64)
            at = ctypes.c_uint64()
            ok(cuda.cuMemAlloc_v2(ctypes.byref(at), ctypes.c_size_t(4096 + need)))
            q, k, v, out, cu, ws = (at.value + x for x in (0, 256, 512, 768, 1024, 4096))
            x = (torch.arange(d) / 8).to(BF)
            for p in (q, k, v):
                ok(cuda.cuMemcpyHtoD_v2(ctypes.c_uint64(p), ctypes.c_void_p(x.data_ptr()), ctypes.c_size_t(2 * d)))
            lens = torch.tensor([0, 1], dtype=torch.int32)
            ok(cuda.cuMemcpyHtoD_v2(ctypes.c_uint64(cu), ctypes.c_void_p(lens.data_ptr()), ctypes.c_size_t(8)))
            row = lambda p: L.PisaRows(p, d, d)
            seen["call"] = lib.pisa_varlen_attention(row(q), row(k), row(v), L.PISA_BF16, cu, 1, 1, 1, 1, d, 0.0, 1,
                                                     row(out), None, None, ws, need, None)
            ok(cuda.cuCtxSynchronize())
            got = torch.zeros(d, dtype=BF)
            ok(cuda.cuMemcpyDtoH_v2(ctypes.c_void_p(got.data_ptr()), ctypes.c_uint64(out), ctypes.c_size_t(2 * d)))
            seen["out"] = torch.equal(got, x)
            seen["still"] = current() == mine.value
            ok(cuda.cuMemFree_v2(at))
        finally:
            ok(cuda.cuCtxDestroy_v2(mine))

    def guarded():
        try:
            body()
        except BaseException as e:
            failed.append(e)

    t = threading.Thread(target=guarded)
    t.start()
    t.join()
    assert not failed, failed
    assert seen == dict(status=L.PISA_ERR_CUDA, kept=True, call=L.PISA_OK, out=True, still=True)


# ---- operands that lie between one another -----------------------------------------------------------

@pytest.mark.parametrize("tokens_first", [False, True])
def test_a_step_on_slices_of_one_projection_and_one_cache(P, tokens_first):
    """q, k, v of one fused tensor, out beside them, keys and values of two layers in one cache tensor."""
    hq, hkv, d, ps, total = 4, 2, 64, 16, 20
    new = [30, 1, 70]
    T = sum(new)
    fused = rows(1, T, 2 * hq + 2 * hkv, d).cuda().transpose(0, 1)
    q, k, v, out = fused[:hq], fused[hq:hq + hkv], fused[hq + hkv:hq + 2 * hkv], fused[hq + 2 * hkv:]
    shape = (total, 4, ps, hkv, d) if tokens_first else (total, 4, hkv, ps, d)
    both = torch.full(shape, 7.0, dtype=BF, device="cuda")
    kc, vc = (both[:, i].transpose(1, 2) if tokens_first else both[:, i] for i in (1, 2))
    sep = [torch.full((total, hkv, ps, d), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    args = lambda: (i32([0, 0, 0]), i32(new), torch.full((3, 6), -1, dtype=torch.int32, device="cuda"),
                    i32(list(range(total))), i32([total]))
    want, _ = P.pisa_paged_step(q.contiguous(), k.contiguous(), v.contiguous(), *sep, *args())
    got, _ = P.pisa_paged_step(q, k, v, kc, vc, *args(), out=out)
    P.pisa_device_status()
    assert torch.equal(got, want) and torch.equal(kc, sep[0]) and torch.equal(vc, sep[1])
    assert (both[:, 0] == 7).all() and (both[:, 3] == 7).all()


# ---- the backward's contract ----------------------------------------------------------------------------

@pytest.mark.parametrize("scale", [0.3, 1.0, 0.02])
@pytest.mark.parametrize("d,causal", [(64, True), (128, True), (128, False)])
def test_gradients_of_an_explicit_scale(P, scale, d, causal):
    lens, hq, hkv = [300, 41, 1], 6, 2
    T = sum(lens)
    q, k, v, g = (rows(i, h, T, d) for i, h in ((1, hq), (2, hkv), (3, hkv), (4, hq)))
    want, bound = U.varlen_grads(*(x.double() for x in (q, k, v, g)), lens, causal, scale, BF)
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    got = torch.autograd.grad(P.varlen_attention(*leaves, i32(U.offsets(lens)), causal, scale), leaves, g.cuda())
    P.pisa_device_status()
    for name, x in zip(("dq", "dk", "dv"), got):
        U.check(x, want[name], bound[name], f"{name} at scale {scale}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[3000, 5, 700], [130, 40]])
def test_backward_into_slices_of_one_gradient(P, lens, d):
    """dq, dk, dv as slices of one [T, Hq + 2 Hkv, d] tensor, long enough that ranges cut units; rows of no
    sequence keep what they held."""
    hq, hkv, pad, first = 4, 2, 9, 3
    n = sum(lens)
    T = first + n + pad
    q, k, v, g = (rows(i, h, T, d) for i, h in ((1, hq), (2, hkv), (3, hkv), (4, hq)))
    cu = i32([first + x for x in U.offsets(lens)])
    dev = [x.cuda() for x in (q, k, v, g)]
    lse, o32 = torch.empty(hq, T, device="cuda"), torch.empty(hq, T, d, device="cuda")
    P.pisa_varlen_attention(*dev[:3], cu, lse=lse, out_f32=o32)
    fused = torch.full((T, hq + 2 * hkv, d), 7.0, dtype=BF, device="cuda").transpose(0, 1)
    parts = (fused[:hq], fused[hq:hq + hkv], fused[hq + hkv:])
    got = P.pisa_varlen_attention_bwd(*dev, lse, o32, cu, grads=parts)
    dense = P.pisa_varlen_attention_bwd(*dev, lse, o32, cu,
                                        grads=tuple(torch.full_like(x, 7.0) for x in dev[:3]))
    P.pisa_device_status()
    r = slice(first, first + n)
    want, bound = U.varlen_grads(*(x[:, r].double() for x in (q, k, v, g)), lens, True, d ** -0.5, BF)
    for name, x, y, z in zip(("dq", "dk", "dv"), got, dense, parts):
        assert x is z and torch.equal(x, y)
        U.check(x[:, r], want[name], bound[name], name)
        assert (x[:, :first] == 7).all() and (x[:, first + n:] == 7).all()


# ---- offsets that are none ----------------------------------------------------------------------------

@pytest.mark.parametrize("cu", [[0, 300] * 40, [0, 100, 50, 300], [0, 100, 301], [-1, 100, 300], [300, 0]])
def test_nothing_is_worked_on_with_bad_offsets(P, cu):
    """Each pair could name every row: the work of such a call is bounded because there is none."""
    from block_sparse_attention_stats_b200 import _lib as L
    T, hq, hkv, d, ps = 300, 4, 2, 64, 16
    q, k, v, g = (rows(i, h, T, d).cuda() for i, h in ((1, hq), (2, hkv), (3, hkv), (4, hq)))
    kept = lambda x: torch.full_like(x, 7.0)
    out, grads = kept(q), tuple(kept(x) for x in (q, k, v))
    lse, o32 = torch.zeros(hq, T, device="cuda"), torch.zeros(hq, T, d, device="cuda")
    kc, vc = (pages_of(x.cpu(), ps).cuda() for x in (k, v))
    B = len(cu) - 1
    paged, few = kept(q), kept(q[:, :B])
    table, kv = i32([list(range(kc.shape[0]))] * B), i32([T] * B)

    def refused():
        with pytest.raises(P.PisaError) as e:
            P.pisa_device_status()
        assert e.value.status == L.PISA_ERR_DEVICE

    P.pisa_varlen_attention(q, k, v, i32(cu), out=out)
    refused()
    P.pisa_varlen_attention_bwd(q, k, v, g, lse, o32, i32(cu), grads=grads)
    refused()
    P.pisa_paged_attention(q, kc, vc, table, i32(cu), kv, out=paged)
    refused()
    P.pisa_paged_attention(q[:, :B], kc, vc, table, i32([c // 100 if c > 99 else c for c in cu[:-1]] + [B + 1]), kv, out=few)
    refused()
    for x in (out, paged, few, *grads):
        assert (x == 7).all()
