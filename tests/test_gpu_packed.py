"""Attention over packed sequences: the kernels against their 64-bit form, with the bounds of
packed_util, at the lengths, heads, layouts and masks where they can go wrong."""
import math
import threading

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


def rows(seed, h, t, d, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(h, t, d, generator=g) * scale).to(dtype)


def cu_of(lens):
    return torch.tensor(U.offsets(lens), dtype=torch.int32, device="cuda")


def tokens_first(x):
    """The same values in a [T, H, d] layout, seen as [H, T, d]."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


CASES = [
    # lens, pad, hq, hkv, d, dtype, causal
    ([1], 0, 1, 1, 64, BF, True),
    ([1], 0, 1, 1, 128, HF, False),
    ([0, 3, 0], 5, 2, 1, 64, HF, True),
    ([127], 0, 1, 1, 128, BF, True),
    ([128, 129], 0, 2, 2, 128, BF, True),
    ([5, 64, 1, 130, 17, 0, 200], 9, 8, 2, 64, HF, True),
    ([300, 41], 2, 6, 2, 128, BF, True),           # 3 heads to a key head: 126 of 128 rows
    ([300, 41], 0, 6, 2, 64, BF, False),
    ([257, 511], 0, 14, 2, 128, HF, True),         # 7 heads
    ([90], 0, 128, 1, 64, BF, True),               # a subtile is one token
    ([33, 7], 0, 100, 1, 128, BF, False),          # 100 rows of 128 used
    ([1030], 0, 4, 4, 64, BF, False),
    ([1500, 2], 0, 3, 1, 128, BF, True),
]


def ids(c):
    return f"{'-'.join(map(str, c[0]))}_h{c[2]}x{c[3]}_d{c[4]}_{'bf16' if c[5] == BF else 'f16'}_{'c' if c[6] else 'n'}"


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(P, case):
    lens, pad, hq, hkv, d, dtype, causal = case
    T = sum(lens) + pad
    q, k, v = rows(1, hq, T, d, dtype, 1.5), rows(2, hkv, T, d, dtype), rows(3, hkv, T, d, dtype)
    want = U.varlen(q.double(), k.double(), v.double(), lens, causal, d ** -0.5, dtype)
    out = torch.full((hq, T, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((hq, T), 7.0, device="cuda")
    got = P.pisa_varlen_attention(q.cuda(), k.cuda(), v.cuda(), cu_of(lens), causal, out=out, lse=lse)
    P.pisa_device_status()
    assert got is out
    n = sum(lens)
    U.check(out[:, :n], want["out"][:, :n], want["bound"][:, :n], "out")
    U.check(lse[:, :n], want["lse"][:, :n], want["lse_bound"][:, :n], "lse")
    assert (out[:, n:] == 7).all() and (lse[:, n:] == 7).all()      # left as they were


@pytest.mark.parametrize("case", [c for c in CASES if c[5] == BF], ids=ids)
def test_gradients(P, case):
    lens, pad, hq, hkv, d, dtype, causal = case
    T, n = sum(lens) + pad, sum(lens)
    q, k, v, g = (rows(1, hq, T, d, dtype, 1.5), rows(2, hkv, T, d, dtype), rows(3, hkv, T, d, dtype),
                  rows(4, hq, T, d, dtype))
    want, bound = U.varlen_grads(q.double(), k.double(), v.double(), g.double(), lens, causal, d ** -0.5, dtype)
    ref = U.varlen(q.double(), k.double(), v.double(), lens, causal, d ** -0.5, dtype)
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    out = P.varlen_attention(*leaves, cu_of(lens), causal)
    U.check(out, ref["out"], ref["bound"] + 1e-30, "out")
    got = torch.autograd.grad(out, leaves, g.cuda())
    P.pisa_device_status()
    for name, x in zip(("dq", "dk", "dv"), got):
        U.check(x, want[name], bound[name], name)
        assert (x[:, n:] == 0).all()


def test_strided_layouts(P):
    """[T, H, d] tensors, slices of one fused projection, a strided out."""
    lens, hq, hkv, d = [70, 200, 1], 6, 2, 64
    T = sum(lens)
    fused = rows(5, hq + 2 * hkv, T, d, BF).transpose(0, 1).contiguous().cuda().transpose(0, 1)
    q, k, v = fused[:hq], fused[hq:hq + hkv], fused[hq + hkv:]
    assert not q.is_contiguous()
    dense = P.pisa_varlen_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu_of(lens))
    out = tokens_first(torch.zeros(hq, T, d, dtype=BF, device="cuda"))
    P.pisa_varlen_attention(q, k, v, cu_of(lens), out=out)
    assert torch.equal(out, dense)
    g = rows(6, hq, T, d, BF).cuda()
    a = [x.clone().detach().requires_grad_() for x in (q, k, v)]
    ga = torch.autograd.grad(P.varlen_attention(*a, cu_of(lens)), a, tokens_first(g))
    b = [x.contiguous().requires_grad_() for x in (q, k, v)]
    gb = torch.autograd.grad(P.varlen_attention(*b, cu_of(lens)), b, g)
    for x, y in zip(ga, gb):
        assert torch.equal(x, y)
    # a gradient that is broadcast (stride 0), as of a sum, is laid out first
    gc = torch.autograd.grad(P.varlen_attention(*b, cu_of(lens)).sum(), b)
    gd = torch.autograd.grad(P.varlen_attention(*b, cu_of(lens)), b, torch.ones_like(g))
    for x, y in zip(gc, gd):
        assert torch.equal(x, y)
    # broadcast keys: their gradient is the sum over the heads that share them
    one = k[:1].detach().contiguous().requires_grad_()
    wide = one.expand(hkv, -1, -1)
    ge, = torch.autograd.grad(P.varlen_attention(b[0], wide, b[2], cu_of(lens)), one, g)
    full = one.detach().repeat(hkv, 1, 1).requires_grad_()
    gf, = torch.autograd.grad(P.varlen_attention(b[0], full, b[2], cu_of(lens)), full, g)
    assert torch.allclose(ge.float(), gf.float().sum(0, keepdim=True), rtol=2 ** -7, atol=1e-3)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_sequences_do_not_touch(P, bad):
    """Non-finite values in one sequence, or behind the last, change no other sequence's bits."""
    lens, pad, hq, hkv, d = [70, 40, 300, 129], 20, 4, 2, 128
    T, at = sum(lens) + pad, U.offsets(lens)
    clean = [x.cuda() for x in (rows(1, hq, T, d, BF, 1.5), rows(2, hkv, T, d, BF), rows(3, hkv, T, d, BF),
                                rows(4, hq, T, d, BF))]
    dirty = [x.clone() for x in clean]
    for x in dirty:
        x[:, at[1]:at[2]] = bad
        x[:, at[4]:] = bad

    def run(q, k, v, g):
        leaves = [x.clone().requires_grad_() for x in (q, k, v)]
        out = P.varlen_attention(*leaves, cu_of(lens))
        return (P.pisa_varlen_attention(q, k, v, cu_of(lens), zero_tail=True), out.detach(),
                *torch.autograd.grad(out, leaves, g))

    keep = torch.ones(T, dtype=torch.bool)
    keep[at[1]:at[2]] = False
    for a, b in zip(run(*clean), run(*dirty)):
        assert torch.isfinite(b[:, keep].float()).all()
        assert torch.equal(a[:, keep], b[:, keep])


def test_peaked_rows(P):
    """Scores so large that one key holds the weight: the running maximum moves by far more than
    its threshold, and dP - Delta cancels."""
    lens, hq, hkv, d = [400, 130], 2, 1, 64
    T = sum(lens)
    q, k, v, g = rows(1, hq, T, d, BF, 12.0), rows(2, hkv, T, d, BF, 2.0), rows(3, hkv, T, d, BF), rows(4, hq, T, d, BF)
    ref = U.varlen(q.double(), k.double(), v.double(), lens, True, d ** -0.5, BF)
    want, bound = U.varlen_grads(q.double(), k.double(), v.double(), g.double(), lens, True, d ** -0.5, BF)
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    out = P.varlen_attention(*leaves, cu_of(lens))
    U.check(out, ref["out"], ref["bound"], "out")
    for name, x in zip(("dq", "dk", "dv"), torch.autograd.grad(out, leaves, g.cuda())):
        U.check(x, want[name], bound[name], name)


def test_gradients_against_differences(P):
    """A directional derivative of the 64-bit form along random directions."""
    lens, hq, hkv, d = [37, 60], 4, 2, 64
    T = sum(lens)
    x = [rows(1, hq, T, d, BF), rows(2, hkv, T, d, BF), rows(3, hkv, T, d, BF)]
    g = rows(4, hq, T, d, BF).double()
    leaves = [y.cuda().requires_grad_() for y in x]
    grads = torch.autograd.grad(P.varlen_attention(*leaves, cu_of(lens)), leaves, g.to(BF).cuda())
    _, bound = U.varlen_grads(*(y.double() for y in x), g, lens, True, d ** -0.5, BF)
    for i in range(3):
        e = rows(50 + i, *x[i].shape, torch.float64)
        up, down = ([y.double() + s * e if j == i else y.double() for j, y in enumerate(x)] for s in (1e-5, -1e-5))
        want = sum(float((U.varlen(*y, lens, True, d ** -0.5, BF)["out"] * g).sum()) * s
                   for y, s in ((up, 1), (down, -1))) / 2e-5
        got = float((grads[i].double().cpu() * e).sum())
        most = float((bound["dq dk dv".split()[i]] * e.abs()).sum())
        assert abs(got - want) <= most + 1e-6 * abs(want), (i, got, want, most)


def test_large_scale_and_default_scale(P):
    lens, d = [200], 64
    q, k, v = (rows(i, 2, 200, d, BF).cuda() for i in (1, 2, 3))
    a = P.pisa_varlen_attention(q, k, v, cu_of(lens))
    b = P.pisa_varlen_attention(q, k, v, cu_of(lens), scale=d ** -0.5)
    assert torch.equal(a, b)
    want = U.varlen(*(x.cpu().double() for x in (q, k, v)), lens, True, 3.0, BF)
    U.check(P.pisa_varlen_attention(q, k, v, cu_of(lens), scale=3.0), want["out"], want["bound"], "scale 3")


def test_repeats_bitwise_and_cut_units_agree(P):
    """A long sequence beside many short ones: ranges cut units; the same bits every time."""
    lens, hq, hkv, d = [2500] + [3] * 40 + [700], 4, 2, 128
    T = sum(lens)
    q, k, v, g = (rows(1, hq, T, d, BF, 1.5), rows(2, hkv, T, d, BF), rows(3, hkv, T, d, BF), rows(4, hq, T, d, BF))
    ref = U.varlen(q.double(), k.double(), v.double(), lens, True, d ** -0.5, BF)
    want, bound = U.varlen_grads(q.double(), k.double(), v.double(), g.double(), lens, True, d ** -0.5, BF)
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    first = None
    for _ in range(3):
        out = P.varlen_attention(*leaves, cu_of(lens))
        got = (out.detach(), *torch.autograd.grad(out, leaves, g.cuda()))
        if first is None:
            first = got
            U.check(out, ref["out"], ref["bound"], "out")
            for name, x in zip(("dq", "dk", "dv"), got[1:]):
                U.check(x, want[name], bound[name], name)
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_graph_replays_with_other_lengths(P):
    """A captured call follows the offsets in its buffers; two graphs keep workspaces of their own."""
    T, hq, hkv, d = 600, 4, 2, 64
    q, k, v = (rows(i, h, T, d, BF).cuda() for i, h in ((1, hq), (2, hkv), (3, hkv)))
    need = P._lib.load().pisa_varlen_attention_workspace_bytes(hq, hkv, d)
    side = torch.cuda.Stream()
    graphs = []
    for lens in ([100, 500, 0], [300, 7, 200]):
        cu, out = cu_of(lens), torch.zeros_like(q)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            P.pisa_varlen_attention(q, k, v, cu, out=out, workspace=ws)
        torch.cuda.current_stream().wait_stream(side)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            P.pisa_varlen_attention(q, k, v, cu, out=out, workspace=ws)
        graphs.append((gr, cu, out, ws))
    for lens in ([600, 0, 0], [1, 598, 1], [0, 0, 0], [200, 200, 100]):
        for gr, cu, out, _ in graphs:
            cu.copy_(cu_of(lens))
            out.fill_(5.0)
            gr.replay()
        want = P.pisa_varlen_attention(q, k, v, cu_of(lens), out=torch.full_like(q, 5.0))
        for _, _, out, _ in graphs:
            assert torch.equal(out, want)
    P.pisa_device_status()
    del graphs


def test_training_step_replays_from_a_graph(P):
    lens, hq, hkv, d = [100, 77], 4, 2, 64
    T = sum(lens)
    leaves = [rows(i, h, T, d, BF).cuda().requires_grad_() for i, h in ((1, hq), (2, hkv), (3, hkv))]
    g, cu = rows(4, hq, T, d, BF).cuda(), cu_of(lens)

    def step():
        out = P.varlen_attention(*leaves, cu)
        return (out, *torch.autograd.grad(out, leaves, g))

    eager = [x.detach().clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        res = step()
    for x in res:
        x.detach().zero_()
    gr.replay()
    torch.cuda.synchronize()
    P.pisa_device_status()
    assert all(torch.equal(a, b) for a, b in zip(eager, res))
    del gr


def test_two_streams_at_once(P):
    lens, hq, hkv, d = [900, 100], 8, 2, 128
    T = sum(lens)
    sets = [[rows(10 * s + i, h, T, d, BF).cuda() for i, h in ((1, hq), (2, hkv), (3, hkv))] for s in (1, 2)]
    want = [P.pisa_varlen_attention(*x, cu_of(lens)) for x in sets]
    torch.cuda.synchronize()
    cu = cu_of(lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            got[i].append(P.pisa_varlen_attention(*sets[i], cu, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_bad_offsets_are_recorded_and_stay_inside(P):
    T, d = 100, 64
    q, k, v = (rows(i, 2, T, d, BF).cuda() for i in (1, 2, 3))
    from block_sparse_attention_stats_b200 import _lib
    for cu in ([0, 50, 400], [-5, 20, 100], [0, 80, 30]):
        P.pisa_varlen_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        with pytest.raises(P.PisaError) as e:
            P.pisa_device_status()
        assert e.value.status == _lib.PISA_ERR_DEVICE
    P.pisa_varlen_attention(q, k, v, cu_of([100]))
    P.pisa_device_status()


def test_nothing_to_do(P):
    """No tokens at all; a batch of empty sequences."""
    q = torch.zeros(4, 0, 64, dtype=BF, device="cuda", requires_grad=True)
    k, v = (torch.zeros(2, 0, 64, dtype=BF, device="cuda", requires_grad=True) for _ in range(2))
    out = P.varlen_attention(q, k, v, cu_of([0, 0]))
    grads = torch.autograd.grad(out.float().sum(), (q, k, v))
    assert out.shape == q.shape and [g.shape for g in grads] == [q.shape, k.shape, v.shape]
    q, k, v = (rows(i, 2, 10, 64, BF).cuda().requires_grad_() for i in (1, 2, 3))
    out = P.varlen_attention(q, k, v, cu_of([0, 0, 0]))
    assert (out == 0).all()
    assert all((g == 0).all() for g in torch.autograd.grad(out.float().sum(), (q, k, v)))
    P.pisa_device_status()


@pytest.mark.parametrize("seed", range(10))
def test_random_batches(P, seed):
    """Batches of any shape: where ranges cut units differs from one to the next."""
    import random
    rng = random.Random(seed)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3])
    hq = hkv * rng.choice([1, 2, 3, 5, 8])
    longest = rng.choice([20, 150, 700])
    lens = [rng.choice([0, 1, rng.randint(1, longest), longest]) for _ in range(rng.randint(1, 9))]
    causal, T = rng.random() < 0.7, sum(lens) + 3
    q, k, v, g = (rows(seed + i, h, T, d, BF, s) for i, h, s in ((1, hq, 1.5), (2, hkv, 1), (3, hkv, 1), (4, hq, 1)))
    ref = U.varlen(q.double(), k.double(), v.double(), lens, causal, d ** -0.5, BF)
    want, bound = U.varlen_grads(q.double(), k.double(), v.double(), g.double(), lens, causal, d ** -0.5, BF)
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    n = sum(lens)
    lse, o32 = torch.zeros(hq, T, device="cuda"), torch.zeros(hq, T, d, device="cuda")
    for f in (None, o32):                    # without and with the float32 output
        out = P.pisa_varlen_attention(*(x.detach() for x in leaves), cu_of(lens), causal, lse=lse, out_f32=f)
        U.check(out[:, :n], ref["out"][:, :n], ref["bound"][:, :n], "out")
        U.check(lse[:, :n], ref["lse"][:, :n], ref["lse_bound"][:, :n], "lse")
    U.check(o32[:, :n].to(BF), ref["out"][:, :n], ref["bound"][:, :n], "out_f32")
    got = torch.autograd.grad(P.varlen_attention(*leaves, cu_of(lens), causal), leaves, g.cuda())
    P.pisa_device_status()
    for name, x in zip(("dq", "dk", "dv"), got):
        U.check(x, want[name], bound[name], name)


def test_backward_on_another_stream(P):
    lens, d = [200, 31], 64
    leaves = [rows(i, h, 231, d, BF).cuda().requires_grad_() for i, h in ((1, 4), (2, 2), (3, 2))]
    g, cu = rows(4, 4, 231, d, BF).cuda(), cu_of(lens)
    want = torch.autograd.grad(P.varlen_attention(*leaves, cu), leaves, g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = torch.autograd.grad(P.varlen_attention(*leaves, cu), leaves, g)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("which", ["forward", "backward", "paged", "write"])
def test_first_call_of_a_thread(P, which):
    """Each thread has a current context of its own, and none before its first call."""
    lens, d = [200, 31], 64
    q, k, v, g = (rows(i, h, 231, d, BF).cuda() for i, h in ((1, 4), (2, 2), (3, 2), (4, 4)))
    cu = cu_of(lens)
    kc, vc = (rows(i, 20 * 2 * 16, 1, d, BF).cuda().view(20, 2, 16, d) for i in (5, 6))
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    kv = torch.tensor([150, 29], dtype=torch.int32, device="cuda")
    lse, o32 = torch.empty(4, 231, device="cuda"), torch.empty(4, 231, d, device="cuda")
    out = P.pisa_varlen_attention(q, k, v, cu, lse=lse, out_f32=o32)
    two = cu_of([1, 1])

    def call():
        if which == "forward":
            return P.pisa_varlen_attention(q, k, v, cu, out=torch.empty_like(q)),
        if which == "backward":
            return P.pisa_varlen_attention_bwd(q, k, v, g, lse, o32, cu)
        if which == "paged":
            return P.pisa_paged_attention(q[:, :2], kc, vc, table, two, kv),
        caches = torch.zeros_like(kc), torch.zeros_like(vc)
        P.pisa_page_write(k, v, torch.arange(231, device="cuda"), *caches)
        return caches

    want = call()      # what it allocates is in the allocator's pool from here on
    torch.cuda.synchronize()
    got = []

    def body():
        try:
            got.extend(call())
            torch.cuda.synchronize()
        except Exception as e:
            got.append(e)

    del out
    worker = threading.Thread(target=body)
    worker.start()
    worker.join()
    assert len(got) == len(want), got
    for a, b in zip(got, want):
        assert torch.is_tensor(a) and torch.equal(a, b), a


def test_second_derivative_is_refused(P):
    leaves = [rows(i, 2, 20, 64, BF).cuda().requires_grad_() for i in (1, 2, 3)]
    out = P.varlen_attention(*leaves, cu_of([20]))
    dq, = torch.autograd.grad(out.float().square().sum(), leaves[:1], create_graph=True)
    with pytest.raises(RuntimeError):
        dq.float().sum().backward()


def test_out_may_not_be_an_input(P):
    q, k, v = (rows(i, 2, 20, 64, BF).cuda() for i in (1, 2, 3))
    for bad in (q, k, v):
        with pytest.raises(P.PisaError):
            P.pisa_varlen_attention(q, k, v, cu_of([20]), out=bad)
    with pytest.raises(ValueError):
        P.pisa_varlen_attention(q, k, v, cu_of([20]).cpu())
    with pytest.raises(ValueError):
        P.pisa_varlen_attention(q, k, v, cu_of([20]).long())
    with pytest.raises(ValueError):
        P.pisa_varlen_attention(q, k, v, cu_of([20]), lse=torch.zeros(2, 21, device="cuda"))
