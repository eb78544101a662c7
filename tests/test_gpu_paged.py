"""The paged key/value cache: plan, write and attention against their plain forms, and the whole
step as a server runs it."""
import math
import random

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


def paged_case(new, kv, hq, hkv, d, ps, dtype, seed=1, behind=math.nan):
    """q, caches whose rows behind every request's last position (and pages of nobody) hold
    `behind`, a table with -1 where no page is needed."""
    need = [-(-m // ps) for m in kv]
    total = sum(need) + 3
    order = list(range(total))
    random.Random(seed).shuffle(order)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (max(need) + 1 - n))
        at += n
    kc, vc = (rows(seed + i, total, hkv, ps, d, dtype=dtype) for i in (2, 3))
    used = torch.zeros(total, ps, dtype=torch.bool)
    for t, m in zip(table, kv):
        for j in range(m):
            used[t[j // ps], j % ps] = True
    dirty = [torch.where(used[:, None, :, None], c, torch.full_like(c, behind)) for c in (kc, vc)]
    return rows(seed + 1, hq, sum(new), d, dtype=dtype, scale=1.5), kc, vc, dirty, table


CASES = [
    # new, kv, hq, hkv, d, page, dtype
    ([1], [1], 1, 1, 64, 16, BF),
    ([1], [777], 8, 8, 64, 16, BF),
    ([1, 1, 1], [128, 129, 1], 4, 4, 128, 16, HF),
    ([1, 1], [3000, 45], 16, 1, 128, 64, BF),            # 16 heads to a key head
    ([1, 0, 1, 1], [500, 30, 0, 17], 40, 8, 128, 32, BF),  # no token; a token without keys
    ([1, 1], [260, 511], 7, 1, 64, 256, HF),
    ([3, 2, 4], [300, 2, 131], 8, 2, 128, 128, BF),      # up to 16 rows a request
    ([5, 8], [200, 8], 12, 4, 64, 16, HF),               # 24 rows in tiles of 30 of 32
    ([9, 20], [700, 20], 6, 2, 128, 32, BF),             # 27, 60: tiles of 63 of 64
    ([1, 1], [400, 333], 64, 1, 64, 64, BF),             # 64 rows, one token each
    ([1, 1], [400, 333], 96, 1, 128, 16, BF),            # the 128-row kernel for single tokens
    ([1, 1, 70, 1, 64, 257], [400, 19, 900, 2000, 64, 1157], 24, 8, 128, 16, BF),
    ([130, 200], [130, 1000], 4, 2, 64, 32, HF),
    ([300], [555], 3, 3, 128, 256, BF),
    ([6, 40], [3, 10], 4, 4, 64, 16, BF),                # fewer keys than tokens: rows without any
    ([2, 3], [1, 0], 4, 4, 64, 16, BF),
    ([8, 8], [200, 8], 12, 4, 64, 16, HF),               # drafts of one length: 24 rows in tiles of 30 of 32
    ([6, 6, 6], [700, 20, 6], 10, 2, 128, 32, BF),       # 30 rows
    ([32, 32], [45, 131], 3, 3, 128, 16, BF),            # 32 rows of one head
    ([1, 1, 1], [400, 1, 333], 40, 2, 64, 64, BF),       # 20 rows, one token each
    ([1] * 20 + [7], list(range(1, 21)) + [90], 4, 2, 128, 16, BF),   # single tokens and a few more: tiles of 16
    ([0] * 9 + [8, 1], [5] * 9 + [260, 30], 24, 8, 64, 16, HF),       # as many tokens as requests, on two of them
    ([1] * 20 + [70], [300] * 21, 20, 1, 128, 64, BF),   # a chunk among them: 128-row products
    # ends of tiles and of pages of 16 and 32, in 128-row products
    ([40] * 12, [40, 41, 129, 136, 137, 144, 145, 247, 248, 249, 256, 257], 6, 2, 128, 16, BF),
    ([23, 1, 8, 9, 130], [23, 1, 8, 9, 130], 12, 3, 128, 16, HF),
    ([40] * 6, [40, 129, 159, 160, 161, 257], 6, 2, 128, 32, BF),
    ([40, 200, 7], [20, 140, 3], 3, 3, 128, 16, BF),     # fewer keys than tokens
]


def ids(c):
    return f"n{'-'.join(map(str, c[0]))}_m{'-'.join(map(str, c[1]))}_h{c[2]}x{c[3]}_d{c[4]}_p{c[5]}"


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_paged_attention(P, case):
    new, kv, hq, hkv, d, ps, dtype = case
    q, kc, vc, dirty, table = paged_case(*case)
    want = U.paged(q.double(), kc.double(), vc.double(), table, new, kv, d ** -0.5, dtype)
    T = sum(new)
    qp = torch.cat([q, q[:, :1]], 1).cuda()               # a row behind the last request
    out = torch.full_like(qp, 7.0)
    lse = torch.full((hq, T + 1), 7.0, device="cuda")
    P.pisa_paged_attention(qp, dirty[0].cuda(), dirty[1].cuda(), i32(table), i32(U.offsets(new)), i32(kv),
                           out=out, lse=lse)
    P.pisa_device_status()
    U.check(out[:, :T], want["out"], want["bound"], "out")
    none = torch.isinf(want["lse"])
    assert torch.equal(torch.isinf(lse[:, :T]).cpu(), none)
    U.check(lse[:, :T].cpu().masked_fill(none, 0), want["lse"].masked_fill(none, 0), want["lse_bound"] + none, "lse")
    assert (out[:, T:] == 7).all() and (lse[:, T:] == 7).all()


def test_strided_caches_and_scale(P):
    """[pages, page_size, heads, d] caches, two layers' caches in one tensor, [T, H, d] queries."""
    case = ([1, 4, 90], [300, 70, 200], 8, 2, 64, 16, BF)
    new, kv, hq, hkv, d, ps, dtype = case
    for new, kv in (([1, 1], [300, 70]), ([60, 90], [300, 200])):
        q, kc, vc, dirty, table = paged_case(new, kv, hq, hkv, d, ps, dtype)
        both = torch.stack([c.transpose(1, 2) for c in dirty], 1).contiguous().cuda()   # [P, 2, ps, H, d]
        k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
        qs = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        a = P.pisa_paged_attention(qs, k, v, i32(table), i32(U.offsets(new)), i32(kv), scale=0.3)
        want = U.paged(q.double(), kc.double(), vc.double(), table, new, kv, 0.3, dtype)
        U.check(a, want["out"], want["bound"], "out")
        b = P.pisa_paged_attention(q.cuda(), k.contiguous(), v.contiguous(), i32(table), i32(U.offsets(new)),
                                   i32(kv), scale=0.3)
        assert torch.equal(a, b)
    P.pisa_device_status()


@pytest.mark.parametrize("new", [[1, 1], [70, 3]])
def test_bad_pages_and_lengths_are_recorded(P, new):
    """Pages outside the cache, lengths past the table: recorded, never followed."""
    from block_sparse_attention_stats_b200 import _lib
    q, kc, vc, _, table = paged_case(new, [300, 100], 4, 2, 64, 16, BF)
    cache, cu = (kc.cuda(), vc.cuda()), i32(U.offsets(new))
    good = P.pisa_paged_attention(q.cuda(), *cache, i32(table), cu, i32([300, 100]))
    P.pisa_device_status()
    for bad in (-1, -2 ** 31, kc.shape[0], 2 ** 31 - 1):
        t = [list(r) for r in table]
        t[0][3] = bad
        out = P.pisa_paged_attention(q.cuda(), *cache, i32(t), cu, i32([300, 100]))
        with pytest.raises(P.PisaError) as e:
            P.pisa_device_status()
        assert e.value.status == _lib.PISA_ERR_DEVICE
        assert torch.equal(out[:, new[0]:], good[:, new[0]:])     # the other request is right
    for kv in ([-1, 100], [2 ** 31 - 1, 100]):
        P.pisa_paged_attention(q.cuda(), *cache, i32([r[:1] for r in table]), cu, i32(kv))
        with pytest.raises(P.PisaError):
            P.pisa_device_status()
    P.pisa_device_status()


@pytest.mark.parametrize("new", [[1], [200]])
def test_offsets_past_32_bits(P, new):
    """Pages whose elements lie beyond 2^31, in the write and in both kernels."""
    hkv, ps, d, pages = 2, 256, 128, 33000                  # 2.16e9 elements a cache
    kc = torch.zeros(pages, hkv, ps, d, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    m = 300
    table = [[pages - 1, pages - 2]]
    k, v, q = rows(1, hkv, m, d), rows(2, hkv, m, d), rows(3, 4, new[0], d)
    slots = torch.tensor([table[0][j // ps] * ps + j % ps for j in range(m)], device="cuda")
    P.pisa_page_write(k.cuda(), v.cuda(), slots, kc, vc)
    assert torch.equal(kc[pages - 1], k[:, :ps].cuda()) and torch.equal(vc[pages - 2, :, :m - ps], v[:, ps:].cuda())
    out = P.pisa_paged_attention(q.cuda(), kc, vc, i32(table), i32([0, new[0]]), i32([m]))
    P.pisa_device_status()
    cut = [torch.zeros(2, hkv, ps, d) for _ in range(2)]
    for c, x in zip(cut, (k, v)):
        c[1], c[0][:, :m - ps] = x[:, :ps].float(), x[:, ps:].float()
    want = U.paged(q.double(), cut[0].double(), cut[1].double(), [[1, 0]], new, [m], d ** -0.5, BF)
    U.check(out, want["out"], want["bound"], "out")


# ---- plan -------------------------------------------------------------------------------------

def plan_case(rng, b, past, new, ps, spare=3):
    have = [-(-p // ps) for p in past]
    need = [-(-(p + n) // ps) - h for p, n, h in zip(past, new, have)]
    width = max(h + n for h, n in zip(have, need)) + rng.randint(0, 3) or 1
    pages = list(range(sum(have) + sum(need) + spare))
    rng.shuffle(pages)
    table, at = [], 0
    for h in have:
        table.append(pages[at:at + h] + [-1] * (max(width, 1) - h))
        at += h
    return table, pages[at:]


def run_plan(P, past, new, table, free, num_free, ps, T):
    t = i32(table)
    r = P.pisa_page_plan(i32(past), i32(new), t, i32(free) if free else i32([0])[:0], i32([num_free]), ps, T)
    return t, r


def same_plan(t, r, want, table):
    assert t.tolist() == table
    assert r["slots"].tolist() == want["slots"]
    assert r["cu_seqlens"].tolist() == want["cu"]
    assert r["kv_lens"].tolist() == want["kv_lens"]
    assert r["num_free"].tolist() == [want["num_free"]]


@pytest.mark.parametrize("b,most_past,most_new,ps", [(1, 0, 1, 16), (1, 40, 0, 16), (3, 50, 40, 16), (31, 0, 70, 32),
                                                     (513, 300, 3, 16), (700, 90, 1, 128), (2049, 20, 5, 256)])
def test_plan(P, b, most_past, most_new, ps):
    rng = random.Random(b)
    past = [rng.randint(0, most_past) for _ in range(b)]
    new = [rng.randint(0, most_new) for _ in range(b)]
    table, free = plan_case(rng, b, past, new, ps)
    T = sum(new) + rng.randint(0, 5)
    want_table = [list(r) for r in table]
    want = U.plan(past, new, want_table, free, len(free), ps, T)
    assert want["ok"]
    t, r = run_plan(P, past, new, table, free, len(free), ps, T)
    P.pisa_device_status()
    same_plan(t, r, want, want_table)
    # again on the same tables: the same entries
    r2 = P.pisa_page_plan(i32(past), i32(new), t, i32(free), i32([len(free)]), ps, T)
    same_plan(t, r2, want, want_table)


def test_plan_takes_all_or_nothing(P):
    past, new, ps = [30, 0, 100], [40, 5, 1], 16
    table, free = plan_case(random.Random(1), 3, past, new, ps, spare=0)
    T = sum(new)
    ok = U.plan(past, new, [list(r) for r in table], free, len(free), ps, T)
    assert ok["ok"] and ok["num_free"] == 0
    refused = [
        (past, new, table, free, len(free) - 1, ps, T),                  # one page short
        (past, new, table, free, len(free), ps, T - 1),                  # more tokens than slots
        (past, [40, -1, 1], table, free, len(free), ps, T),
        ([30, -7, 100], new, table, free, len(free), ps, T),
        (past, new, [r[:6] for r in table], free, len(free), ps, T),     # the third outgrows the table
        ([2 ** 31 - 1, 0, 0], [1, 0, 0], table, free, len(free), ps, T),
        (past, new, table, free, len(free) + 1, ps, T),                  # a count past the list
        (past, new, table, free, -1, ps, T),
    ]
    for args in refused:
        want_table = [list(r) for r in args[2]]
        t, r = run_plan(P, *args)
        with pytest.raises(P.PisaError):
            P.pisa_device_status()
        assert t.tolist() == want_table
        assert r["slots"].tolist() == [-1] * args[6] and r["cu_seqlens"].tolist() == [0] * 4
        assert r["kv_lens"].tolist() == list(args[0]) and r["num_free"].tolist() == [args[4]]
    t, r = run_plan(P, past, new, table, free, len(free), ps, T)
    P.pisa_device_status()
    assert r["num_free"].tolist() == [0]


# ---- write ------------------------------------------------------------------------------------

@pytest.mark.parametrize("t,pages,h,d,ps,dtype", [(1, 1, 1, 64, 16, BF), (33, 5, 3, 128, 16, HF),
                                                  (700, 30, 8, 64, 32, BF), (257, 4, 2, 128, 256, BF)])
def test_write(P, t, pages, h, d, ps, dtype):
    rng = random.Random(t)
    slots = rng.sample(range(pages * ps), t)
    for i in rng.sample(range(t), t // 7):
        slots[i] = -1
    k, v = rows(1, h, t, d, dtype=dtype), rows(2, h, t, d, dtype=dtype)
    kc, vc = (rows(i, pages, h, ps, d, dtype=dtype) for i in (3, 4))
    got = [kc.clone().cuda(), vc.clone().cuda()]
    # [T, H, d] sources, and a cache of another layout
    strided = [x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (kc, vc)]
    s = torch.tensor(slots, device="cuda")
    P.pisa_page_write(k.cuda(), v.cuda(), s, *got)
    P.pisa_page_write(*(x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in (k, v)), s, *strided)
    P.pisa_device_status()
    for c, x in ((kc, k), (vc, v)):
        for i, at in enumerate(slots):
            if at >= 0:
                c[at // ps, :, at % ps] = x[:, i]
    for c, a, b in zip((kc, vc), got, strided):
        assert torch.equal(a.cpu(), c) and torch.equal(b.cpu(), c)


def test_write_leaves_out_bad_slots(P):
    k = rows(1, 2, 4, 64).cuda()
    kc = torch.zeros(3, 2, 16, 64, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    P.pisa_page_write(k, k, torch.tensor([5, 48, 2 ** 40, -9], device="cuda"), kc, vc)
    with pytest.raises(P.PisaError):
        P.pisa_device_status()
    want = torch.zeros_like(kc)
    want[0, :, 5] = k[:, 0]
    assert torch.equal(kc, want) and torch.equal(vc, want)


# ---- the whole step ------------------------------------------------------------------------------

@pytest.mark.parametrize("ps,dtype,hq,hkv,d", [(16, BF, 4, 2, 64), (64, HF, 6, 2, 128), (128, BF, 8, 1, 128)])
def test_server_of_several_steps(P, ps, dtype, hq, hkv, d):
    """Prompts in chunks, then single tokens, requests joining in between: every step's output is
    the one of attention over all positions so far."""
    b, total = 4, 90
    free = i32(list(range(total)))
    num_free = i32([total])
    table = torch.full((b, 40), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((total, hkv, ps, d), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    past = [0] * b
    seen = [[torch.zeros(hkv, 0, d, dtype=dtype) for _ in range(2)] for _ in range(b)]
    for step, new in enumerate([[70, 0, 5, 0], [130, 1, 1, 0], [1, 40, 1, 200], [1, 1, 1, 1], [1, 1, 0, 1]]):
        T = sum(new) + 2
        q, k, v = rows(10 * step, hq, T, d, dtype=dtype), rows(10 * step + 1, hkv, T, d, dtype=dtype), \
            rows(10 * step + 2, hkv, T, d, dtype=dtype)
        out, plan = P.pisa_paged_step(q.cuda(), k.cuda(), v.cuda(), kc, vc, i32(past), i32(new), table, free, num_free,
                                      out=torch.full((hq, T, d), 7.0, dtype=dtype, device="cuda"))
        P.pisa_device_status()
        num_free = plan["num_free"]
        for j, (a, n) in enumerate(zip(U.offsets(new), new)):
            seen[j] = [torch.cat([s, x[:, a:a + n]], 1) for s, x in zip(seen[j], (k, v))]
            past[j] += n
            for h in range(hq if n else 0):
                _, want, bound, _, _, _ = U.attend(
                    q[h, a:a + n].double(), *(s[h // (hq // hkv)].double() for s in seen[j]),
                    torch.arange(past[j] - n, past[j]), d ** -0.5, U.half_step(dtype))
                U.check(out[h, a:a + n], want, bound, f"step {step} request {j} head {h}")
        assert plan["kv_lens"].tolist() == past
        assert (out[:, sum(new):] == 7).all()
    assert num_free.tolist() == [total - sum(-(-p // ps) for p in past)]


def test_a_step_that_does_not_fit_changes_nothing(P):
    hkv, ps, d = 2, 16, 64
    q, k = rows(1, 4, 40, d).cuda(), rows(2, hkv, 40, d).cuda()
    kc = torch.zeros(5, hkv, ps, d, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    P.pisa_paged_step(q, k, k, kc, vc, i32([0, 0]), i32([20, 20]), table, i32([0, 1, 2]), i32([3]), out=out)
    with pytest.raises(P.PisaError):
        P.pisa_device_status()
    assert (out == 7).all() and (kc == 0).all() and (vc == 0).all() and (table == -1).all()


def test_a_captured_step_follows_the_lengths(P):
    """One graph of a decode step serves every length; its counters carry on from replay to replay."""
    b, hq, hkv, ps, d, total = 3, 8, 2, 16, 64, 60
    kc, vc = (torch.zeros(total, hkv, ps, d, dtype=BF, device="cuda") for _ in range(2))
    table = torch.full((b, 20), -1, dtype=torch.int32, device="cuda")
    past, new, free, num_free = i32([0] * b), i32([1] * b), i32(list(range(total))), i32([total])
    q, k, v = (torch.zeros(h, b, d, dtype=BF, device="cuda") for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)
    lib = P._lib.load()
    ws = torch.empty(lib.pisa_paged_attention_workspace_bytes(hq, hkv, d), dtype=torch.uint8, device="cuda")
    plan = dict(slots=torch.empty(b, dtype=torch.int64, device="cuda"), cu_seqlens=i32([0] * (b + 1)),
                kv_lens=i32([0] * b), num_free=i32([0]))

    def step():
        P.pisa_paged_step(q, k, v, kc, vc, past, new, table, free, num_free, out=out, plan=plan, workspace=ws)
        past.copy_(plan["kv_lens"])
        num_free.copy_(plan["num_free"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    past.zero_()
    num_free.fill_(total)
    table.fill_(-1)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    past.zero_()
    num_free.fill_(total)
    table.fill_(-1)
    seen = [[], []]
    for i in range(40):
        x = [rows(100 + 3 * i + j, h, b, d) for j, h in enumerate((hq, hkv, hkv))]
        for dst, src in zip((q, k, v), x):
            dst.copy_(src)
        gr.replay()
        for s, y in zip(seen, x[1:]):
            s.append(y)
        if i in (0, 15, 16, 39):
            for j in range(b):
                ks, vs = (torch.stack([y[:, j] for y in s], 1).double() for s in seen)
                for h in range(hq):
                    _, want, bound, _, _, _ = U.attend(x[0][h, j:j + 1].double(), ks[h // 4], vs[h // 4],
                                                       torch.tensor([i]), d ** -0.5, U.half_step(BF))
                    U.check(out[h, j:j + 1], want, bound, f"step {i} request {j} head {h}")
    P.pisa_device_status()
    assert past.tolist() == [40] * b
    del gr


def test_paged_repeats_bitwise_on_streams(P):
    for new in ([1, 1, 1], [60, 1, 30]):
        kv = [5000, 700, 33]
        q, kc, vc, _, table = paged_case(new, kv, 8, 2, 128, 16, BF)
        args = (q.cuda(), kc.cuda(), vc.cuda(), i32(table), i32(U.offsets(new)), i32(kv))
        want = P.pisa_paged_attention(*args)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = [P.pisa_paged_attention(*args, stream=s) for _ in range(5) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in got)
    P.pisa_device_status()


@pytest.mark.parametrize("seed", range(10))
def test_random_requests(P, seed):
    rng = random.Random(seed)
    d, ps, dtype = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice([BF, HF])
    hkv = rng.choice([1, 2, 5])
    hq = hkv * rng.choice([1, 2, 3, 7, 16])
    most = rng.choice([1, 4, 30, 200])
    kv = [rng.choice([1, rng.randint(1, 40), rng.randint(1, 1500)]) for _ in range(rng.randint(1, 7))]
    new = [rng.choice([0, 1, min(m, rng.randint(1, most))]) for m in kv]
    new[rng.randrange(len(new))] = 1
    q, kc, vc, dirty, table = paged_case(new, kv, hq, hkv, d, ps, dtype, seed)
    want = U.paged(q.double(), kc.double(), vc.double(), table, new, kv, d ** -0.5, dtype)
    lse = torch.zeros(hq, sum(new), device="cuda")
    out = P.pisa_paged_attention(q.cuda(), dirty[0].cuda(), dirty[1].cuda(), i32(table), i32(U.offsets(new)), i32(kv),
                                 lse=lse)
    P.pisa_device_status()
    U.check(out, want["out"], want["bound"], "out")
    U.check(lse, want["lse"], want["lse_bound"], "lse")


def test_a_prompt_in_the_cache_is_the_prompt(P):
    """The same prompts through the packed call and through pages: the same numbers to rounding."""
    new, hq, hkv, d, ps = [300, 45, 129], 6, 2, 128, 32
    T = sum(new)
    q, k, v = rows(1, hq, T, d), rows(2, hkv, T, d), rows(3, hkv, T, d)
    a = P.pisa_varlen_attention(q.cuda(), k.cuda(), v.cuda(), i32(U.offsets(new)))
    table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(40, hkv, ps, d, dtype=BF, device="cuda") for _ in range(2))
    b, _ = P.pisa_paged_step(q.cuda(), k.cuda(), v.cuda(), kc, vc, i32([0] * 3), i32(new), table,
                             i32(list(range(40))), i32([40]))
    P.pisa_device_status()
    want = U.varlen(q.double(), k.double(), v.double(), new, True, d ** -0.5, BF)
    U.check(a, want["out"], want["bound"], "packed")
    U.check(b, want["out"], want["bound"], "paged")
