"""Attention over packed prompts and over a paged key/value cache: what is measured.

Four operators, reached through the package's public calls:

- `varlen_attention` / `pisa_varlen_attention`: softmax attention of every sequence of a packed
  batch over itself, causal or not, grouped key/value heads; with its gradients.
- `pisa_paged_attention`: the newest tokens of every request over that request's pages of a
  key/value cache (one token each when decoding, a chunk of a prompt otherwise).
- `pisa_page_plan`: block tables, slots and offsets of one step from the requests' lengths.
- `pisa_page_write`: new keys and values into their slots of the cache.

Packed tensors are [heads, tokens, d], caches [pages, heads, page_size, d]; lengths, offsets and
tables are int32, slots int64.  Rows of packed tensors behind the last sequence keep what they held.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _ints(text):
    return [int(x) for x in str(text).split(",")]


# ---- the cases ------------------------------------------------------------------------------------


def listed():
    return [
        # a handful of short prompts that arrive together, one of them empty, padding behind them
        dict(name="prefill_short", op="prefill", lens="5,64,1,130,17,0,200", pad=9, hq=8, hkv=2, d=64,
             dtype="f16", causal=True),
        # long prompts packed with a short one
        dict(name="prefill_long", op="prefill", lens="12000,700,4608", pad=0, hq=24, hkv=8, d=128,
             dtype="bf16", causal=True),
        # training on a few short documents, three query heads to a key head
        dict(name="train_short", op="train", lens="64,1,37,300,129", pad=13, hq=6, hkv=2, d=64,
             dtype="bf16", causal=True),
        # training on long documents packed into one row
        dict(name="train_long", op="train", lens="8192,4608,1500", pad=84, hq=24, hkv=8, d=128,
             dtype="bf16", causal=True),
        # one user, one new token: latency
        dict(name="decode_one", op="paged", new="1", kv="777", hq=8, hkv=8, d=64, page=16, dtype="bf16"),
        # a batch of requests of very different lengths, one new token each
        dict(name="decode_batch", op="paged", new=",".join(["1"] * 48),
             kv=",".join(str(1 + (i * 2657) % 8011) for i in range(48)), hq=40, hkv=8, d=128, page=64,
             dtype="bf16"),
        # two very long contexts, eight query heads to a key head
        dict(name="decode_long", op="paged", new="1,1", kv="131072,90001", hq=32, hkv=4, d=128, page=128,
             dtype="f16"),
        # chunks of prompts beside requests that decode
        dict(name="chunk_mixed", op="paged", new="1,1,700,1,64,257", kv="4000,19,9000,20000,64,1157", hq=24,
             hkv=8, d=128, page=16, dtype="bf16"),
        # one step's bookkeeping: a few requests, and a full server
        dict(name="plan_small", op="plan", b=7, low=0, high=40, past=500, page=16, width=64, pick=3),
        dict(name="plan_large", op="plan", b=1500, low=1, high=90, past=30000, page=64, width=512, pick=5),
        # the step's keys and values into the cache: a few tokens, and a whole batch of prompts
        dict(name="write_small", op="write", t=33, pages=40, hkv=8, d=128, page=16, dtype="bf16", skip=3),
        dict(name="write_large", op="write", t=65000, pages=1300, hkv=8, d=128, page=64, dtype="bf16",
             skip=100),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


_HEADS = [(1, 1), (4, 4), (6, 2), (8, 1), (8, 2), (12, 4), (16, 16), (24, 8), (32, 4), (40, 8), (14, 2)]


def draw(rng):
    op = rng.choice(["prefill", "train", "paged", "paged", "plan", "write"])
    hq, hkv = rng.choice(_HEADS)
    d = rng.choice([64, 128])
    if op in ("prefill", "train"):
        most = 4.0e9 if op == "train" else 9.0e9  # padded score elements of the plain form
        n = rng.randint(1, 8)
        longest = _log_int(rng, 2, 8000)
        lens = [rng.choice([0, 1, _log_int(rng, 1, longest), longest]) for _ in range(n)]
        lens[rng.randrange(n)] = longest
        while n * hq * longest * longest > most:
            longest = longest * 2 // 3 + 1
            lens = [min(x, longest) for x in lens]
        return dict(op=op, lens=",".join(map(str, lens)), pad=rng.choice([0, 0, 1, 31]), hq=hq, hkv=hkv, d=d,
                    dtype="bf16" if op == "train" else rng.choice(["bf16", "f16"]),
                    causal=rng.random() < 0.8)
    if op == "paged":
        page = rng.choice([16, 32, 64, 128])
        b = _log_int(rng, 1, 64)
        most = _log_int(rng, 16, 60000)
        kv = [max(1, _log_int(rng, 1, most)) for _ in range(b)]
        chunk = rng.choice([1, 1, 4, 600])
        new = [rng.choice([1, min(k, chunk), min(k, _log_int(rng, 1, chunk))]) for k in kv]
        while b * max(kv) * hkv * d > 1.5e9 or b * max(kv) * hq * max(new) > 3.0e9:
            kv = [k * 2 // 3 + 1 for k in kv]
            new = [min(x, k) for x, k in zip(new, kv)]
        return dict(op=op, new=",".join(map(str, new)), kv=",".join(map(str, kv)), hq=hq, hkv=hkv, d=d,
                    page=page, dtype=rng.choice(["bf16", "f16"]))
    if op == "plan":
        page = rng.choice([16, 32, 64, 128])
        past = _log_int(rng, 1, 20000)
        high = _log_int(rng, 1, 90)
        return dict(op=op, b=_log_int(rng, 1, 1500), low=rng.choice([0, 1]), high=high, past=past, page=page,
                    width=(past + high) // page + 1 + rng.randint(0, 7), pick=rng.randrange(1 << 20))
    page = rng.choice([16, 32, 64, 128])
    t = _log_int(rng, 1, 60000)
    return dict(op=op, t=t, pages=t // page + 1 + rng.randint(0, 30), hkv=min(hkv, 8), d=d, page=page,
                dtype=rng.choice(["bf16", "f16"]), skip=min(t, rng.choice([0, 0, 1, 9])))


# ---- what a user's program has in hand ------------------------------------------------------------


def _plan_lens(case):
    pick = random.Random(case["pick"])
    past = [pick.randint(0, case["past"]) for _ in range(case["b"])]
    new = [pick.randint(case["low"], case["high"]) for _ in range(case["b"])]
    return past, new


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    i32 = dict(dtype=torch.int32, device="cuda")

    def rows(heads, n, dtype, scale=1.0):
        x = torch.randn(heads, n, case["d"], generator=g, device="cuda")
        return (x * scale).to(_DT[dtype])

    s = dict(op=op, case=dict(case))
    if op in ("prefill", "train"):
        lens = _ints(case["lens"])
        t = sum(lens) + case["pad"]
        s.update(lens=lens, cu=torch.tensor(_offsets(lens), **i32), causal=bool(case["causal"]))
        # queries a little larger than unit: some rows attend broadly, others to a few keys
        s["q"], s["k"], s["v"] = (rows(case["hq"], t, case["dtype"], 1.5), rows(case["hkv"], t, case["dtype"]),
                                  rows(case["hkv"], t, case["dtype"]))
        if op == "train":
            s["dout"] = rows(case["hq"], t, case["dtype"])
            for x in "qkv":
                s[x].requires_grad_()
        else:
            s["out"] = torch.zeros_like(s["q"])
    elif op == "paged":
        new, kv = _ints(case["new"]), _ints(case["kv"])
        page = case["page"]
        need = [-(-n // page) for n in kv]
        total = sum(need) + 3
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(kv), max(need) + 2), -1, **i32)
        b = torch.repeat_interleave(torch.arange(len(kv), device="cuda"), torch.tensor(need, device="cuda"))
        first = torch.tensor(_offsets(need)[:-1], device="cuda")
        at = torch.arange(sum(need), device="cuda")
        table[b, at - first[b]] = order[: sum(need)]
        for x in ("kc", "vc"):
            c = torch.randn(total, case["hkv"] * page, case["d"], generator=g, device="cuda")
            s[x] = c.to(_DT[case["dtype"]]).view(total, case["hkv"], page, case["d"])
        s.update(q=rows(case["hq"], sum(new), case["dtype"], 1.5), table=table, new=new, kv=kv,
                 cu=torch.tensor(_offsets(new), **i32), kv_lens=torch.tensor(kv, **i32))
        s["out"] = torch.zeros_like(s["q"])
    elif op == "plan":
        past, new = _plan_lens(case)
        page = case["page"]
        have = torch.tensor([-(-n // page) for n in past], device="cuda")
        free = sum(-(-(p + n) // page) - -(-p // page) for p, n in zip(past, new)) + 5
        ids = torch.randperm(int(have.sum()) + free, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["b"], case["width"]), -1, **i32)
        col = torch.arange(case["width"], device="cuda")
        held = col < have[:, None]
        table[held] = ids[free:]
        s.update(past=torch.tensor(past, **i32), new=torch.tensor(new, **i32), table=table,
                 free=ids[:free].clone(), num_free=torch.tensor([free], **i32), page=page,
                 t=sum(new) + 11, total=sum(new))
    else:
        t, page, hkv = case["t"], case["page"], case["hkv"]
        slots = torch.randperm(case["pages"] * page, generator=g, device="cuda")[:t].contiguous()
        if case["skip"]:
            slots[torch.randperm(t, generator=g, device="cuda")[: case["skip"]]] = -1
        s.update(k=rows(hkv, t, case["dtype"]), v=rows(hkv, t, case["dtype"]), slots=slots)
        for x in ("kc", "vc"):
            c = torch.randn(case["pages"], hkv * page, case["d"], generator=g, device="cuda")
            s[x] = c.to(_DT[case["dtype"]]).view(case["pages"], hkv, page, case["d"])
    return s


# ---- one pass -------------------------------------------------------------------------------------


def run(s):
    op = s["op"]
    if op == "prefill":
        return _own_prefill(s) if own else _plain_prefill(s)
    if op == "train":
        return _own_train(s) if own else _plain_train(s)
    if op == "paged":
        return _own_paged(s) if own else _plain_paged(s)
    if op == "plan":
        return _own_plan(s) if own else _plain_plan(s)
    return _own_write(s) if own else _plain_write(s)


def _own_prefill(s):
    import block_sparse_attention_stats_b200 as pisa

    return pisa.pisa_varlen_attention(s["q"], s["k"], s["v"], s["cu"], causal=s["causal"], out=s["out"])


def _own_train(s):
    import block_sparse_attention_stats_b200 as pisa

    out = pisa.varlen_attention(s["q"], s["k"], s["v"], s["cu"], causal=s["causal"])
    dq, dk, dv = torch.autograd.grad(out, (s["q"], s["k"], s["v"]), s["dout"])
    return dict(out=out.detach(), dq=dq, dk=dk, dv=dv)


def _own_paged(s):
    import block_sparse_attention_stats_b200 as pisa

    return pisa.pisa_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv_lens"], out=s["out"])


def _own_plan(s):
    import block_sparse_attention_stats_b200 as pisa

    r = pisa.pisa_page_plan(s["past"], s["new"], s["table"], s["free"], s["num_free"], s["page"], s["t"])
    return dict(table=s["table"], slots=r["slots"], cu=r["cu_seqlens"], kv_lens=r["kv_lens"],
                num_free=r["num_free"])


def _own_write(s):
    import block_sparse_attention_stats_b200 as pisa

    pisa.pisa_page_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
    return dict(k=s["kc"], v=s["vc"])


# ---- the plain forms ------------------------------------------------------------------------------


def _padded(s):
    """Row of the packed tensors for every (sequence, position), and which positions exist."""
    lens = torch.tensor(s["lens"], device="cuda")
    pos = torch.arange(max(1, max(s["lens"])), device="cuda")
    there = pos < lens[:, None]
    return (s["cu"][:-1, None] + pos) * there, there, pos


def _heads(x, at, hkv):
    """[heads, tokens, d] as float32 [sequences, hkv, heads / hkv, positions, d]."""
    x = x.detach().float()[:, at].movedim(0, 1)
    return x.unflatten(1, (hkv, -1))


def _probabilities(z):
    """Softmax of the last axis, in place; rows of -inf alone give zeros."""
    m = z.amax(-1, keepdim=True)
    z.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    return z.div_(z.sum(-1, keepdim=True).clamp_min(1e-38))


def _softmax_of(s):
    c = s["case"]
    at, there, pos = _padded(s)
    q, k, v = (_heads(s[x], at, c["hkv"]) for x in "qkv")
    seen = there[:, None, :] & there[:, :, None]
    if s["causal"]:
        seen = seen & (pos <= pos[:, None])
    z = (q / math.sqrt(c["d"])) @ k.transpose(-1, -2)
    z.masked_fill_(~seen[:, None, None], -math.inf)
    return at, there, q, k, v, _probabilities(z)


def _packed(x, like, at, there, dtype):
    """[sequences, hkv, group, positions, d] back into packed rows, zeros where no sequence is."""
    out = torch.zeros(like.shape, dtype=dtype, device="cuda")
    out[:, at[there]] = x.flatten(1, 2).movedim(0, 1)[:, there].to(dtype)
    return out


def _plain_prefill(s):
    at, there, q, k, v, p = _softmax_of(s)
    return _packed(p @ v, s["q"], at, there, s["q"].dtype)


def _plain_train(s):
    at, there, q, k, v, p = _softmax_of(s)
    scale = 1 / math.sqrt(s["case"]["d"])
    out = p @ v
    dout = _heads(s["dout"], at, s["case"]["hkv"]) * there[:, None, None, :, None]
    dv = (p.transpose(-1, -2) @ dout).sum(2, keepdim=True)
    dp = dout @ v.transpose(-1, -2)
    dz = dp.sub_((dout * out).sum(-1, keepdim=True)).mul_(p)
    dq = (dz @ k) * scale
    dk = (dz.transpose(-1, -2) @ q).sum(2, keepdim=True) * scale
    t = s["q"].dtype
    return dict(out=_packed(out, s["q"], at, there, t), dq=_packed(dq, s["q"], at, there, t),
                dk=_packed(dk, s["k"], at, there, t), dv=_packed(dv, s["v"], at, there, t))


def _plain_paged(s):
    c = s["case"]
    kv, new = s["kv_lens"], s["cu"][1:] - s["cu"][:-1]
    pages = s["table"][:, : -(-max(s["kv"]) // c["page"])].clamp_min(0)
    # [requests, pages, hkv, page, d] -> [requests, hkv, 1, keys, d]
    k, v = (s[x][pages].float().movedim(2, 1).flatten(2, 3).unsqueeze(2) for x in ("kc", "vc"))
    row = torch.arange(max(s["new"]), device="cuda")
    there = row < new[:, None]
    at = (s["cu"][:-1, None] + row) * there
    q = _heads(s["q"], at, c["hkv"])
    last = (kv - new)[:, None] + row  # position of each new token in its request
    key = torch.arange(k.shape[3], device="cuda")
    seen = (key <= last[..., None]) & there[..., None]
    v = v * (key < kv[:, None])[:, None, None, :, None]
    z = (q / math.sqrt(c["d"])) @ k.transpose(-1, -2)
    z.masked_fill_(~seen[:, None, None], -math.inf)
    return _packed(_probabilities(z) @ v, s["q"], at, there, s["q"].dtype)


def _plain_plan(s):
    past, new, page, table = s["past"].long(), s["new"].long(), s["page"], s["table"]
    have, want = (past + page - 1) // page, (past + new + page - 1) // page
    before = torch.cumsum(want - have, 0) - (want - have)
    col = torch.arange(table.shape[1], device="cuda")
    fresh = (col >= have[:, None]) & (col < want[:, None])
    nth = before[:, None] + col - have[:, None]
    taken = s["free"][(s["num_free"].long() - 1 - nth).clamp(0, s["free"].numel() - 1)]
    table.copy_(torch.where(fresh, taken, table))
    end = torch.cumsum(new, 0)
    row = torch.arange(s["t"], device="cuda")
    b = torch.searchsorted(end, row, right=True)
    inside = b < past.numel()
    b = b.clamp_max(past.numel() - 1)
    pos = past[b] + row - (end - new)[b]
    slots = table[b, (pos // page).clamp_max(table.shape[1] - 1)].long() * page + pos % page
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return dict(table=table, slots=torch.where(inside, slots, -1), cu=torch.cat([zero, end]).int(),
                kv_lens=(past + new).int(), num_free=(s["num_free"] - (want - have).sum()).int())


def _plain_write(s):
    page = s["case"]["page"]
    here = s["slots"] >= 0
    slots = s["slots"][here]
    for x, c in (("k", "kc"), ("v", "vc")):
        s[c][slots // page, :, slots % page] = s[x][:, here].movedim(0, 1)
    return dict(k=s["kc"], v=s["vc"])


# ---- in 64 bits, from the definitions -------------------------------------------------------------


def _attend64(q, k, v, last):
    """One head in float64: row i of q over keys 0 .. last[i]; (probabilities, output)."""
    z = q @ k.T * q.shape[-1] ** -0.5
    z = z.masked_fill(torch.arange(k.shape[0], device=q.device)[None] > last[:, None], -math.inf)
    p = torch.softmax(z, -1)
    return p, p @ v


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("prefill", "train"):
        lens, group = _ints(case["lens"]), case["hq"] // case["hkv"]
        q, k, v = (s[x].detach().double() for x in "qkv")
        out, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for a, n in zip(_offsets(lens), lens):
            if n == 0:
                continue
            r = slice(a, a + n)
            last = torch.arange(n, device="cuda") if case["causal"] else torch.full((n,), n - 1, device="cuda")
            for h in range(case["hq"]):
                j = h // group
                p, o = _attend64(q[h, r], k[j, r], v[j, r], last)
                out[h, r] = o
                if op == "train":
                    go = s["dout"][h, r].double()
                    dv[j, r] += p.T @ go
                    dp = go @ v[j, r].T
                    dz = p * (dp - (p * dp).sum(-1, keepdim=True)) * case["d"] ** -0.5
                    dq[h, r] = dz @ k[j, r]
                    dk[j, r] += dz.T @ q[h, r]
                    del dp, dz
                del p
        return out if op == "prefill" else dict(out=out, dq=dq, dk=dk, dv=dv)
    if op == "paged":
        new, kv, page = _ints(case["new"]), _ints(case["kv"]), case["page"]
        group = case["hq"] // case["hkv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, (n, m) in enumerate(zip(new, kv)):
            a = sum(new[:b])
            ids = s["table"][b, : -(-m // page)].long()
            last = torch.arange(m - n, m, device="cuda")
            for h in range(case["hq"]):
                k, v = (s[x][ids, h // group].reshape(-1, case["d"])[:m].double() for x in ("kc", "vc"))
                out[h, a:a + n] = _attend64(s["q"][h, a:a + n].double(), k, v, last)[1]
        return out
    if op == "plan":
        return None
    where = s["slots"].tolist()
    at = [i for i, x in enumerate(where) if x >= 0]
    slots = torch.tensor([where[i] for i in at], device="cuda", dtype=torch.int64)
    at = torch.tensor(at, device="cuda", dtype=torch.int64)
    out = {}
    for x, c in (("k", "kc"), ("v", "vc")):
        cache = s[c].double().movedim(1, 2).reshape(-1, case["hkv"], case["d"])
        cache[slots] = s[x].double()[:, at].movedim(0, 1)
        out[x] = cache.view(case["pages"], case["page"], case["hkv"], case["d"]).movedim(2, 1).contiguous()
    return out


# ---- what a pass cannot do without ----------------------------------------------------------------


def work(case):
    op = case["op"]
    if op in ("prefill", "train"):
        lens, d = _ints(case["lens"]), case["d"]
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens) * case["hq"]
        rows = sum(lens)
        q, kv = rows * case["hq"] * d * 2, rows * case["hkv"] * d * 2
        if op == "prefill":
            return {"bytes": 2 * q + 2 * kv, "flops": 4 * d * pairs}
        # q, k, v and dout in; out, dq, dk and dv out.  Two products forward, five backward
        return {"bytes": 4 * q + 4 * kv, "flops": 14 * d * pairs}
    if op == "paged":
        new, kv, d = _ints(case["new"]), _ints(case["kv"]), case["d"]
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(new, kv)) * case["hq"]
        tables = sum(-(-m // case["page"]) for m in kv) * 4
        return {"bytes": 4 * sum(kv) * case["hkv"] * d + 4 * sum(new) * case["hq"] * d + tables,
                "flops": 4 * d * pairs}
    if op == "plan":
        past, new = _plan_lens(case)
        page = case["page"]
        fresh = sum(-(-(p + n) // page) - -(-p // page) for p, n in zip(past, new))
        # lengths in, offsets and lengths out, new pages read and entered, slots out
        return {"bytes": 16 * len(past) + 8 * fresh + 8 * (sum(new) + 11), "flops": 0}
    rows = case["t"] - case["skip"]
    return {"bytes": 8 * rows * case["hkv"] * case["d"] + 8 * case["t"], "flops": 0}
