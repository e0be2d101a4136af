"""Cases, plain forms and exact values of the paged memory's operators.

A paged memory keeps each sequence's key and value rows in pages of a pool
instead of in one buffer per sequence.  Pool: k_pages, v_pages
[n_pages, H, page_rows, D].  Book (int32): table [slots, max_pages] (the pages
of a slot, oldest rows first, -1 past its last page), start [slots] (dead rows
at the head of the slot's first page), rows [slots] (live rows), refs
[n_pages] (how often a page stands in the table; 0: free).

  attend   txl_relattn_forward_paged: the new tokens of a ragged batch over
           their slots' rows, their own among them, with the four-term
           relative score; one token per sequence up to whole segments
  roll     txl_pages_reserve, txl_pages_append, txl_pages_free: the new rows
           written behind the old ones and the oldest dropped
  beams    txl_pages_fork, then a roll that writes into shared pages and
           frees the copies
  compact  txl_pages_compact, txl_pages_copy: the live pages moved to the
           front of the pool

Where `own` is false, run() computes them with elementary torch operations.
"""
import random

import torch

own = False


def listed():
    return [
        # A single user's stream, one token at a time: the smallest call, all latency.
        dict(name="decode one", op="attend", dtype="bf16", H=8, D=64, page=64, seqs=1, new_lo=1, new_hi=1, mem_lo=512, mem_hi=512, pattern=1),
        # A serving batch of streams of unlike age, one token each: bound by reading the pages.
        dict(name="decode batch", op="attend", dtype="bf16", H=16, D=64, page=64, seqs=64, new_lo=1, new_hi=1, mem_lo=300, mem_hi=4500, pattern=2),
        # Long memories, the wider head, small pages.
        dict(name="decode long", op="attend", dtype="bf16", H=8, D=128, page=32, seqs=48, new_lo=1, new_hi=1, mem_lo=1600, mem_hi=8100, pattern=3),
        # The base evaluation's segments (22 sequences, 512 tokens over 512 rows of memory), paged.
        dict(name="chunk base", op="attend", dtype="bf16", H=8, D=64, page=64, seqs=22, new_lo=512, new_hi=512, mem_lo=512, mem_hi=512, pattern=4),
        # The wide evaluation's segments (8 sequences, 768 tokens over 768 rows, D = 128), paged.
        dict(name="chunk wide", op="attend", dtype="bf16", H=8, D=128, page=128, seqs=8, new_lo=768, new_hi=768, mem_lo=768, mem_hi=768, pattern=5),
        # A batch that mixes prompts of odd lengths with streams that bring a token, over memories from none to long.
        dict(name="chunk mixed", op="attend", dtype="bf16", H=8, D=64, page=16, seqs=20, new_lo=1, new_hi=601, mem_lo=0, mem_hi=2999, pattern=6),
        # The exact type, with a head size off the tensor cores' path.
        dict(name="chunk float32", op="attend", dtype="f32", H=4, D=40, page=16, seqs=5, new_lo=1, new_hi=130, mem_lo=0, mem_hi=700, pattern=7),
        # One token each into the memories of a serving batch, the oldest row dropped: latency.
        dict(name="roll tokens", op="roll", dtype="bf16", H=16, D=64, page=64, seqs=64, new_lo=1, new_hi=1, mem_lo=1600, mem_hi=1600, pattern=8),
        # A whole segment of the base evaluation into the memories.
        dict(name="roll segments", op="roll", dtype="bf16", H=8, D=64, page=64, seqs=22, new_lo=512, new_hi=512, mem_lo=512, mem_hi=512, pattern=9),
        # Beam search: every sequence forked three times, a token written to each branch, the branches freed.
        dict(name="beams", op="beams", dtype="bf16", H=16, D=64, page=64, seqs=32, beams=3, mem_lo=200, mem_hi=1600, pattern=10),
        # A small pool put in order.
        dict(name="compact small", op="compact", dtype="bf16", H=4, D=64, page=16, pages=600, live=0.5, pattern=11),
        # The pool of a serving batch after most of its sequences have ended.
        dict(name="compact large", op="compact", dtype="bf16", H=16, D=64, page=64, pages=9000, live=0.4, pattern=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "roll", "roll", "beams", "compact"])
    case = dict(op=op, dtype="f32" if rng.random() < 0.2 else "bf16", H=rng.randint(1, 16), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), pattern=rng.randrange(1 << 20))
    if case["dtype"] == "f32":
        case.update(D=rng.randint(1, 100), H=rng.randint(1, 6))
    if op == "compact":
        case.update(pages=_log(rng, 40, 4000), live=round(rng.uniform(0.1, 0.9), 2))
    elif op == "beams":
        case.update(seqs=_log(rng, 1, 32), beams=rng.randint(1, 4), mem_lo=rng.randint(1, 100), mem_hi=_log(rng, 100, 1500))
    elif op == "roll":
        new = _log(rng, 1, 600)
        case.update(seqs=_log(rng, 1, 64), new_lo=rng.randint(1, new), new_hi=new, mem_lo=1, mem_hi=_log(rng, 1, 1600))
        case["seqs"] = min(case["seqs"], max(1, 16000 // new))
    elif case["dtype"] == "f32":
        case.update(seqs=_log(rng, 1, 8), new_lo=1, new_hi=_log(rng, 1, 200), mem_lo=0, mem_hi=_log(rng, 1, 800))
    elif rng.random() < 0.5:  # one to four tokens a sequence
        mem = _log(rng, 60, 8000)
        case.update(seqs=_log(rng, 1, 64), new_lo=1, new_hi=rng.choice([1, 1, 1, 2, 3, 4]), mem_lo=rng.randint(1, mem), mem_hi=mem)
    else:
        new = _log(rng, 5, 700)
        case.update(seqs=_log(rng, 1, 16), new_lo=rng.randint(1, new), new_hi=new, mem_lo=0, mem_hi=_log(rng, 10, 2500), H=rng.randint(1, 8))
    return case


def _lengths(case):
    """Per sequence: rows of memory, new rows, dead rows at the head of the first page.  They go by the case alone."""
    rng = random.Random(case["pattern"])
    n = case["seqs"]
    mem = [rng.randint(case["mem_lo"], max(case["mem_lo"], case["mem_hi"])) for _ in range(n)]
    new = [rng.randint(case.get("new_lo", 1), case.get("new_hi", 1)) for _ in range(n)]
    start = [rng.randrange(case["page"]) if m else 0 for m in mem]
    return mem, new, start


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    row = case["H"] * case["D"] * size
    if case["op"] == "compact":  # the pages past the live count move, keys and values, read and written
        live = round(case["pages"] * case["live"])
        return {"bytes": 4 * case["page"] * row * live * (case["pages"] - live) / case["pages"] + 12 * case["pages"], "flops": 0}
    mem, new, start = _lengths(case)
    if case["op"] == "roll":  # the new rows of keys and values, read and written
        return {"bytes": 4 * row * sum(new) + 16 * case["seqs"], "flops": 0}
    if case["op"] == "beams":  # each branch: half a page copied, a row written; the table's row
        branches = case["seqs"] * (1 + case["beams"])
        return {"bytes": branches * (4 * row * (case["page"] // 2 + 1) + 8 * (sum(mem) / len(mem) / case["page"] + 1)), "flops": 0}
    pairs = sum(n * m + n * (n + 1) // 2 for n, m in zip(new, mem))
    longest = max(n + m for n, m in zip(new, mem))
    moved = row * (2 * sum(new) + 2 * (sum(new) + sum(mem)) + longest)
    return {"bytes": moved, "flops": 6 * case["H"] * case["D"] * pairs}


def _ints(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def _filled(case, g, slots, max_pages, n_pages, start, rows, ids):
    """A pool of random rows and the book of slots that hold `rows` rows each, in the pages `ids`."""
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    shape = (n_pages, case["H"], case["page"], case["D"])
    pool = [torch.empty(shape, device="cuda", dtype=dt).normal_(generator=g) for _ in range(2)]
    table = [[-1] * max_pages for _ in range(slots)]
    refs, at = [0] * n_pages, 0
    for s, (a, m) in enumerate(zip(start, rows)):
        n = -(-(a + m) // case["page"]) if m else 0
        table[s][:n] = ids[at:at + n]
        at += n
    for p in ids[:at]:
        refs[p] = 1
    return pool, dict(table=_ints(table), start=_ints(start), rows=_ints(rows), refs=_ints(refs))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rng = random.Random(int(seed))
    H, D, P = case["H"], case["D"], case["page"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    normal = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=g)  # noqa: E731
    s = dict(op=case["op"], page=P)
    if case["op"] == "compact":
        n = case["pages"]
        live = round(n * case["live"])
        ids = rng.sample(range(n), live)
        per = 9  # pages of a slot
        slots = -(-live // per)
        rows = [per * P] * (live // per) + ([(live % per) * P] if live % per else [])
        pool, book = _filled(case, g, slots, per, n, [0] * slots, rows, ids)
        s.update(k=pool[0], v=pool[1], book=book, before={x: t.clone() for x, t in book.items()}, new_id=_ints([0] * n), src=_ints([0] * n), dst=_ints([0] * n), count=_ints([0]))
        return s
    mem, new, start = _lengths(case)
    rows = [m + n for m, n in zip(mem, new)] if case["op"] == "attend" else mem
    slots = case["seqs"] * (1 + case.get("beams", 0))
    rows_all = rows + [0] * (slots - len(rows))
    start_all = [a if m else 0 for a, m in zip(start + [0] * (slots - len(start)), rows_all)]
    max_pages = max(-(-(P + m + n) // P) for m, n in zip(rows, new)) + 1
    need = sum(-(-(a + m) // P) for a, m in zip(start_all, rows_all))
    room = sum(-(-n // P) + 2 for n in new) * (2 + case.get("beams", 0))
    n_pages = need + room
    pool, book = _filled(case, g, slots, max_pages, n_pages, start_all, rows_all, rng.sample(range(n_pages), n_pages))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s.update(k=pool[0], v=pool[1], book=book, slots=_ints(list(range(case["seqs"]))), cu=_ints(cu))
    if case["op"] == "attend":
        longest = max(rows)
        s.update(q=normal(cu[-1], H, D).to(dt), r=(0.5 * normal(longest, H, D)).to(dt), u=0.1 * normal(H, D), vb=0.1 * normal(H, D), most=max(new), pages=max(-(-(a + m) // P) for a, m in zip(start_all, rows_all)))
        s["o"] = torch.empty_like(s["q"])
        return s
    if case["op"] == "beams":
        branch = list(range(case["seqs"], slots))
        s.update(source=_ints([i % case["seqs"] for i in range(len(branch))]), branch=_ints(branch), ok=_ints([0] * len(branch)), slots=_ints(list(range(slots))), cu=_ints(list(range(slots + 1))))
        cu = list(range(slots + 1))
        keep = mem + [0] * len(branch)
    else:
        keep = mem
    s.update(keep=_ints(keep), new_k=normal(cu[-1], H, D).to(dt), new_v=normal(cu[-1], H, D).to(dt), granted=_ints([0] * slots), src=_ints([0] * slots), dst=_ints([0] * slots))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _attend(s):
    book, P = s["book"], s["page"]
    slot = s["slots"].long()
    cu = s["cu"].long()
    first, n = cu[:-1], cu[1:] - cu[:-1]
    start, rows = book["start"].long()[slot], book["rows"].long()[slot]
    T, H, D = s["q"].shape
    i = torch.arange(s["most"], device="cuda")
    at = (first[:, None] + i).clamp(max=T - 1)  # [B, n]
    q = s["q"][at].float().transpose(1, 2)  # [B, H, n, D]
    page = book["table"].long()[slot, :s["pages"]].clamp(min=0)
    rows_of = lambda pool: pool[page].transpose(1, 2).flatten(2, 3).float()  # noqa: E731  [B, H, L, D]
    x = torch.arange(s["pages"] * P, device="cuda")
    d = (start + rows - n)[:, None, None] + i[:, None] - x  # [B, n, L]
    seen = (d >= 0) & (x >= start[:, None, None])
    far = (q + s["vb"][:, None]) @ s["r"].permute(1, 2, 0).float()  # [B, H, n, n_r]
    z = (q + s["u"][:, None]) @ rows_of(s["k"]).transpose(2, 3)
    z += far.gather(3, d.clamp(0, far.shape[3] - 1)[:, None].expand(z.shape))
    z = (z * D ** -0.5).masked_fill_(~seen[:, None], -torch.inf)
    e = (z - z.amax(3, keepdim=True)).exp_()
    o = (e @ rows_of(s["v"]).masked_fill(~seen.any(1)[:, None, :, None], 0.0)) / e.sum(3, keepdim=True)
    b = torch.bucketize(torch.arange(T, device="cuda"), cu[1:], right=True)
    s["o"].copy_(o.transpose(1, 2)[b, torch.arange(T, device="cuda") - first[b]])
    return s["o"]


def _reserve(s):
    book, P = s["book"], s["page"]
    slot, n = s["slots"].long(), s["cu"].long().diff()
    refs, table = book["refs"].long(), book["table"].long()[slot]
    end = (book["start"] + book["rows"]).long()[slot]
    have, want = (end + P - 1) // P, (end + n + P - 1) // P
    last = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    fits = (want <= table.shape[1]) & (n > 0)
    shared = (end % P > 0) & (refs[last.clamp(min=0)] > 1)
    need = torch.where(fits, want - have + shared, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= (refs == 0).sum()))
    shared &= ok
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)
    base = upto - need
    copy = free[base.clamp(max=len(free) - 1)]
    x = torch.arange(table.shape[1], device="cuda")
    new = ok[:, None] & (x >= have[:, None]) & (x < want[:, None])
    given = torch.where(new, free[((base + shared)[:, None] + x - have[:, None]).clamp(0, len(free) - 1)], table)
    over = shared[:, None] & (x == have[:, None] - 1)
    given = torch.where(over, copy[:, None], given)
    refs = refs.scatter_add(0, given.clamp(min=0).flatten(), (new | over).long().flatten())
    refs.scatter_add_(0, last.clamp(min=0), -shared.long())
    book["table"][slot] = given.int()
    book["refs"].copy_(refs)
    s["granted"].copy_(torch.where(ok, n, 0))
    s["src"].copy_(torch.where(shared, last, -1))
    s["dst"].copy_(torch.where(shared, copy, -1))
    book["rows"][slot] += s["granted"]


def _append(s):
    book, P = s["book"], s["page"]
    slot, cu, granted = s["slots"].long(), s["cu"].long(), s["granted"].long()
    end = (book["start"] + book["rows"]).long()[slot]
    copied = s["src"] >= 0
    src, dst = s["src"].long()[copied], s["dst"].long()[copied]
    old = torch.arange(P, device="cuda") < ((end - granted) % P)[copied][:, None]
    token = torch.arange(len(s["new_k"]), device="cuda")
    b = torch.bucketize(token, cu[1:], right=True)
    token, b = token[granted[b] > 0], b[granted[b] > 0]
    x = (end - granted)[b] + token - cu[b]
    page = book["table"].long()[slot[b], x // P]
    s["k"][dst] = torch.where(old[:, None, :, None], s["k"][src], s["k"][dst])
    s["v"][dst] = torch.where(old[:, None, :, None], s["v"][src], s["v"][dst])
    s["k"][page, :, x % P] = s["new_k"][token]
    s["v"][page, :, x % P] = s["new_v"][token]


def _free(s):
    book, P = s["book"], s["page"]
    slot = s["slots"].long()
    start, rows, table = book["start"].long()[slot], book["rows"].long()[slot], book["table"].long()[slot]
    kept = torch.minimum(rows, s["keep"].long())
    begin = start + rows - kept
    dead = torch.where(kept > 0, begin // P, (start + rows + P - 1) // P)
    x = torch.arange(table.shape[1], device="cuda")
    gone = (x < dead[:, None]) & (table >= 0)
    book["refs"].scatter_add_(0, table.clamp(min=0).flatten(), -gone.int().flatten())
    y = x + dead[:, None]
    book["table"][slot] = torch.where(y < table.shape[1], table.gather(1, y.clamp(max=table.shape[1] - 1)), -1).int()
    book["start"][slot] = torch.where(kept > 0, begin % P, 0).int()
    book["rows"][slot] = kept.int()


def _fork(s):
    book = s["book"]
    a, b = s["source"].long(), s["branch"].long()
    table = book["table"][a]
    book["table"][b] = table
    book["start"][b] = book["start"][a]
    book["rows"][b] = book["rows"][a]
    book["refs"].scatter_add_(0, table.long().clamp(min=0).flatten(), (table >= 0).int().flatten())
    s["ok"].fill_(1)


def _compact(s):
    book = s["book"]
    refs = book["refs"].long()
    live, x = refs > 0, torch.arange(len(refs), device="cuda")
    n = live.sum()
    hole, moved = ~live & (x < n), live & (x >= n)
    to = torch.argsort((~hole).to(torch.int8), stable=True)
    origin = torch.argsort((~moved).to(torch.int8), stable=True)
    new_id = torch.where(moved, to[(moved.cumsum(0) - 1).clamp(min=0)], torch.where(live, x, -1))
    count = moved.sum()
    s["new_id"].copy_(new_id)
    s["count"].copy_(count.reshape(1))
    s["src"].copy_(torch.where(x < count, origin, -1))
    s["dst"].copy_(torch.where(x < count, to, -1))
    book["refs"].copy_(torch.zeros_like(refs).scatter_add_(0, new_id.clamp(min=0), torch.where(live, refs, 0)))
    table = book["table"].long()
    book["table"].copy_(torch.where(table >= 0, new_id[table.clamp(min=0)], -1))
    src, dst = s["src"][s["src"] >= 0].long(), s["dst"][s["src"] >= 0].long()
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]


def _plain(s):
    if s["op"] == "attend":
        return _attend(s)
    if s["op"] == "compact":
        return _compact(s)
    if s["op"] == "beams":
        _fork(s)
    _reserve(s)
    _append(s)
    return _free(s)


def _library(s):
    import transformer_xl_relative_txl_gb300 as txl

    book, P = s["book"], s["page"]
    if s["op"] == "attend":
        if "workspace" not in s:  # kept by a program beside its pool
            T, H, D = s["q"].shape
            size = txl.txl_relattn_paged_workspace_bytes(len(s["slots"]), T, H, D, s["q"].dtype)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return txl.txl_relattn_forward_paged(s["q"], s["k"], s["v"], book, s["slots"], s["cu"], s["r"], s["u"], s["vb"], s["o"], s["workspace"], max_new=s["most"])
    if s["op"] == "compact":
        txl.txl_pages_compact(book, P, s["new_id"], s["src"], s["dst"], s["count"])
        return txl.txl_pages_copy(s["k"], s["v"], s["src"], s["dst"])
    if s["op"] == "beams":
        txl.txl_pages_fork(book, P, s["source"], s["branch"], s["ok"])
    txl.txl_pages_reserve(book, P, s["slots"], s["cu"], s["granted"], s["src"], s["dst"])
    txl.txl_pages_append(book, s["k"], s["v"], s["slots"], s["cu"], s["granted"], s["src"], s["dst"], s["new_k"], s["new_v"])
    return txl.txl_pages_free(book, P, s["slots"], s["keep"])


def run(s):
    if s["op"] == "compact":  # the pool as it was before, so that every pass has the same pages to move
        s["book"]["table"].copy_(s["before"]["table"])
        s["book"]["refs"].copy_(s["before"]["refs"])
    if own:
        _library(s)
    else:
        _plain(s)
    if s["op"] == "attend":
        return s["o"]
    out = dict(s["book"], k=s["k"], v=s["v"], src=s["src"], dst=s["dst"])
    out.update({x: s[x] for x in ("granted", "ok", "new_id", "count") if x in s})
    return out


# ---------------------------------------------------------------------------
# exact values
# ---------------------------------------------------------------------------
def exact(case, seed):
    """The attention by its definition in 64 bits, a sequence at a time: every key row fetched by its own place in the
    table, the distance rows laid out for each query.  The other operators move rows and count: they have no such value."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    D, P = case["D"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, table = s["cu"].tolist(), s["book"]["table"].tolist()
    r = s["r"].double()
    for b, slot in enumerate(s["slots"].tolist()):
        a, m = int(s["book"]["start"][slot]), int(s["book"]["rows"][slot])
        where = torch.arange(a, a + m)
        pages = torch.tensor([table[slot][y] for y in (where // P).tolist()], device="cuda")
        inside = (where % P).cuda()
        n = cu[b + 1] - cu[b]
        for h in range(case["H"]):
            k, v = s["k"][pages, h, inside].double(), s["v"][pages, h, inside].double()
            q = s["q"][cu[b]:cu[b + 1], h].double()
            i = torch.arange(m - n, m, device="cuda")[:, None]
            j = torch.arange(m, device="cuda")[None]
            along = torch.einsum("id,jd->ij", q + s["vb"][h].double(), r[:m, h])
            z = torch.einsum("id,jd->ij", q + s["u"][h].double(), k) + along[torch.arange(n, device="cuda")[:, None], (i - j).clamp(min=0)]
            z = torch.where(j <= i, z / D ** 0.5, torch.full_like(z, -torch.inf))
            out[cu[b]:cu[b + 1], h] = torch.softmax(z, 1) @ v
    return out
