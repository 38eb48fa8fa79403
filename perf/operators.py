"""The paged-cache operators as they are measured: plain forms in elementary torch operations beside the
library's calls, on the same inputs.

  plan    block tables and slot maps from request lengths (tq.plan_pages)
  append  new keys and values into paged pools, with the channel bounds of every page they touch (tq.append_pages)
  select  the pages of each (sequence, kv head) that a channel-bound score ranks highest (tq.select_pages)
  attend  attention of one new token over a paged fp16 / bf16 cache, whole or over selected pages (tq.attend_pages)

A page holds 16 tokens.  `own` chooses between the library's calls and the plain forms.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_LIB = None


def _tq():
    global _LIB
    if _LIB is None:
        from kv_cache_vector_norm_b200 import tq
        _LIB = tq
    return _LIB


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 running requests: one new token each (latency)
        dict(name="plan_decode_64", op="plan", batch=64, heads=8, tokens=4096, new=1, scarce=False),
        # admission of 64 ragged prompts, some requests finished, too few free pages for all
        dict(name="plan_prefill_64x4096", op="plan", batch=64, heads=8, tokens=4096, new=4096, scarce=True),
        # the step's 64 new keys and values, bounds updated (latency)
        dict(name="append_decode_64_d64", op="append", batch=64, heads=8, q_heads=32, d=64, low=1, high=1, dtype="bf16",
             values=True),
        # ragged prefill of 8 prompts, keys and values cut out of a fused projection
        dict(name="append_prefill_8x8192_d128", op="append", batch=8, heads=8, q_heads=32, d=128, low=777, high=8192,
             dtype="fp16", values=True),
        # bounds alone, for a cache whose keys and values are stored compressed
        dict(name="append_bounds_64x1024_d256", op="append", batch=64, heads=8, q_heads=32, d=256, low=130, high=1024,
             dtype="fp16", values=False),
        # 64 requests of up to 4097 tokens keep 64 pages of each kv head
        dict(name="select_64x4096_d64", op="select", batch=64, heads=8, group=4, d=64, low=700, high=4097, budget=64,
             dtype="bf16"),
        # one long request keeps 512 of 8192 pages
        dict(name="select_128k_d128", op="select", batch=1, heads=8, group=8, d=128, low=131072, high=131072,
             budget=512, dtype="fp16"),
        # the first tokens of one chat request (latency)
        dict(name="attend_1x200_d128", op="attend", batch=1, heads=8, group=4, d=128, low=200, high=200, budget=0,
             dtype="fp16"),
        # a layer of 8 requests of 8192 tokens, 32 query heads
        dict(name="attend_8x8192_d128", op="attend", batch=8, heads=8, group=4, d=128, low=8192, high=8192, budget=0,
             dtype="fp16"),
        # one request of 128K tokens, 64 query heads
        dict(name="attend_128k_d128", op="attend", batch=1, heads=8, group=8, d=128, low=131072, high=131072, budget=0,
             dtype="bf16"),
        # 64 requests of 1 to 4097 tokens
        dict(name="attend_ragged_64x4096_d64", op="attend", batch=64, heads=8, group=4, d=64, low=1, high=4097,
             budget=0, dtype="bf16"),
        # the same cache at d = 256, every kv head reading 64 selected pages
        dict(name="attend_selected_64_d256", op="attend", batch=64, heads=8, group=4, d=256, low=1500, high=4097,
             budget=64, dtype="fp16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["plan", "append", "select", "attend"])
    heads = rng.choice([1, 2, 3, 4, 8])
    if op == "plan":
        tokens = _log(rng, 64, 4096)
        return dict(op=op, batch=_log(rng, 1, 64), heads=heads, tokens=tokens,
                    new=rng.choice([1, 2, max(2, tokens // 3), tokens]), scarce=rng.random() < 0.3)
    d = rng.choice([64, 128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8])
    batch = _log(rng, 1, 64)
    if op == "append":
        high = _log(rng, 1, max(2, (8192 * 8 * 128) // (batch * d * 2)))
        return dict(op=op, batch=batch, heads=heads, q_heads=heads * group, d=d, low=rng.randint(1, high), high=high,
                    dtype=dtype, values=rng.random() < 0.7)
    high = _log(rng, 1, max(2, min(131072, (131072 * 128) // (batch * d))))
    low = rng.randint(0, high) if batch > 1 else high
    if op == "select":
        return dict(op=op, batch=batch, heads=heads, group=group, d=d, low=low, high=high, budget=_log(rng, 2, 256),
                    dtype=dtype)
    return dict(op=op, batch=batch, heads=heads, group=group, d=d, low=low, high=high,
                budget=rng.choice([0, 0, _log(rng, 2, 128)]), dtype=dtype)


def _lengths(case):
    """Token counts spread evenly from low to high (every run of a case has the same ones, in another order)."""
    b, low, high = case["batch"], case["low"], case["high"]
    if b == 1:
        return np.array([high], dtype=np.int64)
    return low + (high - low) * np.arange(b, dtype=np.int64) // (b - 1)


def _plan_news(case):
    """New tokens of each request: -1 for every 9th (finished), else spread from 0 or 1 to `new`."""
    b, new = case["batch"], case["new"]
    if new <= 2:
        return np.full(b, new, dtype=np.int64)
    n = new * np.arange(b, dtype=np.int64) // max(1, b - 1)
    return np.where(np.arange(b) % 9 == 4, -1, n if b > 1 else new)


def work(case):
    if case["op"] == "plan":
        news = np.maximum(_plan_news(case), 0)
        pages = int(np.sum((news + PAGE - 1) // PAGE))
        # lengths, row starts and positions per request; a free page read and a table entry written per page; slots
        return dict(bytes=case["batch"] * 5 * 4 + pages * 8 + int(news.sum()) * case["heads"] * 8, flops=0)
    lens = _lengths(case)
    h, d = case["heads"], case["d"]
    pages = (lens + PAGE - 1) // PAGE
    if case["op"] == "append":
        rows = int(lens.sum()) * h
        copies = 4 if case["values"] else 1          # keys and values read and written; else keys read
        return dict(bytes=rows * (copies * d * 2 + 8) + int(pages.sum()) * h * 2 * d * 2, flops=rows * d * 2)
    hq = h * case["group"]
    if case["op"] == "select":
        scored = int(pages[pages > case["budget"]].sum())
        kept = int(np.minimum(pages, case["budget"]).sum())
        return dict(bytes=scored * h * 2 * d * 2 + case["batch"] * hq * d * 2 + scored * 4 + kept * h * 4,
                    flops=scored * hq * d * 2)
    if case["budget"]:
        lens = np.where(pages <= case["budget"], lens, (case["budget"] - 1) * PAGE + lens - (pages - 1) * PAGE)
    tokens = int(lens.sum())
    return dict(bytes=tokens * h * d * 4 + case["batch"] * hq * d * 6, flops=tokens * hq * d * 4)


# ----------------------------------------------------------------------------------------------- inputs

def _table(pages, width, total, g, dev):
    """A block table whose rows name disjoint random pages of a pool of `total`; -1 past each row's pages."""
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    start = torch.cumsum(pages, 0) - pages
    col = torch.arange(width, device=dev)
    at = (start[:, None] + col[None, :]).clamp(max=total - 1)
    return torch.where(col[None, :] < pages[:, None], perm[at], torch.full((), -1, dtype=torch.int32, device=dev))


def _keys(shape, dtype, g, dev):
    """Keys of a cache: per-channel scales exp(N(0, 1) / 2), a drift from page to page, noise."""
    n, h, t, d = shape
    scale = torch.exp(0.5 * torch.randn((1, h, 1, d), generator=g, device=dev))
    base = torch.randn((n, h, 1, d), generator=g, device=dev)
    out = torch.empty(shape, dtype=dtype, device=dev)
    step = max(1, (1 << 26) // (h * t * d))
    for i in range(0, n, step):
        noise = torch.randn((min(step, n - i), h, t, d), generator=g, device=dev)
        out[i:i + step] = ((0.7 * noise + 0.7 * base[i:i + step]) * scale).to(dtype)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op, b, h = case["op"], case["batch"], case["heads"]
    mix = torch.randperm(b, generator=g, device=dev)
    if op == "plan":
        new = torch.from_numpy(_plan_news(case)).to(dev)[mix]
        width = (2 * case["tokens"] + PAGE - 1) // PAGE
        lens = torch.randint(0, case["tokens"] + 1, (b,), generator=g, device=dev)
        pages = (lens + PAGE - 1) // PAGE
        total = int(2 * b * ((case["tokens"] + PAGE - 1) // PAGE) + 3)
        table = _table(pages, width, total, g, dev)
        used = torch.zeros(total, dtype=torch.bool, device=dev)
        used[table[table >= 0].long()] = True
        free = torch.nonzero(~used).reshape(-1).to(torch.int32)
        free = free[torch.randperm(free.numel(), generator=g, device=dev)]
        need = int(((lens + new.clamp(min=0) + PAGE - 1) // PAGE - pages).sum())
        count = min(free.numel(), need * 3 // 4) if case["scarce"] else free.numel()
        head = int(torch.randint(0, total, (1,), generator=g, device=dev))
        ring = torch.full((total,), -1, dtype=torch.int32, device=dev)
        ring[(head + torch.arange(count, device=dev)) % total] = free[:count]
        rows = int(new.clamp(min=0).sum()) + 5                       # a padded batch: rows without a token
        return dict(op=op, heads=h, new_lens=new.to(torch.int32), seq_lens=lens.to(torch.int32), table=table, ring=ring,
                    free=torch.tensor([head, count], dtype=torch.int32, device=dev),
                    slots=torch.empty(rows * h, dtype=torch.int64, device=dev),
                    row_start=torch.empty(b + 1, dtype=torch.int32, device=dev),
                    start_pos=torch.empty(b, dtype=torch.int32, device=dev),
                    seq_lens_out=torch.empty(b, dtype=torch.int32, device=dev),
                    free_out=torch.empty(2, dtype=torch.int32, device=dev))
    dtype, d = DTYPES[case["dtype"]], case["d"]
    lens = torch.from_numpy(_lengths(case)).to(dev)[mix]
    if op == "append":
        old = torch.randint(0, 40, (b,), generator=g, device=dev)      # tokens that are cached already
        pages = (old + lens + PAGE - 1) // PAGE
        most = (lens + 39 + PAGE - 1) // PAGE
        total = int(most.sum()) + 2
        table = _table(pages, int(most.max()), total, g, dev)
        n = int(lens.sum())
        which = torch.repeat_interleave(torch.arange(b, device=dev), lens)
        pos = torch.arange(n, device=dev) - (torch.cumsum(lens, 0) - lens)[which] + old[which]
        page = table[which, pos // PAGE].long()
        slots = ((page[:, None] * h + torch.arange(h, device=dev)) * PAGE + (pos % PAGE)[:, None]).reshape(-1)
        pool = _keys((total, h, PAGE, d), dtype, g, dev)
        hq = case["q_heads"]
        qkv = torch.randn((n, hq + 2 * h, d), generator=g, device=dev, dtype=torch.float32).to(dtype)
        state = dict(op=op, k=qkv[:, hq:hq + h], v=qkv[:, hq + h:], slots=slots,
                     bounds=torch.stack((pool.amin(2), pool.amax(2)), 2).contiguous(), k_pool=None, v_pool=None)
        if case["values"]:
            state.update(k_pool=pool, v_pool=torch.zeros_like(pool))
        return state
    hq = h * case["group"]
    pages = (lens + PAGE - 1) // PAGE
    total = int(pages.sum()) + 3
    table = _table(pages, max(1, int(pages.max())), total, g, dev)
    q = torch.randn((b, hq, d), generator=g, device=dev).to(dtype)
    k_pool = _keys((total, h, PAGE, d), dtype, g, dev)
    if op == "select":
        budget = case["budget"]
        return dict(op=op, q=q, bounds=torch.stack((k_pool.amin(2), k_pool.amax(2)), 2).contiguous(), table=table,
                    seq_lens=lens.to(torch.int32), budget=budget,
                    pages=torch.empty((b, h, budget), dtype=torch.int32, device=dev),
                    lens=torch.empty((b, h), dtype=torch.int32, device=dev))
    seq_lens = lens.to(torch.int32)
    if case["budget"]:
        # pages that a selection kept: random ones of each kv head in ascending order, the last page among them
        budget = case["budget"]
        rank = torch.rand((b, h, table.shape[1]), generator=g, device=dev)
        col = torch.arange(table.shape[1], device=dev)
        rank = torch.where(col == (pages - 1)[:, None, None], 2.0, torch.where(col < pages[:, None, None], rank, -1.0))
        kept = torch.zeros_like(rank, dtype=torch.bool)
        top = rank.topk(min(budget, table.shape[1]), dim=2)
        kept.scatter_(2, top.indices, top.values >= 0)
        order = torch.where(kept, col, table.shape[1]).sort(dim=2).values[:, :, :budget]
        ids = table[:, None, :].expand(b, h, -1).gather(2, order.clamp(max=table.shape[1] - 1))
        ids = torch.where(order < table.shape[1], ids * h + torch.arange(h, device=dev, dtype=torch.int32)[:, None], -1)
        table = torch.full((b, h, budget), -1, dtype=torch.int32, device=dev)
        table[:, :, :ids.shape[2]] = ids
        short = torch.where(pages <= budget, lens, (budget - 1) * PAGE + lens - (pages - 1) * PAGE)
        seq_lens = short.to(torch.int32)[:, None].expand(b, h).contiguous()
    return dict(op=op, q=q, k_pool=k_pool, v_pool=torch.randn(k_pool.shape, generator=g, device=dev, dtype=dtype),
                table=table, seq_lens=seq_lens, out=torch.empty((b, hq, d), dtype=torch.float32, device=dev),
                workspace=torch.empty(1 << 24, dtype=torch.uint8, device=dev))


# ------------------------------------------------------------------------------------------ one pass each

def run(state):
    op = state["op"]
    if own:
        return _own(state)
    if op == "plan":
        return _plan(state)
    if op == "append":
        return _append(state)
    if op == "select":
        return _select(state)
    return _attend(state)


def _own(s):
    tq, op = _tq(), s["op"]
    if op == "plan":
        p = tq.plan_pages(s["new_lens"], s["seq_lens"], s["table"], s["ring"], s["free"], num_kv_heads=s["heads"],
                          slots=s["slots"], row_start=s["row_start"], start_pos=s["start_pos"],
                          seq_lens_out=s["seq_lens_out"], free_state_out=s["free_out"])
        return dict(table=s["table"], ring=s["ring"], slots=p.slots, row_start=p.row_start, start_pos=p.start_pos,
                    seq_lens=p.seq_lens, free=p.free_state)
    if op == "append":
        tq.append_pages(s["k"], s["v"] if s["v_pool"] is not None else None, s["slots"], k_pool=s["k_pool"],
                        v_pool=s["v_pool"], bounds=s["bounds"])
        return dict(bounds=s["bounds"], k_pool=s["k_pool"], v_pool=s["v_pool"])
    if op == "select":
        pages, lens = tq.select_pages(s["q"], s["bounds"], s["table"], s["seq_lens"], budget=s["budget"], keep_first=1,
                                      keep_last=1, pages=s["pages"], lens=s["lens"])
        return dict(pages=pages, lens=lens)
    return tq.attend_pages(s["q"], s["k_pool"], s["v_pool"], s["table"], s["seq_lens"], out=s["out"],
                           workspace=s["workspace"])


def _plan(s):
    new, lens, table, ring, heads = s["new_lens"].long(), s["seq_lens"].long(), s["table"], s["ring"], s["heads"]
    width, cap, rows = table.shape[1], ring.numel(), s["slots"].numel() // heads
    head, count = s["free"][0].long(), s["free"][1].long()
    old_pages, req = (lens + PAGE - 1) // PAGE, new.clamp(min=0)
    end = torch.cumsum(req, 0)
    fits = (new >= 0) & (lens + req <= width * PAGE) & (end <= rows)
    need = torch.where(fits, (lens + req + PAGE - 1) // PAGE - old_pages, 0)
    upto = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (upto <= count))
    need = torch.where(ok, need, 0)
    gone = torch.where(new < 0, old_pages, 0)
    # finished requests' pages go to the ring's end, new pages come from its start
    col = torch.arange(width, device=table.device)
    pushed = col < gone[:, None]
    at = (head + count + (torch.cumsum(gone, 0) - gone)[:, None] + col) % cap
    rel = col - old_pages[:, None]
    fresh = (rel >= 0) & (rel < need[:, None])
    got = ring[(head + (upto - need)[:, None] + rel) % cap]
    ring[at[pushed]] = table[pushed]
    table.copy_(torch.where(fresh, got, table))
    start = torch.cat((end.new_zeros(1), end))
    start_pos = torch.where(ok, lens, -1)
    token = torch.arange(rows, device=table.device)
    which = torch.searchsorted(end, token, right=True).clamp(max=new.numel() - 1)
    pos = start_pos[which] + token - start[which]
    there = (token < end[-1]) & ok[which]
    page = table[which, torch.where(there, pos, 0) // PAGE].long()
    slots = (page[:, None] * heads + torch.arange(heads, device=table.device)) * PAGE + (pos % PAGE)[:, None]
    slots = torch.where(there[:, None], slots, -1).reshape(-1)
    seq_lens = torch.where(new < 0, 0, lens + torch.where(ok, req, 0))
    free = torch.stack(((head + need.sum()) % cap, count - need.sum() + gone.sum()))
    return dict(table=table, ring=ring, slots=slots, row_start=start.int(), start_pos=start_pos.int(),
                seq_lens=seq_lens.int(), free=free.int())


def _append(s):
    k, bounds, slots = s["k"], s["bounds"], s["slots"]
    n, h, d = k.shape
    if s["v_pool"] is not None:
        s["k_pool"].view(-1, d)[slots] = k.reshape(n * h, d)
        s["v_pool"].view(-1, d)[slots] = s["v"].reshape(n * h, d)
    flat = bounds.view(-1, 2, d)
    where = slots // PAGE
    fresh = where[slots % PAGE == 0]
    flat[fresh, 0] = math.inf
    flat[fresh, 1] = -math.inf
    rows, where = k.reshape(n * h, d).float(), where[:, None].expand(n * h, d)
    low = flat[:, 0].float().scatter_reduce(0, where, rows, "amin")
    high = flat[:, 1].float().scatter_reduce(0, where, rows, "amax")
    flat[:, 0], flat[:, 1] = low.to(bounds.dtype), high.to(bounds.dtype)
    return dict(bounds=bounds, k_pool=s["k_pool"], v_pool=s["v_pool"])


def _select(s):
    q, bounds, table, lens, budget = s["q"], s["bounds"], s["table"], s["seq_lens"].long(), s["budget"]
    b, hq, d = q.shape
    h, width = bounds.shape[1], table.shape[1]
    near = bounds[table.clamp(min=0).long()].permute(3, 0, 2, 1, 4).float()          # [2, B, H, pages, d]
    qf = q.float().view(b, h, hq // h, 1, d)
    # the largest q . k a key inside the page's bounds can have.  Products of 16-bit values are exact in 32 bits; the
    # order of the sum is the operator's: 8 channels as even and odd chains, then halves added to halves
    p = torch.maximum(qf * near[0][:, :, None], qf * near[1][:, :, None]).view(b, h, hq // h, width, d // 8, 4, 2)
    p = p[..., 0, :] + p[..., 1, :] + p[..., 2, :] + p[..., 3, :]
    p = p[..., 0] + p[..., 1]
    p = p[..., :16] + p[..., 16:] if d == 256 else p
    p = p[..., :8] + p[..., 8:] if d >= 128 else p
    p = p[..., :4] + p[..., 4:]
    p = p[..., :2] + p[..., 2:]
    score = (p[..., 0] + p[..., 1]).amax(2) + 0.0                                      # [B, H, pages]
    col = torch.arange(width, device=q.device)
    pages = (lens + PAGE - 1) // PAGE
    valid = col < pages[:, None, None]
    score = torch.where((col < 1) | (col >= (pages - 1)[:, None, None]), math.inf, score)   # kept always
    score = torch.where(valid, score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices[:, :, :budget]
    kept = torch.zeros_like(valid.expand(b, h, width)).scatter(2, order, True) & valid
    order = torch.where(kept, col, width).sort(dim=2).values[:, :, :budget]
    ids = table[:, None, :].expand(b, h, width).gather(2, order.clamp(max=width - 1))
    ids = torch.where(order < width, ids * h + torch.arange(h, device=q.device)[:, None], -1)
    s["pages"].fill_(-1)
    s["pages"][:, :, :ids.shape[2]] = ids
    short = torch.where(pages <= budget, lens, (budget - 1) * PAGE + lens - (pages - 1) * PAGE)
    s["lens"].copy_(short[:, None].expand(b, h))
    return dict(pages=s["pages"], lens=s["lens"])


def _attend(s):
    q, k_pool, v_pool, table, lens = s["q"], s["k_pool"], s["v_pool"], s["table"].long(), s["seq_lens"]
    b, hq, d = q.shape
    h = k_pool.shape[1]
    heads = torch.arange(h, device=q.device)[:, None]
    ids = (table if table.dim() == 3 else table[:, None, :] * h + heads).clamp(min=0)   # [B, H, pages]
    k = k_pool.view(-1, PAGE, d)[ids].view(b, h, -1, d).float()
    v = v_pool.view(-1, PAGE, d)[ids].view(b, h, -1, d).float()
    lens = lens if lens.dim() == 2 else lens[:, None].expand(b, h)
    hidden = torch.arange(k.shape[2], device=q.device) >= lens[:, :, None]              # [B, H, T]
    v = v.masked_fill_(hidden[..., None], 0.0)
    score = torch.matmul(q.float().view(b, h, hq // h, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    score = score.masked_fill_(hidden[:, :, None], -math.inf)
    top = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    return (torch.matmul(p, v) / torch.where(total == 0, 1.0, total)).view(b, hq, d)


# -------------------------------------------------------------------------------------- 64-bit definitions

def exact(case, seed):
    if case["op"] in ("plan", "select"):
        return None                                                                    # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "append":
        k, slots, lo_hi = s["k"].double(), s["slots"], s["bounds"].double()
        n, h, d = k.shape
        # every page's rows in a padded [page, 16] grid: what was there counts unless its first token is new
        total = lo_hi.shape[0] * h
        grid = torch.full((total * PAGE, d), math.nan, dtype=torch.float64, device=k.device)
        grid[slots] = k.reshape(n * h, d)
        grid = grid.view(total, PAGE, d)
        new = ~torch.isnan(grid)
        lo = torch.where(new, grid, math.inf).amin(1)
        hi = torch.where(new, grid, -math.inf).amax(1)
        keep = ~new[:, 0]
        lo = torch.where(keep, torch.minimum(lo, lo_hi.view(total, 2, d)[:, 0]), lo)
        hi = torch.where(keep, torch.maximum(hi, lo_hi.view(total, 2, d)[:, 1]), hi)
        return dict(bounds=torch.stack((lo, hi), 1).view(lo_hi.shape), k_pool=None, v_pool=None)
    q, table, lens = s["q"].double(), s["table"].long(), s["seq_lens"].long()
    b, hq, d = q.shape
    h = case["heads"]
    out = torch.zeros((b, h, hq // h, d), dtype=torch.float64, device=q.device)
    for i in range(b):                                                                 # one (sequence, kv head) at a time
        for j in range(h):
            t = int(lens[i, j] if lens.dim() == 2 else lens[i])
            if t <= 0:
                continue
            row = table[i, j] if table.dim() == 3 else table[i] * h + j
            row = row[:(t + PAGE - 1) // PAGE]
            k = s["k_pool"].view(-1, PAGE, d)[row].reshape(-1, d)[:t].double()
            v = s["v_pool"].view(-1, PAGE, d)[row].reshape(-1, d)[:t].double()
            logits = (q[i].view(h, hq // h, d)[j] @ k.T) / math.sqrt(d)
            out[i, j] = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True)) @ v
    return out.view(b, hq, d)
