"""The paged cache's operators on the GPU against plain implementations (oracle/pages_oracle.py).

Planning, appending and selecting are compared bit for bit (the selection's 32-bit sums have a defined order).
Attention is compared element by element with the error bound the oracle derives from the inputs: d products per
logit, the weights' 2^-20, and the token sums, each rounding in 32 bits.
"""
import numpy as np
import pytest
import torch

from kv_cache_vector_norm_b200 import tq
from oracle import pages_oracle as po

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def random_table(rng, lens, width, num_pages, extra=0):
    """Disjoint random pages for every sequence; -1 behind them."""
    perm = rng.permutation(num_pages)
    table, at = np.full((len(lens), width), -1, dtype=np.int64), 0
    for b, n in enumerate(lens):
        k = min(-(-int(n) // 16) + extra, width)
        table[b, :k] = perm[at:at + k]
        at += k
    assert at <= num_pages
    return table, perm[at:]


# ------------------------------------------------------------------------------------------------ planning

def run_plan(new, lens, table, ring, state, heads, max_tokens, alias=False):
    t_table, t_ring, t_state, t_lens = i32(table), i32(ring), i32(state), i32(lens)
    kw = dict(seq_lens_out=t_lens, free_state_out=t_state) if alias else {}
    plan = tq.plan_pages(i32(new), t_lens, t_table, t_ring, t_state, num_kv_heads=heads, max_tokens=max_tokens, **kw)
    torch.cuda.synchronize()
    return dict(table=t_table, ring=t_ring, slots=plan.slots, row_start=plan.row_start, start_pos=plan.start_pos,
                seq_lens=plan.seq_lens, free_state=plan.free_state)


def check_plan(new, lens, table, ring, state, heads, max_tokens, alias=False):
    want = po.plan(new, lens, table, ring, state, heads, max_tokens)
    got = run_plan(new, lens, table, ring, state, heads, max_tokens, alias)
    for name, w in want.items():
        assert np.array_equal(got[name].cpu().numpy(), w), name
    return want


@pytest.mark.parametrize("batch,heads,top,step,alias", [
    (1, 1, 40, 1, False), (1, 8, 5000, 5000, False), (7, 3, 100, 33, True), (64, 8, 600, 1, True), (64, 2, 300, 300, False),
    (1024, 1, 60, 2, False), (1025, 2, 40, 20, True), (2500, 1, 30, 1, False), (3, 2, 9000, 700, True)])
@pytest.mark.parametrize("scarce", [False, True])
def test_plan(batch, heads, top, step, alias, scarce):
    rng = np.random.default_rng(batch * 7 + heads + 1000 * scarce)
    width = -(-(top + step) // 16)
    lens = rng.integers(0, top + 1, batch)
    new = rng.integers(0, step + 1, batch)
    new[rng.random(batch) < 0.1] = -1
    num_pages = batch * width + 3
    table, free = random_table(rng, lens, width, num_pages)
    need = int(sum(-(-(l + max(n, 0)) // 16) - -(-l // 16) for l, n in zip(lens, new)))
    count = min(len(free), need // 2 if scarce else need + 5)
    head = int(rng.integers(0, num_pages))
    ring = np.full(num_pages, -7, dtype=np.int64)
    ring[(head + np.arange(count)) % num_pages] = free[:count]
    rows = int(np.maximum(new, 0).sum()) + 9
    want = check_plan(new, lens, table, ring, [head, count], heads, rows, alias)
    stored = want["slots"][want["slots"] >= 0]
    assert len(set(stored.tolist())) == len(stored)


@pytest.mark.parametrize("batch,heads,step", [(200, 8, 600), (256, 1, 500), (257, 1, 500), (256, 3, 6), (255, 4, 1), (256, 4, 1), (1, 5, 99999)])
@pytest.mark.parametrize("scarce", [False, True])
def test_plan_writes_over_its_inputs(batch, heads, step, scarce):
    """Lengths and ring state updated in place, at the batch and slot counts where the launches change."""
    rng = np.random.default_rng(batch + heads + 1000 * scarce)
    lens, new = rng.integers(0, 99, batch), rng.integers(min(step, 2), step + 1, batch)
    lens[::7], new[batch // 2:batch // 2 + 2] = 0, [-1, 0][:len(new[batch // 2:batch // 2 + 2])]
    if batch == 1:
        new[0] = step
    width = -(-(99 + step) // 16)
    num_pages = batch * width + 1
    table, free = random_table(rng, lens, width, num_pages)
    need = int(sum(-(-(l + max(n, 0)) // 16) - -(-l // 16) for l, n in zip(lens, new)))
    count, head = need * 3 // 4 if scarce else need, num_pages - 3
    ring = np.full(num_pages, -7, dtype=np.int64)
    ring[(head + np.arange(count)) % num_pages] = free[:count]
    check_plan(new, lens, table, ring, [head, count], heads, int(np.maximum(new, 0).sum()), True)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,heads", [(100, 8), (256, 2), (300, 4)])
def test_plan_steps_without_a_pause(captured, in_place, batch, heads):
    """Many steps of large calls one behind the other, each on the lengths, table and ring that the one before left, with
    requests that finish and a pool too small for all."""
    rng = np.random.default_rng(batch)
    steps, width, rows = 24, 12, 4000
    num_pages = batch * width // 3
    news = [np.where(rng.random(batch) < 0.15, -1, rng.integers(0, 60, batch)) for _ in range(steps)]
    state = dict(table=np.full((batch, width), -1, dtype=np.int64), ring=rng.permutation(num_pages), seq_lens=np.zeros(batch, dtype=np.int64),
                 free_state=np.array([0, num_pages]))
    t_table, t_ring, t_lens, t_state = i32(state["table"]), i32(state["ring"]), i32(state["seq_lens"]), i32(state["free_state"])
    t_news = [i32(n) for n in news]
    outs = [(torch.empty(rows * heads, dtype=torch.int64, device=DEV), torch.empty(batch + 1, dtype=torch.int32, device=DEV),
             torch.empty(batch, dtype=torch.int32, device=DEV)) for _ in news]

    other_lens, other_state = torch.empty_like(t_lens), torch.empty_like(t_state)

    def run():                                           # an even number of steps: the last one ends in t_lens, t_state
        lens, free, next_lens, next_free = t_lens, t_state, *((t_lens, t_state) if in_place else (other_lens, other_state))
        for new, (slots, row_start, start_pos) in zip(t_news, outs):
            tq.plan_pages(new, lens, t_table, t_ring, free, num_kv_heads=heads, slots=slots, row_start=row_start,
                          start_pos=start_pos, seq_lens_out=next_lens, free_state_out=next_free)
            lens, free, next_lens, next_free = next_lens, next_free, lens, free

    if captured:
        graph, kept = torch.cuda.CUDAGraph(), [t.clone() for t in (t_table, t_ring, t_lens, t_state)]
        run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run()
        for t, k in zip((t_table, t_ring, t_lens, t_state), kept):
            t.copy_(k)
        for o in outs:
            o[0].fill_(-9)
        graph.replay()
    else:
        run()
    torch.cuda.synchronize()
    refused = 0
    for new, (slots, row_start, start_pos) in zip(news, outs):
        state = po.plan(new, state["seq_lens"], state["table"], state["ring"], state["free_state"], heads, rows)
        refused += int(((state["start_pos"] < 0) & (new >= 0)).sum())
        assert np.array_equal(slots.cpu().numpy(), state["slots"])
        assert np.array_equal(row_start.cpu().numpy(), state["row_start"])
        assert np.array_equal(start_pos.cpu().numpy(), state["start_pos"])
    assert refused > batch
    for t, name in ((t_table, "table"), (t_ring, "ring"), (t_lens, "seq_lens"), (t_state, "free_state")):
        assert np.array_equal(t.cpu().numpy(), state[name]), name


def test_plan_refuses_what_does_not_fit():
    # request 1 passes its table row, 3 the input rows (and so do all behind it), 5 finishes all the same
    lens, new = [10, 60, 0, 5, 20, 33], [6, 10, 16, 40, 1, -1]
    table, free = random_table(np.random.default_rng(0), lens, 4, 40, extra=0)
    ring = np.full(40, -1, dtype=np.int64)
    ring[:len(free)] = free
    check_plan(new, lens, table, ring, [0, len(free)], 2, 50)
    # no free page at all: requests that need none go on
    check_plan([3, 1, 0], [10, 16, 7], np.array([[3, -1], [4, -1], [5, -1]]), np.full(9, -1), [4, 0], 2, 6)
    # lengths that pass 32 bits together; an empty input
    check_plan([2 ** 30] * 3 + [1], [0, 0, 0, 1], np.array([[0], [1], [2], [3]]), np.arange(8), [0, 0], 1, 5)
    check_plan([0, -1], [0, 20], np.array([[-1, -1], [6, 2]]), np.full(8, -1), [7, 0], 4, 0)


def test_plan_of_a_large_batch_with_few_tokens():
    # more requests than the planning CTA has threads, and slots few enough that it writes them itself
    rng = np.random.default_rng(2)
    lens, new = rng.integers(0, 50, 1500), np.zeros(1500, dtype=np.int64)
    new[[0, 3, 700, 1023, 1024, 1025, 1499]] = [40, 1, -1, 17, 33, -1, 2]
    table, free = random_table(rng, lens, 6, 9000)
    ring = np.full(9000, -1, dtype=np.int64)
    ring[:len(free)] = free
    check_plan(new, lens, table, ring, [0, len(free)], 3, 100)


def test_plan_lengths_and_pages_that_are_wrong_are_contained():
    # a length past the table row counts as a full row, a negative one as empty; table entries that name no page give
    # slot -1
    table = np.array([[1, 2], [9, 3], [-5, 4], [3, 100]])
    check_plan([1, 4, 3, 2], [1000, -3, 8, 20], table, np.array([5, 6, 7, 0, 0, 0, 0, 0, 0]), [0, 3], 2, 12)


# ----------------------------------------------------------------------------------------------- appending

def make_rows(gen, n, h, d, dtype, fused):
    if fused:                                     # keys and values inside a fused projection
        qkv = torch.randn((n, 3 * h + 1, d), generator=gen, device=DEV).to(dtype)
        return qkv[:, h:2 * h], qkv[:, 2 * h:3 * h]
    return (torch.randn((n, h, d), generator=gen, device=DEV).to(dtype),
            torch.randn((n, h, d), generator=gen, device=DEV).to(dtype))


def ragged_slots(rng, new, old, h, num_pages, pad=0):
    """Slots of new[b] tokens at positions old[b].. of sequences with random pages; `pad` rows of -1 behind."""
    table, _ = random_table(rng, [o + n for o, n in zip(old, new)], max(-(-(o + n) // 16) for o, n in zip(old, new)), num_pages)
    slots = [(table[b, t // 16] * h + j) * 16 + t % 16 for b, (o, n) in enumerate(zip(old, new)) for t in range(o, o + n)
             for j in range(h)]
    return np.array(slots + [-1] * (pad * h), dtype=np.int64)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,old,h", [
    ([1], [0], 1), ([1], [17], 8), ([1, 1, 1, 0, 1], [15, 16, 0, 3, 40], 3), ([33, 0, 16, 1, 47], [5, 9, 16, 31, 0], 2),
    ([700, 1500, 64], [3, 0, 11], 8)])
def test_append(dtype, d, new, old, h):
    rng = np.random.default_rng(d + len(new))
    gen = torch.Generator(device=DEV).manual_seed(d)
    num_pages = sum(-(-(o + n) // 16) for o, n in zip(old, new)) + 3
    slots = ragged_slots(rng, new, old, h, num_pages, pad=3)
    k, v = make_rows(gen, len(slots) // h, h, d, DTYPES[dtype], fused=True)
    pools = [torch.randn((num_pages, h, 16, d), generator=gen, device=DEV).to(DTYPES[dtype]) for _ in range(2)]
    bounds = torch.stack((pools[0].amin(2), pools[0].amax(2)), 2).contiguous()
    want = po.append(np64(k), np64(v), slots, *map(np64, pools), np64(bounds))
    tq.append_pages(k, v, torch.from_numpy(slots).to(DEV), k_pool=pools[0], v_pool=pools[1], bounds=bounds)
    for got, w in zip((*pools, bounds), want):
        assert np.array_equal(np64(got), w)


@pytest.mark.parametrize("which", ["k", "v", "kv", "bounds"])
def test_append_parts(which):
    rng = np.random.default_rng(5)
    gen = torch.Generator(device=DEV).manual_seed(5)
    h, d, num_pages = 2, 128, 12
    slots = ragged_slots(rng, [20, 7, 40], [3, 0, 13], h, num_pages)
    k, v = make_rows(gen, len(slots) // h, h, d, torch.float16, fused=False)
    shape = (num_pages, h, 16, d)
    kp = torch.randn(shape, generator=gen, device=DEV).half() if "k" in which else None
    vp = torch.randn(shape, generator=gen, device=DEV).half() if "v" in which else None
    bounds = torch.zeros((num_pages, h, 2, d), device=DEV).half() if which == "bounds" else None
    want = po.append(np64(k), np64(v), slots, *(None if t is None else np64(t) for t in (kp, vp, bounds)))
    tq.append_pages(k, v if vp is not None else None, torch.from_numpy(slots).to(DEV), k_pool=kp, v_pool=vp, bounds=bounds)
    for got, w in zip((kp, vp, bounds), want):
        assert (got is None) == (w is None) and (w is None or np.array_equal(np64(got), w))


def test_append_odd_slots():
    # slots past the pool and negative ones skip the row; a slot named twice (as a long run of one page, too) keeps one
    # of its rows; runs that cross a warp's tile and end the input
    gen = torch.Generator(device=DEV).manual_seed(1)
    d, num_pages = 64, 5
    k = torch.randn((90, 1, d), generator=gen, device=DEV).half()
    pool = torch.zeros((num_pages, 1, 16, d), device=DEV).half()
    bounds = torch.zeros((num_pages, 1, 2, d), device=DEV).half()
    slots = np.full(90, -1, dtype=np.int64)
    slots[:3] = [num_pages * 16, 2 ** 40, -9]
    slots[5:55] = 16 + 3                           # one slot of page 1, fifty times
    slots[60:76] = 48 + np.arange(16)              # a whole page 3
    slots[76:90] = 64 + np.arange(14)              # page 4, to the end of the input
    tq.append_pages(k, None, torch.from_numpy(slots).to(DEV), k_pool=pool, bounds=bounds)
    kk, p = k[:, 0], pool[:, 0]
    assert bool((kk[5:55] == p[1, 3]).all(1).any())
    assert torch.equal(p[3], kk[60:76]) and torch.equal(p[4, :14], kk[76:90])
    rest = torch.ones(num_pages * 16, dtype=torch.bool)
    rest[19], rest[48:78] = False, False
    assert not p.reshape(-1, d)[rest.to(DEV)].any()
    assert torch.equal(bounds[1, 0, 0], torch.minimum(kk[5:55].amin(0), torch.zeros_like(kk[0])))
    assert torch.equal(bounds[3, 0, 1], kk[60:76].amax(0)) and torch.equal(bounds[4, 0, 0], kk[76:90].amin(0))
    assert not bounds[0].any() and not bounds[2].any()


# ----------------------------------------------------------------------------------------------- selecting

def check_select(q, bounds, table, lens, budget, first, last):
    pages, tokens = tq.select_pages(q, bounds, i32(table), i32(lens), budget=budget, keep_first=first, keep_last=last)
    want_pages, want_tokens = po.select(q.float().cpu().numpy(), bounds.float().cpu().numpy(), np.asarray(table), lens, budget,
                                        first, last)
    assert np.array_equal(tokens.cpu().numpy(), want_tokens)
    assert np.array_equal(pages.cpu().numpy(), want_pages)


def page_bounds(gen, num_pages, h, d, dtype):
    mid = torch.randn((num_pages, h, 1, d), generator=gen, device=DEV)
    half = torch.rand((num_pages, h, 1, d), generator=gen, device=DEV)
    return torch.cat((mid - half, mid + half), 2).to(dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,h,g,budget,first,last", [
    ([0], 1, 1, 1, 0, 1), ([1, 16, 17], 2, 8, 2, 1, 1), ([100, 650, 0, 32, 641], 3, 4, 5, 1, 2), ([2049, 5000], 1, 7, 40, 4, 8),
    ([9001], 2, 3, 100, 1, 1), ([40000, 39999], 1, 2, 64, 0, 1), ([16 * 24600 + 3], 1, 1, 700, 2, 1),
    ([3000] * 80, 2, 1, 30, 1, 1), ([5000], 1, 5, 312, 1, 1)])
def test_select(dtype, d, lens, h, g, budget, first, last):
    rng = np.random.default_rng(d + g)
    gen = torch.Generator(device=DEV).manual_seed(d + g)
    width = max(1, -(-max(lens) // 16) + 2)
    num_pages = sum(-(-n // 16) for n in lens) + 2
    table, _ = random_table(rng, lens, width, num_pages)
    q = torch.randn((len(lens), h * g, d), generator=gen, device=DEV).to(DTYPES[dtype])
    check_select(q, page_bounds(gen, num_pages, h, d, DTYPES[dtype]), table, lens, budget, first, last)


def test_select_ties_go_to_the_lowest_index():
    gen = torch.Generator(device=DEV).manual_seed(0)
    h, d, n = 2, 128, 500
    bounds = page_bounds(gen, 4, h, d, torch.float16)[torch.arange(n, device=DEV) % 4].contiguous()    # four different scores
    q = torch.randn((1, h, d), generator=gen, device=DEV).half()
    for budget in (3, 100, 126, 127, 250, 499, 500, 501):
        check_select(q, bounds, np.arange(n)[None], [n * 16 - 5], budget, 1, 1)
    check_select(torch.zeros_like(q), -bounds.abs(), np.arange(n)[None], [n * 16], 77, 0, 1)           # zeros of either sign


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_select_scores_that_only_the_defined_order_tells_apart(dtype, d):
    """Pages whose scores differ by less than the sums' own rounding: large terms, one channel a step apart.  A few of them
    or more than a row's list of doubtful pages holds, with the threshold among them; the others lie above or below."""
    gen = torch.Generator(device=DEV).manual_seed(d)
    n = 700
    dt = DTYPES[dtype]
    q = torch.randn((1, 3, d), generator=gen, device=DEV).to(dt)
    base = torch.sort(torch.randn((2, d), generator=gen, device=DEV), dim=0).values * 30
    for near in (12, 200, 300, 650):
        scale = torch.rand(n, generator=gen, device=DEV) * 0.5 + 1.2          # above, or the same below
        scale[torch.arange(n, device=DEV) % 2 == 0] *= -1
        bounds = torch.sort((base * scale[:, None, None]).to(dt).float(), dim=1).values
        at = torch.randperm(n, generator=gen, device=DEV)[:near]
        group = base.to(dt).float().repeat(near, 1, 1)
        step = torch.randint(-3, 4, (near, 4), generator=gen, device=DEV) * torch.finfo(dt).eps
        channel = torch.randint(0, d, (near, 4), generator=gen, device=DEV)
        group[:, 1].scatter_(1, channel, group[:, 1].gather(1, channel) * (1 + step))
        bounds[at] = torch.sort(group, dim=1).values
        bounds = bounds.to(dt)[:, None].contiguous()
        score = po.page_scores(q[0].float().cpu().numpy(), *(bounds[:, 0, i].float().cpu().numpy() for i in (0, 1)))
        above = int((score > score[at.cpu().numpy()].max()).sum())
        for budget in (above + 3, above + near // 2, above + near - 2):
            check_select(q, bounds, np.arange(n)[None], [n * 16], min(max(budget, 2), n - 1), 1, 1)


def test_select_bad_pages_and_numbers():
    gen = torch.Generator(device=DEV).manual_seed(3)
    h, d, n = 1, 64, 300
    bounds = page_bounds(gen, n, h, d, torch.bfloat16)
    bounds[5], bounds[17, 0, 0, 3] = float("nan"), float("nan")
    table = np.arange(n)[None].repeat(2, 0)
    table[0, [2, 40, 41]] = [-1, n, 2 ** 30]
    q = torch.randn((2, 4, d), generator=gen, device=DEV).bfloat16()
    for budget in (20, 296, 299):
        check_select(q, bounds, table, [n * 16, n * 16 - 30], budget, 3, 1)


@pytest.mark.parametrize("b", [1, 9, 18, 37, 80])
@pytest.mark.parametrize("budget", [3, 90, 510, 517, 700])
def test_select_long_rows_in_batches(b, budget):
    """Rows of very different lengths, so few of them that several CTAs make a row's choice, or so many that one does; most
    scores equal to others, and more or fewer pages wanted than the choice's CTA has threads."""
    rng = np.random.default_rng(b + budget)
    gen = torch.Generator(device=DEV).manual_seed(b + budget)
    h, d, n, width = 2, 64, 1800, 1500
    bounds = page_bounds(gen, n, h, d, torch.bfloat16)
    bounds[::2] = bounds[torch.randint(0, 40, (n // 2,), generator=gen, device=DEV)]
    table = np.stack([rng.permutation(n)[:width] for _ in range(b)])
    lens = rng.integers(0, 16 * width + 40, b)
    lens[0] = 16 * width - 3
    q = torch.randn((b, h * 3, d), generator=gen, device=DEV).bfloat16()
    check_select(q, bounds, table, lens, budget, 1, 1)


def test_select_does_not_depend_on_the_call():
    """A row gets the same pages alone (in several CTAs) and in a large batch (one CTA), and on every run."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    b, h, g, d, n = 40, 8, 4, 128, 1200
    bounds = page_bounds(gen, n, h, d, torch.float16)
    q = torch.randn((b, h * g, d), generator=gen, device=DEV).half()
    table = torch.stack([torch.randperm(n, generator=gen, device=DEV) for _ in range(b)]).int()
    lens = torch.randint(16 * 200, 16 * n, (b,), generator=gen, device=DEV).int()
    pages, tokens = tq.select_pages(q, bounds, table, lens, budget=64)
    for i in (0, 7, 39):
        one, t = tq.select_pages(q[i:i + 1], bounds, table[i:i + 1], lens[i:i + 1], budget=64)
        assert torch.equal(one[0], pages[i]) and torch.equal(t[0], tokens[i])
    for _ in range(3):
        again, _ = tq.select_pages(q, bounds, table, lens, budget=64)
        assert torch.equal(again, pages)


# ----------------------------------------------------------------------------------------------- attention

def check_attend(q, kp, vp, table, lens, scale=0.0, **kw):
    selected = np.asarray(table).ndim == 3
    want, err = po.attend(np64(q), np64(kp), np64(vp), np.asarray(table), np.asarray(lens), scale or q.shape[2] ** -0.5,
                          selected)
    got = tq.attend_pages(q, kp, vp, i32(table), i32(lens), scale=scale, **kw)
    diff = np.abs(got.double().cpu().numpy() - want)
    assert np.all(diff <= err[:, :, None]), (diff / np.maximum(err[:, :, None], 1e-30)).max()
    return got


def pools(gen, num_pages, h, d, dtype):
    scale = torch.exp(0.5 * torch.randn((1, h, 1, d), generator=gen, device=DEV))
    return ((torch.randn((num_pages, h, 16, d), generator=gen, device=DEV) * scale).to(dtype),
            torch.randn((num_pages, h, 16, d), generator=gen, device=DEV).to(dtype))


def forget_unused(kp, vp, table, lens):
    """NaN in every pool row that no sequence's tokens occupy."""
    used = torch.zeros(kp.shape[0], 16, dtype=torch.bool)
    for row, n in zip(table, lens):
        for t in range(int(n)):
            used[int(row[t // 16]), t % 16] = True
    for t in (kp, vp):
        t[~used.to(DEV)[:, None, :].expand(t.shape[:3])] = float("nan")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,h,g", [
    ([0], 1, 1), ([1], 1, 8), ([15, 16, 17], 2, 3), ([200, 0, 33, 0], 8, 4), ([64, 1, 0, 700, 129], 3, 5), ([3000], 2, 8),
    ([0, 0, 1], 1, 2), ([1111, 5, 2048], 1, 7), ([0, 600, 0], 2, 1), ([530, 2], 150, 2)])
def test_attend_pages(dtype, d, lens, h, g):
    rng = np.random.default_rng(d + h)
    gen = torch.Generator(device=DEV).manual_seed(d + g)
    num_pages = sum(-(-n // 16) for n in lens) + 2
    table, _ = random_table(rng, lens, max(1, -(-max(lens) // 16)), num_pages)
    kp, vp = pools(gen, num_pages, h, d, DTYPES[dtype])
    forget_unused(kp, vp, table, lens)
    q = torch.randn((len(lens), h * g, d), generator=gen, device=DEV).to(DTYPES[dtype])
    check_attend(q, kp, vp, table, lens)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,width,long", [(64, 4, 0), (64, 40, 0), (128, 40, 0), (256, 40, 0), (64, 400, 6000), (256, 200, 3100)])
def test_attend_pages_many_sequences(dtype, d, width, long):
    """More sequences than a CTA has threads and more rows than CTAs: empty ones between, all short, or a long one among
    them that lies in many CTAs' shares.  Table rows of few pages take a CTA each."""
    rng = np.random.default_rng(1)
    gen = torch.Generator(device=DEV).manual_seed(2)
    lens = rng.integers(0, 60, 300)
    lens[::5], lens[128:140] = 0, 0
    if long:
        lens[77] = long
    num_pages = int(sum(-(-lens // 16)))
    table, _ = random_table(rng, lens, width, num_pages)
    kp, vp = pools(gen, num_pages, 2, d, DTYPES[dtype])
    q = torch.randn((300, 6, d), generator=gen, device=DEV).to(DTYPES[dtype])
    check_attend(q, kp, vp, table, lens)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("b,h,width", [(1, 1, 2), (1, 1, 48), (1, 1, 49), (37, 2, 48), (37, 2, 50), (74, 1, 49), (75, 1, 64), (75, 1, 65),
                                       (148, 1, 20), (149, 1, 33), (148, 1, 64)])
def test_attend_pages_where_the_split_begins(dtype, d, b, h, width):
    """Rows few and short enough for a CTA each, with eight warps or four, and the first that are split."""
    rng = np.random.default_rng(b + width)
    gen = torch.Generator(device=DEV).manual_seed(b + width)
    lens = rng.integers(0, 16 * width + 1, b)
    lens[0], lens[-1] = 16 * width - 7, 16 * width
    num_pages = int(sum(-(-lens // 16))) + 1
    table, _ = random_table(rng, lens, width, num_pages)
    kp, vp = pools(gen, num_pages, h, d, DTYPES[dtype])
    forget_unused(kp, vp, table, lens)
    q = torch.randn((b, h * 3, d), generator=gen, device=DEV).to(DTYPES[dtype])
    check_attend(q, kp, vp, table, lens)


def test_attend_pages_strided_operands_and_scale():
    rng = np.random.default_rng(3)
    gen = torch.Generator(device=DEV).manual_seed(3)
    lens, h, g, d = [300, 77], 2, 4, 128
    table, _ = random_table(rng, lens, 25, 40)
    joint = torch.randn((40, 2, h, 16, d), generator=gen, device=DEV).half()      # keys and values in one pool
    fused = torch.randn((2, h * g + 2 * h, d), generator=gen, device=DEV).half()  # queries in a fused projection
    for scale in (0.0, 0.031, -0.2):
        check_attend(fused[:, :h * g], joint[:, 0], joint[:, 1], table, lens, scale)


def test_attend_pages_bad_pages_and_lengths():
    """Entries that name no page are left out; lengths are clamped to the table row; rows without a page give zeros."""
    rng = np.random.default_rng(4)
    gen = torch.Generator(device=DEV).manual_seed(4)
    h, g, d, num = 2, 2, 64, 30
    kp, vp = pools(gen, num, h, d, torch.bfloat16)
    q = torch.randn((4, h * g, d), generator=gen, device=DEV).bfloat16()
    table = rng.integers(0, num, (4, 7))
    table[0, [0, 3]], table[1, 6], table[2] = [-1, num], 2 ** 31 - 1, -5
    got = check_attend(q, kp, vp, table, [100, 5000, 60, -8])
    assert not got[2].any() and not got[3].any()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("width", [8, 120])
def test_attend_pages_numbers_that_are_none(dtype, d, width):
    """A NaN or an infinite score shows in the heads that read it, an infinite value in its column, and nowhere else; rows
    whose scores are all -infinity give zeros.  Rows of one CTA, and rows joined from several."""
    rng = np.random.default_rng(5)
    gen = torch.Generator(device=DEV).manual_seed(5)
    h, g, n = 2, 3, 16 * width - 5
    table, _ = random_table(rng, [n] * 5, width, 5 * width)
    kp, vp = pools(gen, 5 * width, h, d, DTYPES[dtype])
    q = torch.randn((5, h * g, d), generator=gen, device=DEV).abs().add(0.1).to(DTYPES[dtype])
    at = width - 2                                       # a page that is neither the first nor the last of its row
    kp[int(table[0, at]), 1, 3, 7] = float("nan")
    kp[int(table[1, at]), 0, 4, 0] = float("inf")
    vp[int(table[2, at]), 1, 5, 9] = float("inf")
    kp[torch.as_tensor(table[3]).long().to(DEV), 0, :, 2] = float("-inf")
    q[4, 5, d - 1] = float("nan")
    got = tq.attend_pages(q, kp, vp, torch.as_tensor(table, dtype=torch.int32, device=DEV),
                          torch.full((5,), n, dtype=torch.int32, device=DEV)).cpu()
    want = torch.zeros_like(got, dtype=torch.bool)
    want[0, g:], want[1, :g], want[2, g:, 9], want[4, 5] = True, True, True, True
    assert torch.equal(got.isfinite(), ~want)
    assert got[0, g:].isnan().all() and got[1, :g].isnan().all() and got[4, 5].isnan().all()
    assert not got[3, :g].any() and got[3, g:].all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_pages_large_logits(d):
    """Logits far apart (running maximum, rescaling) and far from zero in every order of tokens."""
    gen = torch.Generator(device=DEV).manual_seed(d)
    n = 640
    ramp = torch.linspace(-1, 1, n, device=DEV)
    for order in (ramp, -ramp, ramp[torch.randperm(n, generator=gen, device=DEV)]):
        u = torch.randn(d, generator=gen, device=DEV)
        keys = (order[:, None] * u * 6).half().view(n // 16, 1, 16, d).contiguous()
        vals = torch.randn((n // 16, 1, 16, d), generator=gen, device=DEV).half()
        q = (u * torch.tensor([[1.0], [-1.0], [0.0], [3.0]], device=DEV)).half()[None]
        check_attend(q, keys, vals, np.arange(n // 16)[None], [n])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 256])
def test_attend_selected_pages(dtype, d):
    rng = np.random.default_rng(6)
    gen = torch.Generator(device=DEV).manual_seed(6)
    h, g, lens = 3, 4, [500, 17, 0, 3000]
    num_pages = sum(-(-n // 16) for n in lens) + 1
    table, _ = random_table(rng, lens, -(-max(lens) // 16), num_pages)
    kp, vp = pools(gen, num_pages, h, d, DTYPES[dtype])
    bounds = torch.stack((kp.amin(2), kp.amax(2)), 2).contiguous()
    q = torch.randn((len(lens), h * g, d), generator=gen, device=DEV).to(DTYPES[dtype])
    pages, tokens = tq.select_pages(q, bounds, i32(table), i32(lens), budget=20, keep_first=1, keep_last=2)
    check_attend(q, kp, vp, pages.cpu().numpy(), tokens.cpu().numpy())
    # a budget that holds everything is attention over the whole cache, bit for bit on short sequences
    pages, tokens = tq.select_pages(q, bounds, i32(table), i32(lens), budget=table.shape[1])
    check_attend(q, kp, vp, pages.cpu().numpy(), tokens.cpu().numpy())


def test_attend_pages_past_32_bit_offsets():
    """Pages whose first element lies past 2^31 elements (and 2^32 bytes) of a pool."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    h, d, num = 8, 256, 66000
    kp = torch.empty((num, h, 16, d), dtype=torch.float16, device=DEV)
    vp = torch.empty_like(kp)
    bounds = torch.empty((num, h, 2, d), dtype=torch.float16, device=DEV)
    ids = np.array([[65999, 3, 65537, 65600]])
    at = torch.from_numpy(ids[0]).to(DEV)
    n = 61
    k, v = torch.randn((2, n, h, d), generator=gen, device=DEV).half()
    slots = torch.tensor([(int(ids[0][t // 16]) * h + j) * 16 + t % 16 for t in range(n) for j in range(h)], device=DEV)
    tq.append_pages(k, v, slots, k_pool=kp, v_pool=vp, bounds=bounds)
    small = [t[at].contiguous() for t in (kp, vp, bounds)]
    q = torch.randn((1, h, d), generator=gen, device=DEV).half()
    got = tq.attend_pages(q, kp, vp, i32(ids), i32([n]))
    want, err = po.attend(np64(q), np64(small[0]), np64(small[1]), np.arange(4)[None], [n], d ** -0.5)
    assert np.all(np.abs(np64(got) - want) <= err[:, :, None])
    assert torch.equal(small[0].transpose(1, 2).reshape(64, h, d)[:n], k)
    pages, _ = tq.select_pages(q, bounds, i32(ids), i32([n]), budget=3)
    near, _ = po.select(q.float().cpu().numpy(), small[2].float().cpu().numpy(), np.arange(4)[None], [n], 3, 1, 1)
    assert np.array_equal(pages.cpu().numpy(), ids[0][near // h] * h + near % h)


def test_pages_repeat_bitwise_and_on_two_streams():
    gen = torch.Generator(device=DEV).manual_seed(8)
    h, g, d = 2, 4, 128
    lens = [4000, 900, 31]
    num_pages = sum(-(-n // 16) for n in lens)
    table, _ = random_table(np.random.default_rng(8), lens, 250, num_pages)
    kp, vp = pools(gen, num_pages, h, d, torch.float16)
    q = torch.randn((3, h * g, d), generator=gen, device=DEV).half()
    tab, ln = i32(table), i32(lens)
    first = tq.attend_pages(q, kp, vp, tab, ln)
    spaces = [tq.attend_pages_workspace(q, kp, vp, tab, ln) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(20):                                   # two calls at once, each with its own workspace
        with torch.cuda.stream(streams[i % 2]):
            outs.append(tq.attend_pages(q, kp, vp, tab, ln, workspace=spaces[i % 2]))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


def test_binding_refusals():
    """Wrong dtypes, shapes, layouts and devices are refused before anything is launched; so is what the library refuses."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    h, d, n = 2, 64, 9
    kp, vp = pools(gen, n, h, d, torch.float16)
    q = torch.zeros((3, 4, d), dtype=torch.float16, device=DEV)
    tab, lens = i32(np.zeros((3, 40))), i32([1, 1, 1])
    bounds = torch.zeros((n, h, 2, d), dtype=torch.float16, device=DEV)
    slots = torch.zeros(10 * h, dtype=torch.int64, device=DEV)
    k = torch.zeros((10, h, d), dtype=torch.float16, device=DEV)
    state, ring = i32([0, 0]), i32(np.zeros(n))

    def attend(q=q, kp=kp, vp=vp, tab=tab, lens=lens, **kw):
        return tq.attend_pages(q, kp, vp, tab, lens, **kw)

    def select(q=q, bounds=bounds, tab=tab, lens=lens, budget=4, **kw):
        return tq.select_pages(q, bounds, tab, lens, budget=budget, **kw)

    def append(k=k, v=k, slots=slots, kp=kp, vp=vp, bounds=bounds):
        return tq.append_pages(k, v, slots, k_pool=kp, v_pool=vp, bounds=bounds)

    def plan(new=lens, lens=lens, tab=tab, ring=ring, state=state, **kw):
        return tq.plan_pages(new, lens, tab, ring, state, **{**dict(num_kv_heads=h, max_tokens=10), **kw})

    attend(), select(), append(), plan()
    bad = [
        (TypeError, "float16", lambda: attend(q=q.float())), (TypeError, "CUDA", lambda: attend(q=q.cpu())),
        (TypeError, "k_pool", lambda: attend(kp=kp.bfloat16())), (TypeError, "v_pool", lambda: attend(vp=vp.cpu())),
        (ValueError, "v_pool", lambda: attend(vp=vp[:-1])), (ValueError, "k_pool", lambda: attend(kp=kp.transpose(1, 2))),
        (TypeError, "block_table", lambda: attend(tab=tab.long())), (ValueError, "block_table", lambda: attend(tab=tab[:2])),
        (ValueError, "block_table", lambda: attend(tab=tab.t().contiguous().t())), (ValueError, "seq_lens", lambda: attend(lens=lens[:2])),
        (ValueError, "q must", lambda: attend(q=q.transpose(0, 1))), (ValueError, "out", lambda: attend(out=torch.zeros(3, 4, 2 * d, device=DEV))),
        (TypeError, "workspace", lambda: attend(workspace=torch.zeros(1 << 20))),
        (tq.TQError, "workspace of", lambda: attend(workspace=torch.zeros(16, device=DEV))),
        (tq.TQError, "multiple", lambda: attend(q=q[:, :3].contiguous())), (TypeError, "must be real number", lambda: attend(scale="a")),
        (TypeError, "bounds", lambda: select(bounds=bounds.bfloat16())), (ValueError, "bounds", lambda: select(bounds=bounds[:, :, :1].contiguous())),
        (tq.TQError, "budget=1", lambda: select(budget=1)), (ValueError, "pages", lambda: select(pages=i32(np.zeros((3, h, 5))))),
        (ValueError, "v must", lambda: append(v=k[:5])), (ValueError, "v_pool needs v", lambda: append(v=None)),
        (ValueError, "slots", lambda: append(slots=slots[1:])), (TypeError, "slots", lambda: append(slots=slots.int())),
        (ValueError, "bounds", lambda: append(bounds=bounds[1:])), (ValueError, "needs k_pool", lambda: append(kp=None, vp=None, bounds=None)),
        (ValueError, "seq_lens", lambda: plan(lens=lens[:2])), (ValueError, "max_tokens or slots", lambda: plan(max_tokens=None)),
        (ValueError, "slots", lambda: plan(slots=slots, max_tokens=3)), (TypeError, "free_pages", lambda: plan(ring=ring.cpu())),
        (tq.TQError, "num_kv_heads=0", lambda: plan(num_kv_heads=0)), (tq.TQError, "max_tokens=-1", lambda: plan(slots=slots, max_tokens=-1))]
    for kind, what, call in bad[:-1]:
        with pytest.raises(kind, match=what):
            call()
    with pytest.raises((ValueError, tq.TQError)):
        bad[-1][2]()
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------- used together

@pytest.mark.parametrize("captured", [False, True])
def test_a_decode_loop(captured):
    """Steps of a serving loop: plan, store (uncompressed, and compressed with bounds), select, attend; compared with the
    oracle after every step.  Captured: one graph holds the step, replayed with new lengths, keys and queries."""
    rng = np.random.default_rng(11)
    gen = torch.Generator(device=DEV).manual_seed(11)
    b, h, g, d, width, num_pages, budget = 5, 2, 4, 128, 24, 90, 6
    rows = 150
    codec = tq.Codec(d, 4, 0)
    new, lens, state = i32([0] * b), i32([0] * b), i32([0, num_pages])
    table, ring = i32(np.full((b, width), -1)), i32(rng.permutation(num_pages))
    k = torch.zeros((rows, h, d), dtype=torch.float16, device=DEV)
    v, q = torch.zeros_like(k), torch.zeros((b, h * g, d), dtype=torch.float16, device=DEV)
    kp = torch.full((num_pages, h, 16, d), float("nan"), dtype=torch.float16, device=DEV)
    vp = kp.clone()
    bounds = torch.zeros((num_pages, h, 2, d), dtype=torch.float16, device=DEV)
    n_rows = num_pages * h * 16
    packed = torch.zeros((n_rows, d // 2), dtype=torch.uint8, device=DEV)
    norms = torch.zeros(n_rows, device=DEV)
    data = torch.zeros((n_rows, d // 2), dtype=torch.uint8, device=DEV)
    scales, zeros = (torch.zeros((n_rows, d // 32), dtype=torch.float16, device=DEV) for _ in range(2))
    cache = tq.Cache(packed, norms, data, scales, zeros)
    slots = torch.empty(rows * h, dtype=torch.int64, device=DEV)
    row_start, start_pos = i32([0] * (b + 1)), i32([0] * b)
    pages, tokens = i32(np.zeros((b, h, budget))), i32(np.zeros((b, h)))
    outs = [torch.zeros((b, h * g, d), device=DEV) for _ in range(4)]
    space = [tq.attend_pages_workspace(q, kp, vp, table, lens), tq.attend_pages_workspace(q, kp, vp, pages, tokens)]
    kw = dict(num_kv_heads=h, v_bits=4, v_group=32)
    cspace = [tq.attend_workspace(codec, q, cache, block_table=t, seq_lens=s, max_seq_len=None, scale=0.0, **kw)
              for t, s in ((table, lens), (pages, tokens))]

    def step():
        tq.plan_pages(new, lens, table, ring, state, num_kv_heads=h, slots=slots, row_start=row_start, start_pos=start_pos,
                      seq_lens_out=lens, free_state_out=state)
        tq.append_pages(k, v, slots, k_pool=kp, v_pool=vp, bounds=bounds)
        codec.encode_k(k.view(-1, d), slots, packed, norms)
        tq.encode_v(v.view(-1, d), 4, 32, slots, data, scales, zeros)
        tq.select_pages(q, bounds, table, lens, budget=budget, pages=pages, lens=tokens)
        tq.attend_pages(q, kp, vp, table, lens, out=outs[0], workspace=space[0])
        tq.attend_pages(q, kp, vp, pages, tokens, out=outs[1], workspace=space[1])
        tq.attend_decode(codec, q, cache, block_table=table, seq_lens=lens, out=outs[2], workspace=cspace[0], **kw)
        tq.attend_decode(codec, q, cache, block_table=pages, seq_lens=tokens, out=outs[3], workspace=cspace[1], **kw)

    step()                                                # nothing to add: also the warm-up before a capture
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    steps = [[20, 1, 0, 100, 3], [1, 1, 1, 1, 1], [1, -1, 30, 1, 14], [1, 40, 1, -1, 1], [80, 1, 1, 16, 1], [1, 1, 1, 1, 1]]
    for adds in steps:
        before = [t.cpu().numpy() for t in (lens, table, ring, state)]
        new.copy_(i32(adds))
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        prior = [np64(t) for t in (kp, vp, bounds)]
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        want = po.plan(adds, before[0], before[1], before[2], before[3], h, rows)
        for name, t in dict(table=table, ring=ring, slots=slots, row_start=row_start, start_pos=start_pos, seq_lens=lens,
                            free_state=state).items():
            assert np.array_equal(t.cpu().numpy(), want[name]), name
        kp64, vp64, bounds64 = po.append(np64(k), np64(v), want["slots"], *prior)
        assert np.array_equal(np64(kp), kp64, equal_nan=True) and np.array_equal(np64(vp), vp64, equal_nan=True)
        assert np.array_equal(np64(bounds), bounds64)
        ids, toks = po.select(q.float().cpu().numpy(), bounds64, want["table"], want["seq_lens"], budget, 1, 1)
        assert np.array_equal(pages.cpu().numpy(), ids) and np.array_equal(tokens.cpu().numpy(), toks)
        kc = codec.decode_k(packed, norms, out_dtype=torch.float32).view(num_pages, h, 16, d)
        vc = tq.decode_v(data, scales, zeros, d, 4, 32, out_dtype=torch.float32).view(num_pages, h, 16, d)
        for o, tab, ln, sel in ((0, want["table"], want["seq_lens"], False), (1, ids, toks, True)):
            ref, err = po.attend(np64(q), kp64, vp64, tab, ln, d ** -0.5, sel)
            assert np.all(np.abs(np64(outs[o]) - ref) <= err[:, :, None])
            ref, _ = po.attend(np64(q), np64(kc), np64(vc), tab, ln, d ** -0.5, sel)
            assert np.linalg.norm(np64(outs[o + 2]) - ref) <= 1e-3 * np.linalg.norm(ref)
