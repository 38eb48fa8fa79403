"""The paged cache's operators one behind the other where selection and attention take two launches each, overlapping
selections, attention's accuracy on ordinary inputs, and calls at the edge of what the operators take."""
import numpy as np
import pytest
import torch

from kv_cache_vector_norm_b200 import tq
from oracle import pages_oracle as po
from _tqh import L2_RTOL
from test_gpu_pages import DEV, DTYPES, check_attend, check_select, i32, np64, page_bounds, pools, random_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_a_decode_loop_of_long_rows(captured, given):
    """A prompt of 6300 tokens among shorter ones, then single tokens, back to back on the GPU: rows of up to 400 pages, so few
    that scores take a grid of their own and attention is split and joined.  Workspaces given, or allocated by the calls (in a
    capture, from its pool)."""
    rng = np.random.default_rng(21)
    gen = torch.Generator(device=DEV).manual_seed(21)
    b, h, g, d, width, num_pages, budget = 4, 2, 4, 128, 400, 700, 60
    rows = 8000
    codec = tq.Codec(d, 4, 0)
    new, lens, state = i32([0] * b), i32([0] * b), i32([0, num_pages])
    table, ring = i32(np.full((b, width), -1)), i32(rng.permutation(num_pages))
    k = torch.zeros((rows, h, d), dtype=torch.float16, device=DEV)
    v, q = torch.zeros_like(k), torch.zeros((b, h * g, d), dtype=torch.float16, device=DEV)
    kp = torch.full((num_pages, h, 16, d), float("nan"), dtype=torch.float16, device=DEV)
    vp = kp.clone()
    bounds = torch.full((num_pages, h, 2, d), float("nan"), dtype=torch.float16, device=DEV)
    n_rows = num_pages * h * 16
    cache = tq.Cache(torch.zeros((n_rows, d // 2), dtype=torch.uint8, device=DEV), torch.zeros(n_rows, device=DEV),
                     torch.zeros((n_rows, d // 2), dtype=torch.uint8, device=DEV),
                     *(torch.zeros((n_rows, d // 32), dtype=torch.float16, device=DEV) for _ in range(2)))
    slots = torch.empty(rows * h, dtype=torch.int64, device=DEV)
    row_start, start_pos = i32([0] * (b + 1)), i32([0] * b)
    pages, tokens = i32(np.zeros((b, h, budget))), i32(np.zeros((b, h)))
    outs = [torch.zeros((b, h * g, d), device=DEV) for _ in range(4)]
    kw = dict(num_kv_heads=h, v_bits=4, v_group=32)
    space = [None] * 5
    if given:
        space = [torch.full((5 * b * h * (width + 127),), 0xFF, dtype=torch.uint8, device=DEV),
                 tq.attend_pages_workspace(q, kp, vp, table, lens).fill_(0xFF),
                 tq.attend_pages_workspace(q, kp, vp, pages, tokens).fill_(0xFF),
                 *(tq.attend_workspace(codec, q, cache, block_table=t, seq_lens=s, max_seq_len=None, scale=0.0, **kw)
                   for t, s in ((table, lens), (pages, tokens)))]

    def step():
        tq.plan_pages(new, lens, table, ring, state, num_kv_heads=h, slots=slots, row_start=row_start, start_pos=start_pos,
                      seq_lens_out=lens, free_state_out=state)
        tq.append_pages(k, v, slots, k_pool=kp, v_pool=vp, bounds=bounds)
        codec.encode_k(k.view(-1, d), slots, cache.k_packed, cache.k_norms)
        tq.encode_v(v.view(-1, d), 4, 32, slots, cache.v_data, cache.v_scales, cache.v_zeros)
        tq.select_pages(q, bounds, table, lens, budget=budget, pages=pages, lens=tokens, workspace=space[0])
        tq.attend_pages(q, kp, vp, table, lens, out=outs[0], workspace=space[1])
        tq.attend_pages(q, kp, vp, pages, tokens, out=outs[1], workspace=space[2])
        tq.attend_decode(codec, q, cache, block_table=table, seq_lens=lens, out=outs[2], workspace=space[3], **kw)
        tq.attend_decode(codec, q, cache, block_table=pages, seq_lens=tokens, out=outs[3], workspace=space[4], **kw)

    step()                                                # nothing to add: also the warm-up before a capture
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for adds in ([6300, 17, 0, 900], [1, 1, 1500, 1], [1, -1, 1, 70], [1, 40, 1, 1]):
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
        assert np.array_equal(np64(bounds), bounds64, equal_nan=True)
        ids, toks = po.select(q.float().cpu().numpy(), bounds64, want["table"], want["seq_lens"], budget, 1, 1)
        assert np.array_equal(pages.cpu().numpy(), ids) and np.array_equal(tokens.cpu().numpy(), toks)
        kc = codec.decode_k(cache.k_packed, cache.k_norms, out_dtype=torch.float32).view(num_pages, h, 16, d)
        vc = tq.decode_v(cache.v_data, cache.v_scales, cache.v_zeros, d, 4, 32, out_dtype=torch.float32).view(num_pages, h, 16, d)
        for o, tab, ln, sel in ((0, want["table"], want["seq_lens"], False), (1, ids, toks, True)):
            ref, err = po.attend(np64(q), kp64, vp64, tab, ln, d ** -0.5, sel)
            assert np.all(np.abs(np64(outs[o]) - ref) <= err[:, :, None])
            ref, _ = po.attend(np64(q), np64(kc), np64(vc), tab, ln, d ** -0.5, sel)
            assert np.linalg.norm(np64(outs[o + 2]) - ref) <= L2_RTOL * np.linalg.norm(ref)


def test_selections_at_once():
    """Two selections of few long rows at a time, on two streams, each with its own workspace, and through a graph."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    h, g, d, n = 2, 4, 128, 1500
    bounds = page_bounds(gen, n, h, d, torch.float16)
    qs = [torch.randn((2, h * g, d), generator=gen, device=DEV).half() for _ in range(2)]
    table = torch.stack([torch.randperm(n, generator=gen, device=DEV) for _ in range(2)]).int()
    lens = i32([16 * n - 3, 16 * 700])
    first = [tq.select_pages(q, bounds, table, lens, budget=90) for q in qs]
    spaces = [torch.empty(5 * 2 * h * (n + 127), dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graph, held = torch.cuda.CUDAGraph(), None
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = tq.select_pages(qs[0], bounds, table, lens, budget=90)
    outs = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(tq.select_pages(qs[i % 2], bounds, table, lens, budget=90, workspace=spaces[i % 2]))
            if i == 7:
                graph.replay()                            # its workspace is the graph's own
    torch.cuda.synchronize()
    for i, (pages, tokens) in enumerate(outs):
        assert torch.equal(pages, first[i % 2][0]) and torch.equal(tokens, first[i % 2][1])
    assert torch.equal(held[0], first[0][0]) and torch.equal(held[1], first[0][1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_selection_of_everything_is_the_whole_cache(dtype, d):
    """Where neither form splits its rows, attention over a selection that keeps all pages has the same bits as attention over
    the table."""
    rng = np.random.default_rng(d)
    gen = torch.Generator(device=DEV).manual_seed(d)
    h, g, lens, width = 3, 4, [500, 17, 0, 390], 32
    num_pages = sum(-(-n // 16) for n in lens) + 1
    table, _ = random_table(rng, lens, width, num_pages)
    kp, vp = pools(gen, num_pages, h, d, DTYPES[dtype])
    bounds = torch.stack((kp.amin(2), kp.amax(2)), 2).contiguous()
    q = torch.randn((len(lens), h * g, d), generator=gen, device=DEV).to(DTYPES[dtype])
    pages, tokens = tq.select_pages(q, bounds, i32(table), i32(lens), budget=width)
    assert torch.equal(tq.attend_pages(q, kp, vp, pages, tokens), tq.attend_pages(q, kp, vp, i32(table), i32(lens)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("b,width", [(2, 20), (160, 24), (2, 120), (3, 300)])
def test_attend_pages_accuracy(dtype, d, b, width):
    """Ordinary inputs: every output row within po.ROW_RTOL of the 64-bit result in relative L2 error.  One CTA per row (of eight
    warps, of four), and rows joined from several."""
    rng = np.random.default_rng(b + d)
    gen = torch.Generator(device=DEV).manual_seed(b + d)
    h, g = 1, 4
    lens = rng.integers(8 * width, 16 * width + 1, b)
    num_pages = int(sum(-(-lens // 16)))
    table, _ = random_table(rng, lens, width, num_pages)
    kp, vp = (torch.randn((num_pages, h, 16, d), generator=gen, device=DEV).to(DTYPES[dtype]) for _ in range(2))
    q = torch.randn((b, h * g, d), generator=gen, device=DEV).to(DTYPES[dtype])
    got = np64(tq.attend_pages(q, kp, vp, i32(table), i32(lens)))
    want, _ = po.attend(np64(q), np64(kp), np64(vp), table, lens, d ** -0.5)
    assert po.row_error(got, want).max() <= po.ROW_RTOL, po.row_error(got, want).max()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("b,n", [(40, 150), (3, 700)])
def test_select_with_infinite_bounds(dtype, d, b, n):
    """Keys that are infinite in a channel: a page's score is what the formula gives (finite, infinite, or not a number where
    infinities of both signs or 0 * infinity meet), by one kernel and by two."""
    rng = np.random.default_rng(d + b)
    gen = torch.Generator(device=DEV).manual_seed(d + b)
    h, g, num = 2, 3, 900
    bounds = page_bounds(gen, num, h, d, DTYPES[dtype])
    kind = torch.as_tensor(rng.integers(0, 12, (num, h)), device=DEV)      # half of the pages have an infinite bound
    channel = torch.as_tensor(rng.integers(0, d, (num, h, 2)), device=DEV)
    for e in range(num):
        for j in range(h):
            k, (x, y) = int(kind[e, j]), channel[e, j].tolist()
            if k in (0, 1):
                bounds[e, j, 0, x] = -torch.inf
            if k in (2, 1):
                bounds[e, j, 1, x] = torch.inf
            if k == 3:
                bounds[e, j, :, x] = -torch.inf
            if k == 4:
                bounds[e, j, 0, x], bounds[e, j, 0, y] = -torch.inf, -torch.inf
            if k == 5:
                bounds[e, j, :, x], bounds[e, j, 1, y] = -torch.inf, torch.inf
    q = torch.randn((b, h * g, d), generator=gen, device=DEV).to(DTYPES[dtype])
    q[0, 0, :d // 2] = 0
    table = np.stack([rng.permutation(num)[:n] for _ in range(b)])
    lens = rng.integers(16 * n // 2, 16 * n + 1, b)
    with np.errstate(invalid="ignore"):
        for budget in (12, n // 3):
            check_select(q, bounds, table, lens, budget, 1, 1)


def last_first(t):
    """A tensor with a leading dimension of one entry whose stride is 1: contiguous, as torch counts."""
    return t.contiguous()[..., None].movedim(-1, 0)


def test_strides_of_dimensions_of_one_entry():
    """A dimension of one entry has no step: whatever stride it carries is not looked at."""
    gen = torch.Generator(device=DEV).manual_seed(6)
    g, d, n = 4, 64, 40
    kp, vp = pools(gen, 3, 1, d, torch.float16)
    bounds = torch.stack((kp.amin(2), kp.amax(2)), 2).contiguous()
    q = torch.randn((1, g, d), generator=gen, device=DEV).half()
    table, lens = i32([[2, 0, 1]]), i32([n])
    want = tq.attend_pages(q, kp, vp, table, lens)
    odd_q = last_first(q[0])
    odd_k, odd_v = (t[:, 0].contiguous()[..., None].movedim(-1, 1) for t in (kp, vp))                  # one head
    assert odd_q.stride(0) == 1 and odd_k.stride(1) == 1 and odd_q.is_contiguous() and odd_k.is_contiguous()
    assert torch.equal(tq.attend_pages(odd_q, odd_k, odd_v, table, lens), want)
    for a, b in zip(tq.select_pages(odd_q, bounds, table, lens, budget=2), tq.select_pages(q, bounds, table, lens, budget=2)):
        assert torch.equal(a, b)
    one = [last_first(t[2]) for t in (kp, vp)]                                                         # one page
    lists, tokens = i32([[[0]]]), i32([[16]])
    assert one[0].stride(0) == 1 and torch.equal(tq.attend_pages(q, *one, lists, tokens), tq.attend_pages(q, kp, vp, i32([[[2]]]), tokens))
    far = torch.stack((kp, vp), 1)[2:]                                                                 # one page of a joint pool
    assert torch.equal(tq.attend_pages(q, far[:, 0], far[:, 1], lists, tokens), tq.attend_pages(q, kp, vp, i32([[[2]]]), tokens))
    for h, rows in ((3, 1), (1, 5), (1, 1)):
        k, v = torch.randn((2, rows, h, d), generator=gen, device=DEV).half()
        odd = [last_first(t[0]) if rows == 1 else t[:, 0].contiguous()[..., None].movedim(-1, 1) for t in (k, v)]
        assert 1 in odd[0].stride()[:2]
        slots = torch.arange(rows * h, device=DEV) * 16
        got, ref = ([torch.zeros((rows, h, 16, d), device=DEV).half() for _ in range(2)] for _ in range(2))
        near = [torch.zeros((rows, h, 2, d), device=DEV).half() for _ in range(2)]
        tq.append_pages(*odd, slots, k_pool=got[0], v_pool=got[1], bounds=near[0])
        tq.append_pages(k, v, slots, k_pool=ref[0], v_pool=ref[1], bounds=near[1])
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and torch.equal(*near)
        assert torch.equal(got[0].view(-1, d)[slots], k.view(-1, d))
