"""Reading pages of a compressed cache: what lies behind a sequence's last token counts for nothing, and every reader takes the
pages that a selection picked for each kv head.

Attention is compared with 64-bit attention over the decoded pools by relative L2 error (L2_RTOL, the tolerance of the
compressed cache's attention)."""
import numpy as np
import pytest
import torch

from kv_cache_vector_norm_b200 import tq
from oracle import pages_oracle as po
from _tqh import L2_RTOL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def np64(t):
    return t.detach().double().cpu().numpy()


class Compressed:
    """Random rows in compressed pools of `rows` rows, whose codec has QJL residual keys or not."""

    def __init__(self, rows, d, bits, v_bits, v_group, qjl=False, seed=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        x, y = torch.randn((2, rows, d), generator=gen, device=DEV).half()
        self.d, self.rows, self.qjl, self.v_bits, self.v_group = d, rows, qjl, v_bits, v_group
        self.signs = self.rho = None
        if qjl:
            self.codec = tq.QjlCodec(d, bits, 0)
            packed, norms, self.signs, self.rho = self.codec.encode_k_qjl(x)
        else:
            self.codec = tq.Codec(d, bits, 0)
            packed, norms = self.codec.encode_k(x)
        self.cache = tq.Cache(packed, norms, *tq.encode_v(y, v_bits, v_group))
        self.kw = dict(v_bits=v_bits, v_group=v_group)

    def pools(self):
        arrays = [self.cache.k_packed, self.cache.k_norms, self.cache.v_data, self.cache.v_scales, self.cache.v_zeros]
        return arrays + ([self.signs, self.rho] if self.qjl else [])

    def attend(self, q, h, **kw):
        if self.qjl:
            return tq.attend_decode_qjl(self.codec, q, self.cache, self.signs, self.rho, num_kv_heads=h, **self.kw, **kw)
        return tq.attend_decode(self.codec, q, self.cache, num_kv_heads=h, **self.kw, **kw)

    def decoded(self, h):
        k = self.codec.decode_k(self.cache.k_packed, self.cache.k_norms, out_dtype=torch.float32)
        v = tq.decode_v(self.cache.v_data, self.cache.v_scales, self.cache.v_zeros, self.d, self.v_bits, self.v_group,
                        out_dtype=torch.float32)
        return np64(k).reshape(-1, h, 16, self.d), np64(v).reshape(-1, h, 16, self.d)


def spoil(t, rows):
    """Bytes in rows of a pool that no code, norm or scale has reason to hold: NaN where the pool holds numbers."""
    t[rows] = float("nan") if t.is_floating_point() else 0xA5


FORMATS = [(64, 2, 2, 32, False), (64, 4, 4, 64, False), (64, 3, 4, 32, True), (128, 4, 4, 32, False), (128, 2, 8, 128, False),
           (128, 6, 4, 32, False), (128, 3, 2, 32, True), (256, 4, 4, 32, True), (256, 3, 3, 256, False), (256, 4, 8, 32, False)]


@pytest.mark.parametrize("d,bits,v_bits,v_group,qjl", FORMATS)
@pytest.mark.parametrize("paged", [False, True])
def test_rows_behind_the_last_token(d, bits, v_bits, v_group, qjl, paged):
    """The same bits whatever the pools hold behind each sequence's last token: lengths that end inside a page, at one, in the
    first and in a later one, one split and many."""
    h, g, lens = 2, 3, [1, 15, 16, 0, 333, 2047, 2048]
    b, width = len(lens), 128
    c = Compressed(b * width * 16 * h, d, bits, v_bits, v_group, qjl)
    q = torch.randn((b, h * g, d), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).half()
    table = np.random.default_rng(0).permutation(b * width).reshape(b, width)
    kw = dict(block_table=i32(table)) if paged else dict(max_seq_len=width * 16)
    kw["seq_lens"] = i32(lens)
    want = c.attend(q, h, **kw)
    assert want.isfinite().all()
    t = np.arange(width * 16)
    for i, n in enumerate(lens):
        for j in range(h):
            row = (table[i, t // 16] * h + j) * 16 + t % 16 if paged else (i * h + j) * width * 16 + t
            for pool in c.pools():
                spoil(pool, torch.as_tensor(row[n:]).to(DEV))
    assert torch.equal(c.attend(q, h, **kw), want)


def selection(rng, b, h, n, pages, lens):
    """Head pages of random pages for each (sequence, kv head), and the tokens of each list."""
    ids = np.stack([[rng.permutation(pages)[:n] * h + j for j in range(h)] for _ in range(b)])
    return ids, np.asarray(lens)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_reader_takes_selected_pages(d):
    """attend_decode, attend_decode_noalloc, attend_decode_qjl and attend_scores on a list of pages per (sequence, kv head)."""
    rng = np.random.default_rng(d)
    b, h, g, n, num = 3, 2, 4, 11, 30
    gen = torch.Generator(device=DEV).manual_seed(d)
    q = torch.randn((b, h * g, d), generator=gen, device=DEV).half()
    ids, lens = selection(rng, b, h, n, num, [[170, 176], [5, 0], [100, 161]])
    kw = dict(block_table=i32(ids), seq_lens=i32(lens))
    c = Compressed(num * h * 16, d, 4, 4, 32)
    k, v = c.decoded(h)
    ref, _ = po.attend(np64(q), k, v, ids, lens, d ** -0.5, True)
    first = c.attend(q, h, **kw)
    assert np.linalg.norm(np64(first) - ref) <= L2_RTOL * np.linalg.norm(ref)
    assert not first[1, g:].any()
    assert torch.equal(tq.attend_decode_noalloc(c.codec, q, c.cache, num_kv_heads=h, **c.kw, **kw), first)
    scores = np64(tq.attend_scores(c.codec, q, c.cache, num_kv_heads=h, **c.kw, **kw))
    assert scores.shape == (b, h * g, n * 16)
    for i in range(b):
        for j in range(h):
            for x in range(g):
                t = np.arange(lens[i, j])
                want = k[ids[i, j, t // 16] // h, j, t % 16] @ np64(q)[i, j * g + x] * d ** -0.5
                got = scores[i, j * g + x]
                assert np.linalg.norm(got[:len(t)] - want) <= L2_RTOL * np.linalg.norm(want) and np.isneginf(got[len(t):]).all()
    # residual keys: one list for every kv head gives what the table of those pages gives
    c = Compressed(num * h * 16, d, 3, 4, 32, qjl=True)
    pages = rng.permutation(num)[None, :n].repeat(b, 0)
    lens = np.array([176, 3, 90])
    whole = c.attend(q, h, block_table=i32(pages), seq_lens=i32(lens))
    lists = np.stack([pages * h + j for j in range(h)], 1)
    got = c.attend(q, h, block_table=i32(lists), seq_lens=i32(lens[:, None].repeat(h, 1)))
    assert np.linalg.norm(np64(got - whole)) <= L2_RTOL * np.linalg.norm(np64(whole))


@pytest.mark.parametrize("d,bits,v_bits,v_group,qjl", FORMATS)
@pytest.mark.parametrize("b,n", [(2, 5), (3, 40), (1, 700)])
def test_negative_entries_are_left_out(d, bits, v_bits, v_group, qjl, b, n):
    """Entries of -1 (and other negative ones) at the start, inside and at the end of a row, for whole rows, for a whole stage
    of the copies; few pages and so many that the rows are split and block ids are read in several rounds."""
    rng = np.random.default_rng(d + n)
    h, g, num = 2, 3, n + 9
    c = Compressed(num * h * 16, d, bits, v_bits, v_group, qjl)
    gen = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn((b, h * g, d), generator=gen, device=DEV).half()
    table = np.stack([rng.permutation(num)[:n] for _ in range(b)])
    table[0, [0, n // 2, n - 1]] = [-1, -7, -2 ** 31]
    table[0, 4:8] = -1
    if b > 1:
        table[1] = -1
    if b > 2:
        table[2, rng.random(n) < 0.4] = -1
    lens = np.array([16 * n - 5, 16 * n - 16, 16 * n][:b])
    got = np64(c.attend(q, h, block_table=i32(table), seq_lens=i32(lens)))
    assert np.isfinite(got).all()
    if b > 1:
        assert not got[1].any()
    if not qjl:
        k, v = c.decoded(h)
        ref, _ = po.attend(np64(q), k, v, table, lens, d ** -0.5)
        assert np.linalg.norm(got - ref) <= L2_RTOL * np.linalg.norm(ref)
        lists = np.stack([np.where(table < 0, -1, table * h + j) for j in range(h)], 1)
        sel = np64(c.attend(q, h, block_table=i32(lists), seq_lens=i32(lens[:, None].repeat(h, 1))))
        assert np.linalg.norm(sel - ref) <= L2_RTOL * np.linalg.norm(ref)
        scores = tq.attend_scores(c.codec, q, c.cache, num_kv_heads=h, **c.kw, block_table=i32(table), seq_lens=i32(lens))
        there = (table.repeat(16, 1) >= 0) & (np.arange(16 * n) < lens[:, None])
        assert np.array_equal(np.isfinite(np64(scores)), there[:, None].repeat(h * g, 1))
        return
    # residual keys: the same pages in the same order without the others, whose last one is whole
    lens[:] = 16 * n
    got = np64(c.attend(q, h, block_table=i32(table), seq_lens=i32(lens)))
    short = np.full((b, n), 0)
    for i in range(b):
        good = table[i][table[i] >= 0]
        short[i, :len(good)], lens[i] = good, 16 * len(good)
    ref = np64(c.attend(q, h, block_table=i32(short), seq_lens=i32(lens)))
    assert np.linalg.norm(got - ref) <= L2_RTOL * np.linalg.norm(ref)


def test_a_selection_with_pages_that_are_none():
    """First and last pages are listed whatever their table entry names: the -1 that a selection gives for them goes through
    attention over compressed pages."""
    rng = np.random.default_rng(5)
    gen = torch.Generator(device=DEV).manual_seed(5)
    b, h, g, d, n, num, budget = 3, 2, 4, 128, 30, 100, 8
    c = Compressed(num * h * 16, d, 4, 4, 32)
    k, v = c.decoded(h)
    keys = torch.as_tensor(k, device=DEV).half()
    bounds = torch.stack((keys.amin(2), keys.amax(2)), 2).contiguous()
    table = np.stack([rng.permutation(num)[:n] for _ in range(b)])
    table[0, 0], table[1, n - 1], table[2, 3] = -1, num + 3, -1
    lens = np.array([16 * n - 3, 16 * n - 9, 70])
    q = torch.randn((b, h * g, d), generator=gen, device=DEV).half()
    pages, tokens = tq.select_pages(q, bounds, i32(table), i32(lens), budget=budget)
    assert (pages[0, :, 0] == -1).all() and (pages[1, :, budget - 1] == -1).all() and (pages[2, :, 3] == -1).all()
    got = np64(c.attend(q, h, block_table=pages, seq_lens=tokens))
    ref, _ = po.attend(np64(q), k, v, pages.cpu().numpy(), tokens.cpu().numpy(), d ** -0.5, True)
    assert np.linalg.norm(got - ref) <= L2_RTOL * np.linalg.norm(ref)


def test_operands_that_would_be_misread_are_refused():
    """Types, layouts and shapes of the query, the table, the lengths and the output that the kernels would read as something else
    are refused on the host, by every reader."""
    b, h, g, d, n, num = 2, 2, 4, 64, 3, 8
    c = Compressed(num * h * 16, d, 4, 4, 32)
    r = Compressed(num * h * 16, d, 3, 4, 32, qjl=True)
    q = torch.zeros((b, h * g, d), dtype=torch.float16, device=DEV)
    wide = torch.zeros((b, h * g + 2 * h, d), dtype=torch.float16, device=DEV)
    table, lens = i32(np.zeros((b, n))), i32([16, 20])
    lists, tokens = i32(np.zeros((b, h, n))), i32(np.full((b, h), 16))
    out = torch.zeros((b, h * g, d), device=DEV)

    def decode(q, out=out, **kw):
        return tq.attend_decode(c.codec, q, c.cache, num_kv_heads=h, out=out, **c.kw, **kw)

    def noalloc(q, out=out, **kw):
        return tq.attend_decode_noalloc(c.codec, q, c.cache, num_kv_heads=h, out=out, **c.kw, **kw)

    def qjl(q, out=out, **kw):
        return r.attend(q, h, out=out, **kw)

    def scores(q, out=None, **kw):
        return tq.attend_scores(c.codec, q, c.cache, num_kv_heads=h, **c.kw, **kw)

    bad = [(TypeError, "block_table", dict(block_table=table.long())), (TypeError, "seq_lens", dict(seq_lens=lens.long())),
           (ValueError, "q must be contiguous", dict(q=wide[:, :h * g])), (TypeError, "block_table", dict(block_table=table.cpu())),
           (ValueError, "block_table must be contiguous", dict(block_table=i32(np.zeros((n, b))).t())),
           (ValueError, "seq_lens must be contiguous", dict(seq_lens=i32([1, 1, 1, 1])[::2])),
           (ValueError, "block_table must be", dict(block_table=i32(np.zeros((1, n))))),
           (ValueError, "seq_lens must be", dict(seq_lens=i32([16, 16, 16]))), (ValueError, "seq_lens must be", dict(seq_lens=tokens)),
           (ValueError, "selected pages need", dict(block_table=lists)),
           (ValueError, "block_table", dict(block_table=i32(np.zeros((b, n, h))).transpose(1, 2), seq_lens=tokens)),
           (ValueError, "seq_lens must be contiguous", dict(block_table=lists, seq_lens=i32(np.full((h, b), 16)).t())),
           (ValueError, "selected pages need", dict(block_table=lists[:, :1].contiguous(), seq_lens=tokens))]
    bad_out = [(TypeError, "out", dict(out=out.half())), (ValueError, "out must be contiguous", dict(out=torch.zeros((b, h * g, 2 * d), device=DEV)[:, :, :d])),
               (ValueError, "shape of q", dict(out=out[:1]))]
    for read in (decode, noalloc, qjl, scores):
        read(q, block_table=table, seq_lens=lens), read(q, block_table=lists, seq_lens=tokens)
        for kind, what, kw in bad + (bad_out if read is not scores else []):
            with pytest.raises(kind, match=what):
                read(**{**dict(q=q, block_table=table, seq_lens=lens), **kw})
    torch.cuda.synchronize()
