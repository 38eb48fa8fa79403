"""CPU-side checks of the paged-cache entry points: argument errors are reported without touching a GPU, workspace sizes,
and the plain implementations the GPU tests compare against, on cases worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

from kv_cache_vector_norm_b200 import tq
from oracle import pages_oracle as po

FAKE = 1 << 12                                        # an aligned address that is never followed


def refused(fn, args, what, status=tq.TQ_ERR_INVALID_ARG):
    assert getattr(tq.LIB, fn)(ctypes.byref(args), None) == status, what
    assert what.encode() in tq.LIB.tq_last_error(), (what, tq.LIB.tq_last_error())


def filled(cls, **kw):
    a = cls()
    for name, kind in cls._fields_:
        if kind is ctypes.c_void_p:
            setattr(a, name, FAKE)
    for name, value in kw.items():
        setattr(a, name, value)
    return a


def plan_args(**kw):
    return filled(tq.PlanArgs, **{**dict(batch=4, num_kv_heads=8, max_blocks=16, num_pages=64, max_tokens=64), **kw})


def append_args(**kw):
    return filled(tq.AppendArgs, **{**dict(dtype=tq.TQ_F16, head_dim=128, num_kv_heads=8, num_pages=64, num_tokens=3,
                                           k_token_stride=1024, k_head_stride=128, v_token_stride=1024, v_head_stride=128), **kw})


def select_args(**kw):
    return filled(tq.SelectArgs, **{**dict(dtype=tq.TQ_BF16, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, max_blocks=9,
                                           num_pages=64, budget=4, keep_first=1, keep_last=1, q_stride=512), **kw})


def attend_args(**kw):
    d = kw.get("head_dim", 128)
    return filled(tq.AttendPagesArgs, **{**dict(dtype=tq.TQ_F16, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                                                max_blocks=90, num_pages=64, selected=0, q_stride=1024, k_page_stride=32 * d,
                                                v_page_stride=32 * d, workspace_bytes=1 << 23), **kw})


@pytest.mark.parametrize("kw,what", [
    (dict(batch=0), "batch=0"), (dict(batch=(1 << 24) + 1), "batch="), (dict(num_kv_heads=0), "num_kv_heads=0"),
    (dict(max_blocks=0), "max_blocks=0"), (dict(num_pages=0), "num_pages=0"), (dict(num_pages=1 << 28), "num_pages="),
    (dict(max_tokens=-1), "max_tokens=-1"), (dict(max_tokens=1 << 31), "max_tokens="), (dict(new_lens=None), "NULL"),
    (dict(slots=None), "NULL"), (dict(free_state_out=None), "NULL"), (dict(slots=FAKE + 4), "misaligned"),
    (dict(block_table=FAKE + 2), "misaligned")])
def test_plan_refusals(kw, what):
    refused("tq_plan_pages", plan_args(**kw), what)


@pytest.mark.parametrize("kw,what,unsupported", [
    (dict(head_dim=96), "head_dim=96", True), (dict(dtype=tq.TQ_F32), "dtype=1", True), (dict(num_kv_heads=0), "num_kv_heads=0", False),
    (dict(num_pages=0), "num_pages=0", False), (dict(num_tokens=-1), "num_tokens=-1", False),
    (dict(k_pool=None, v_pool=None, bounds=None), "all NULL", False), (dict(k=None), "non-NULL", False),
    (dict(slots=None), "non-NULL", False), (dict(v=None), "v_pool without v", False), (dict(k=FAKE + 8), "16-byte", False),
    (dict(k_token_stride=1020), "k strides", False), (dict(v_head_stride=-8), "v strides", False)])
def test_append_refusals(kw, what, unsupported):
    refused("tq_append_pages", append_args(**kw), what, tq.TQ_ERR_UNSUPPORTED if unsupported else tq.TQ_ERR_INVALID_ARG)


def test_append_of_nothing_is_a_no_op():
    assert tq.LIB.tq_append_pages(ctypes.byref(append_args(num_tokens=0, k=None, slots=None)), None) == tq.TQ_OK


@pytest.mark.parametrize("kw,what,unsupported", [
    (dict(batch=0), "batch", False), (dict(num_q_heads=7), "multiple", False), (dict(num_q_heads=32), "GQA group 16", True),
    (dict(head_dim=32), "head_dim=32", True), (dict(dtype=3), "dtype=3", True), (dict(max_blocks=0), "max_blocks=0", False),
    (dict(budget=0, keep_first=0), "budget=0", False), (dict(keep_last=0), "keep_last=0", False),
    (dict(keep_first=-1), "keep_first=-1", False), (dict(keep_first=2, keep_last=3), "budget=4", False),
    (dict(bounds=None), "NULL", False), (dict(q=FAKE + 2), "16-byte", False), (dict(q_stride=12), "q_stride", False),
    (dict(pages=FAKE + 1), "misaligned", False)])
def test_select_refusals(kw, what, unsupported):
    refused("tq_select_pages", select_args(**kw), what, tq.TQ_ERR_UNSUPPORTED if unsupported else tq.TQ_ERR_INVALID_ARG)


@pytest.mark.parametrize("kw,what,unsupported", [
    (dict(num_kv_heads=0), "num_kv_heads", False), (dict(num_q_heads=18), "GQA group 9", True),
    (dict(head_dim=192), "head_dim=192", True), (dict(dtype=tq.TQ_F32), "dtype=1", True), (dict(num_pages=-1), "num_pages=-1", False),
    (dict(max_blocks=0), "max_blocks=0", False), (dict(selected=2), "selected=2", False), (dict(out=None), "NULL", False),
    (dict(workspace=None), "workspace of", False), (dict(workspace_bytes=64), "workspace of", False),
    (dict(k_pool=FAKE + 8), "16-byte", False), (dict(seq_lens=FAKE + 2), "4-byte", False), (dict(q_stride=4), "q_stride", False),
    (dict(k_page_stride=32 * 128 - 8), "page strides", False), (dict(selected=1, v_page_stride=64 * 128), "contiguous", False)])
def test_attend_pages_refusals(kw, what, unsupported):
    refused("tq_attend_pages", attend_args(**kw), what, tq.TQ_ERR_UNSUPPORTED if unsupported else tq.TQ_ERR_INVALID_ARG)


def test_null_arguments():
    for fn in ("tq_plan_pages", "tq_append_pages", "tq_select_pages", "tq_attend_pages"):
        assert getattr(tq.LIB, fn)(None, None) == tq.TQ_ERR_INVALID_ARG
        assert b"args is NULL" in tq.LIB.tq_last_error()
    assert tq.LIB.tq_attend_pages_workspace_bytes(ctypes.byref(attend_args()), None) == tq.TQ_ERR_INVALID_ARG


@pytest.mark.parametrize("d", [64, 128, 256])
def test_workspace_stays_small(d):
    nb = ctypes.c_size_t()
    for kw in (dict(batch=1, max_blocks=1), dict(batch=64, max_blocks=256), dict(batch=1, num_kv_heads=1, max_blocks=1 << 20)):
        a = attend_args(head_dim=d, **kw)
        assert tq.LIB.tq_attend_pages_workspace_bytes(ctypes.byref(a), ctypes.byref(nb)) == tq.TQ_OK
        assert (kw["max_blocks"] > 32) == (nb.value > 0) and nb.value <= 8 << 20


def test_binding_checks_tensors():
    cpu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="new_lens"):
        tq.plan_pages(cpu, cpu, cpu, cpu, cpu, num_kv_heads=1, max_tokens=4)
    with pytest.raises(TypeError, match="k must"):
        tq.append_pages(torch.zeros(1, 1, 64, dtype=torch.float16), None, cpu)
    with pytest.raises(TypeError, match="q must"):
        tq.select_pages(torch.zeros(1, 1, 64), torch.zeros(1, 1, 2, 64), cpu, cpu, budget=4)
    with pytest.raises(TypeError, match="q must"):
        tq.attend_pages(torch.zeros(1, 1, 64, dtype=torch.float16), cpu, cpu, cpu, cpu, workspace=cpu)
    with pytest.raises(TypeError, match="k must be a tensor, got list"):
        tq.append_pages([1], None, cpu)
    with pytest.raises(TypeError, match="expected 12 arguments"):
        tq._bind.plan_pages(cpu)


# ------------------------------------------------------------------------------ the plain implementations

def test_plan_by_hand():
    # pages of 16: request 0 has 10 tokens and adds 7 (one page), 1 is finished (two pages back), 2 adds 20 (two pages, one
    # too many), 3 adds 2 without a page
    got = po.plan([7, -1, 20, 2], [10, 17, 0, 3], np.array([[5, -1], [2, 7], [-1, -1], [4, -1]]), np.array([0, 1, 9, 9, 9, 9]),
                  [0, 2], 1, 30)
    assert got["table"].tolist() == [[5, 0], [2, 7], [-1, -1], [4, -1]]
    assert got["row_start"].tolist() == [0, 7, 7, 27, 29] and got["start_pos"].tolist() == [10, -1, -1, 3]
    assert got["seq_lens"].tolist() == [17, 0, 0, 5] and got["free_state"].tolist() == [1, 3]
    assert got["ring"].tolist() == [0, 1, 2, 7, 9, 9]
    assert got["slots"].tolist() == [5 * 16 + t for t in range(10, 16)] + [0] + [-1] * 20 + [4 * 16 + 3, 4 * 16 + 4] + [-1]


def test_append_by_hand():
    d = 64
    k = np.arange(3 * d, dtype=np.float64).reshape(3, 1, d)
    bounds = np.stack((np.full((2, 1, d), 50.0), np.full((2, 1, d), 60.0)), 2)
    pool, _, near = po.append(k, None, [15, 16, -1], np.zeros((2, 1, 16, d)), None, bounds)
    assert np.array_equal(pool[0, 0, 15], k[0, 0]) and np.array_equal(pool[1, 0, 0], k[1, 0]) and pool.sum() == k[:2].sum()
    assert np.array_equal(near[0, 0], [np.minimum(k[0, 0], 50), np.maximum(k[0, 0], 60)])      # the page had tokens
    assert np.array_equal(near[1, 0], [k[1, 0], k[1, 0]])                                      # a new page


def test_scores_bound_every_key_of_a_page():
    rng = np.random.default_rng(0)
    keys, q = rng.standard_normal((20, 16, 64)).astype(np.float16), rng.standard_normal((3, 64)).astype(np.float16)
    scores = po.page_scores(q, keys.min(1), keys.max(1)).astype(np.float64)
    exact = np.einsum("ntc,gc->ngt", keys.astype(np.float64), q.astype(np.float64)).max((1, 2))
    assert np.all(scores >= exact - 64 * 2.0 ** -24 * 200)
    wide = sum(np.maximum(q[:, None, c].astype(np.float64) * keys.min(1)[None, :, c], q[:, None, c].astype(np.float64) *
                          keys.max(1)[None, :, c]) for c in range(64)).max(0)
    assert np.all(np.abs(scores - wide) <= 64 * 2.0 ** -24 * 200)          # 64 roundings of sums below 200


def test_select_and_attend_by_hand():
    bounds = np.zeros((6, 1, 2, 64), dtype=np.float32)
    bounds[:, 0, :, 0] = np.array([[0, 1], [5, 6], [5, 6], [7, 8], [0, 2], [0, 0]])
    q = np.zeros((1, 1, 64), dtype=np.float32)
    q[0, 0, 0] = 1
    pages, lens = po.select(q, bounds, np.array([[5, 4, 2, 1, 3, 0]]), [85], 4, 1, 1)
    assert pages.tolist() == [[[5, 2, 3, 0]]] and lens.tolist() == [[53]]   # page 2 before its equal, page 1
    k, v = np.zeros((2, 1, 16, 64)), np.ones((2, 1, 16, 64))
    k[1, 0, 0, 0], v[1, 0, 0] = np.log(3.0), 5.0
    out, err = po.attend(np.array(q, dtype=np.float64), k, v, np.array([[0, 1]]), [17], 1.0)
    assert np.allclose(out, (16 * 1 + 3 * 5) / 19) and err.max() < 1e-3
    assert not po.attend(np.array(q, dtype=np.float64), k, v, np.array([[0, 1]]), [0], 1.0)[0].any()


def test_kernels_that_start_early_load_coherently():
    """The paged cache's kernels are resident while the work before them still writes what they read: none of their loads is a
    non-coherent one (__ldg, ld.global.nc, or a const __restrict__ pointer, which the compiler may load that way)."""
    import os
    with open(os.path.join(os.path.dirname(tq.__file__), "csrc", "tq_pages_kernels.cuh")) as f:
        text = f.read()
    assert "griddepcontrol.wait" in text
    for what in ("__ldg(", ".nc.", "__restrict__"):
        assert what not in text, what


@pytest.mark.parametrize("d,n", [(64, 200), (128, 1800), (256, 700)])
@pytest.mark.parametrize("kind,terms,passes", [("fp16", 1, False), ("fp16", 2, True), ("bf16", 2, False), ("bf16", 3, True)])
def test_row_tolerance_tells_the_weights_apart(d, n, kind, terms, passes):
    """Weights of one term too few (11 or 16 bits) miss the tolerance of attention over uncompressed pages, the kernels' own do
    not come near it."""
    rng = np.random.default_rng(d + n)
    got, want = [], []
    for _ in range(8):
        q, k, v = (rng.standard_normal(s).astype(np.float16).astype(np.float64) for s in ((d,), (n, d), (n, d)))
        s = k @ q / np.sqrt(d) * np.log2(np.e)
        p = np.exp2(s - s.max() + 12)
        rest, weights = p.astype(np.float32), np.zeros(n)
        for _ in range(terms):
            if kind == "fp16":
                term = rest.astype(np.float16).astype(np.float32)
            else:
                term = (rest.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
            weights += term
            rest = rest - term
        got.append(weights @ v / p.sum())
        want.append(p @ v / p.sum())
    err = po.row_error(np.stack(got), np.stack(want)).max()
    assert err <= po.ROW_RTOL / 10 if passes else err > 2 * po.ROW_RTOL


def test_compressed_attention_takes_as_many_sequences_as_a_grid():
    """B * H_kv lists of a selection are sequences of one kv head to compressed attention, whose grid holds 65535."""
    a, nb = tq.AttendArgs(), ctypes.c_size_t()
    a.batch, a.num_q_heads, a.num_kv_heads, a.head_dim, a.v_bits, a.v_group = 65535, 4, 1, 128, 4, 32
    a.max_seq_len = 64
    assert tq.LIB.tq_attend_workspace_bytes(ctypes.byref(a), ctypes.byref(nb)) == tq.TQ_OK
    a.batch = 65536
    assert tq.LIB.tq_attend_workspace_bytes(ctypes.byref(a), ctypes.byref(nb)) == tq.TQ_ERR_UNSUPPORTED
    assert b"65535" in tq.LIB.tq_last_error()
