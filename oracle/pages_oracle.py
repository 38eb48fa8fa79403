"""The paged cache's operators, plainly: planning, append with page bounds, page selection, attention over pages.

Loops over requests, tokens and pages in numpy; 64-bit arithmetic, except the selection score, whose 32-bit sums and
their order are the operator's definition.  Test infrastructure only; shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np

PAGE = 16


def plan(new_lens, seq_lens, table, ring, state, heads, max_tokens):
    """tq_plan_pages by its rules, one request after the other.  Returns a dict of the outputs; table and ring are
    copies."""
    table, ring = table.copy(), ring.copy()
    num_pages, width = len(ring), table.shape[1]
    head, count = int(state[0]), int(state[1])
    slots = np.full((max_tokens, heads), -1, dtype=np.int64)
    row_start, start_pos, lens_out = [0], [], []
    asked = taken = 0                                   # pages asked for by requests that fit; pages handed out
    given_back = []
    for b, new in enumerate(int(x) for x in new_lens):
        length = min(max(int(seq_lens[b]), 0), width * PAGE)
        req = max(new, 0)
        row_start.append(row_start[-1] + req)
        have = -(-length // PAGE)
        if new < 0:
            given_back += [int(x) for x in table[b, :have]]
            start_pos.append(-1)
            lens_out.append(0)
            continue
        need = -(-(length + req) // PAGE) - have
        fits = length + req <= width * PAGE and row_start[-1] <= max_tokens
        asked += need if fits else 0
        if not fits or (need and asked > count):
            start_pos.append(-1)
            lens_out.append(length)
            continue
        for j in range(need):
            table[b, have + j] = ring[(head + taken) % num_pages]
            taken += 1
        for i in range(req):
            t = length + i
            page = int(table[b, t // PAGE])
            if 0 <= page < num_pages:
                for h in range(heads):
                    slots[row_start[b] + i, h] = (page * heads + h) * PAGE + t % PAGE
        start_pos.append(length)
        lens_out.append(length + req)
    for i, page in enumerate(given_back):
        ring[(head + count + i) % num_pages] = page
    return dict(table=table, ring=ring, slots=slots.reshape(-1), row_start=np.minimum(row_start, 2**31 - 1), start_pos=np.array(start_pos),
                seq_lens=np.array(lens_out),
                free_state=np.array([(head + taken) % num_pages, count - taken + len(given_back)]))


def append(k, v, slots, k_pool, v_pool, bounds):
    """tq_append_pages: k, v [N, H, d]; pools [P, H, 16, d], bounds [P, H, 2, d], any of the three None.  float64 in and
    out (copies)."""
    n, h, d = k.shape
    outs = [None if t is None else t.copy() for t in (k_pool, v_pool, bounds)]
    some = next(t for t in outs if t is not None)
    rows = some.shape[0] * h * PAGE
    touched = {}
    for t in range(n):
        for j in range(h):
            s = int(slots[t * h + j])
            if not 0 <= s < rows:
                continue
            if outs[0] is not None:
                outs[0].reshape(-1, d)[s] = k[t, j]
            if outs[1] is not None:
                outs[1].reshape(-1, d)[s] = v[t, j]
            touched.setdefault(s // PAGE, []).append((s % PAGE, t, j))
    if outs[2] is not None:
        flat = outs[2].reshape(-1, 2, d)
        for e, items in touched.items():
            keys = np.stack([k[t, j] for _, t, j in items])
            lo, hi = keys.min(0), keys.max(0)
            if all(off for off, _, _ in items):         # the page had tokens before
                lo, hi = np.minimum(lo, flat[e, 0]), np.maximum(hi, flat[e, 1])
            flat[e, 0], flat[e, 1] = lo, hi
    return outs


def page_scores(q, lo, hi):
    """Scores of pages [n, d] for the query heads [G, d] of one kv head, in the operator's 32-bit order: the even and
    the odd channels of every 8 in turn, the two together, then the upper half of the sums onto the lower."""
    q, lo, hi = (np.asarray(x, dtype=np.float32) for x in (q, lo, hi))
    best = np.full(lo.shape[0], -np.inf, dtype=np.float32)
    bad = np.zeros(lo.shape[0], dtype=bool)
    for row in q:
        terms = np.maximum(row * lo, row * hi).reshape(lo.shape[0], -1, 8)
        even, odd = terms[:, :, 0].copy(), terms[:, :, 1].copy()
        for i in (2, 4, 6):
            even += terms[:, :, i]
            odd += terms[:, :, i + 1]
        sums = even + odd
        while sums.shape[1] > 1:
            half = sums.shape[1] // 2
            sums = sums[:, :half] + sums[:, half:]
        bad |= np.isnan(sums[:, 0])
        best = np.fmax(best, sums[:, 0])
    best[bad] = np.nan
    return best


def select(q, bounds, table, seq_lens, budget, keep_first, keep_last):
    """tq_select_pages: q [B, Hq, d], bounds [P, H, 2, d]; returns (pages [B, H, budget], lens [B, H])."""
    b, hq, _ = q.shape
    num, h = bounds.shape[:2]
    g = hq // h
    pages = np.full((b, h, budget), -1, dtype=np.int64)
    lens = np.zeros((b, h), dtype=np.int64)
    for i in range(b):
        length = min(max(int(seq_lens[i]), 0), table.shape[1] * PAGE)
        n = -(-length // PAGE)
        ids = table[i, :n].astype(np.int64)
        ok = (ids >= 0) & (ids < num)
        for j in range(h):
            kept = np.arange(n)
            if n > budget:
                near = bounds[np.where(ok, ids, 0), j]
                score = page_scores(q[i, j * g:(j + 1) * g], near[:, 0], near[:, 1]).astype(np.float64)
                last = ~ok | np.isnan(score)             # these rank behind every number
                score[last] = 0.0
                forced = (np.arange(n) < keep_first) | (np.arange(n) >= n - keep_last)
                order = sorted(range(n), key=lambda x: (not forced[x], last[x], -score[x], x))
                kept = np.sort(np.array(order[:budget]))
            pages[i, j, :len(kept)] = np.where(ok[kept], ids[kept] * h + j, -1)
            lens[i, j] = length if n <= budget else length - (n - budget) * PAGE
    return pages, lens


def attend(q, k_pool, v_pool, table, seq_lens, scale, selected=False):
    """Attention over pages in 64 bits: q [B, Hq, d], pools [P, H, 16, d] float64.  Returns (out [B, Hq, d], a bound of
    the error that 32-bit sums may make in each output row, [B, Hq])."""
    b, hq, d = q.shape
    num, h = k_pool.shape[:2]
    g = hq // h
    out, err = np.zeros((b, hq, d)), np.zeros((b, hq))
    for i in range(b):
        for j in range(h):
            row = table[i, j] if selected else table[i]
            length = int(seq_lens[i, j] if selected else seq_lens[i])
            length = min(max(length, 0), len(row) * PAGE)
            keys, values = [], []
            for t in range(length):
                e = int(row[t // PAGE])
                page, head = (e // h, e % h) if selected else (e, j)
                if e < 0 or page >= num:
                    continue
                keys.append(k_pool[page, head, t % PAGE])
                values.append(v_pool[page, head, t % PAGE])
            if not keys:
                continue
            keys, values = np.stack(keys), np.stack(values)
            for x in range(g):
                qv = q[i, j * g + x]
                s = scale * (keys @ qv)
                p = np.exp(s - s.max())
                out[i, j * g + x] = p @ values / p.sum()
                # a logit: d products added in 32 bits (two roundings each allowed), times the scale, minus the
                # maximum; the exponential and the 16-bit terms of a weight: 2^-20; sums over the tokens, 16 at a time
                logit = abs(scale) * np.abs(keys * qv).sum(1).max() * (2 * d) * 2.0 ** -24 + np.abs(s).max() * 2.0 ** -21
                sums = 2 * (len(keys) / 16 + 64) * 2.0 ** -23
                err[i, j * g + x] = np.abs(values).max() * (2 * logit + 2.0 ** -20 + sums)
    return out, err


# Relative L2 error of an attention output row (row_error) that 32-bit arithmetic stays below on ordinary inputs: queries, keys and
# values of about unit normal entries, at most 256 channels, scale d^-0.5.  A row is sum p_t v_t / sum p_t with values of random
# signs, so an error e_t of the t-th weight, relative to it, comes out as the root mean square of the e_t weighted with p_t^2.
# Their parts, per weight:
#   the logit: at most 256 / 16 steps of sums cut off behind 24 bits, each below 2^-23 of a partial sum that stays around
#     sqrt(d) / 2 times the scale: 16 * 2^-24 on average with one sign, 1.0e-6; in two chains half of it, 0.5e-6
#   its scaling and the subtraction of the maximum, of numbers up to 8: 2 * 2^-24 * 8 / sqrt(3), 0.6e-6
#   the exponential, 2^-22: 0.2e-6; two fp16 or three bf16 terms of a weight, 2^-23: 0.1e-6
#   the sums over tokens and their join, rounded in 32 bits: 16 tokens at a time, 2^-24 sqrt(300): 1.0e-6
# together (adding up) 2.4e-6.  Weights of 11 bits are off by 2^-12 / sqrt(3) = 1.4e-4, of 16 bits, cut off, by up to 2^-16 = 1.5e-5.
ROW_RTOL = 3e-6


def row_error(got, want):
    """Relative L2 error of each output row [..., d] (0 where both rows are zero)."""
    size = np.linalg.norm(want, axis=-1)
    return np.linalg.norm(got - want, axis=-1) / np.where(size == 0, 1, size)
