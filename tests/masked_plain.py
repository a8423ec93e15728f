"""Plain fp64 forms of the masks (sinks, drafted trees), and inputs for their
tests.  Written from the definitions in include/fa_gb300.h, on the CPU."""
import math
import random

import torch

import paged_plain as plain


def random_parents(n, seed, roots=0.05, chain=0.3):
    """Parents of a tree of n nodes: some follow the node before, some any."""
    rng = random.Random(seed)
    out = []
    for i in range(n):
        if i == 0 or rng.random() < roots:
            out.append(-1)
        elif rng.random() < chain:
            out.append(i - 1)
        else:
            out.append(rng.randrange(i))
    return out


def path_of(parents, i):
    """Node i and its ancestors."""
    path = [i]
    while 0 <= parents[path[-1]] < path[-1]:
        path.append(parents[path[-1]])
    return path


def words_of(nodes, words):
    """A mask's words (as signed 32-bit numbers) that name `nodes`."""
    row = [0] * words
    for p in nodes:
        if p < 32 * words:
            row[p // 32] |= 1 << (p % 32)
    return [w - (1 << 32) if w >> 31 else w for w in row]


def tree_masks(trees, words):
    """int32 [nodes of all trees, words]."""
    rows = [words_of(path_of(t, i), words) for t in trees for i in range(len(t))]
    return torch.tensor(rows, dtype=torch.int32).reshape(-1, words)


def named(row, p):
    """Whether bit p of a mask row (signed words) is set."""
    return p < 32 * len(row) and bool((row[p // 32] >> (p % 32)) & 1)


def seen_keys(i, n, length, keys, causal, wl, wr, sinks, row=None):
    """Truth values of the `keys` first keys for row i of n at bottom-right
    position length - n + i, or for node i of a tree with mask `row`."""
    j = torch.arange(keys)
    ctx = length - n
    if row is not None:
        depth = max(sum(bin(w & 0xFFFFFFFF).count("1") for w in row) - 1, 0)
        at = ctx + depth
        seen = torch.ones(keys, dtype=torch.bool)
        if wl >= 0:
            seen = (j >= at - wl) | (j < sinks)
        for x in range(max(ctx, 0), keys):
            seen[x] = named(row, x - ctx)
        return seen
    at = ctx + i
    seen = torch.ones(keys, dtype=torch.bool)
    if causal:
        seen &= j <= at
    elif wr >= 0:
        seen &= j <= at + wr
    if wl >= 0:
        seen &= (j >= at - wl) | (j < sinks)
    return seen


def attend(row, k, v, seen, scale):
    """(O, LSE, sum p |v|, largest scale * sum |q k|) of one row over keys."""
    d = v.shape[1]
    if not seen.any():
        zero = torch.zeros(d, dtype=torch.float64)
        return zero, -math.inf, zero, 0.0
    row = row.double()
    x = k[seen] @ row * scale
    top = x.max()
    p = torch.exp(x - top)
    return (p @ v[seen] / p.sum(), top + torch.log(p.sum()), p @ v[seen].abs() / p.sum(),
            (k[seen].abs() @ row.abs()).max() * scale)


def paged_attention(q, kc, vc, ks, vs, cu, lens, pages, scale, causal=True, window=-1, sinks=0,
                    mask=None):
    """As paged_plain.attention, with the masks."""
    T, H, d = q.shape
    hks = kc.shape[1]
    o = torch.zeros((T, H, d), dtype=torch.float64)
    w = torch.zeros((T, H, d), dtype=torch.float64)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    big = torch.zeros((H, T), dtype=torch.float64)
    rows = None if mask is None else mask.tolist()
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        keys = min(max(length, 0), pages.shape[1] * 64)
        if n <= 0 or keys == 0:
            continue
        seen = [seen_keys(i, n, length, keys, causal, window, -1, sinks,
                          None if rows is None else rows[cu[b] + i]) for i in range(n)]
        for hk in range(hks):
            k, held = plain.keys_of(b, keys, pages, kc, ks, hk)
            v, _ = plain.keys_of(b, keys, pages, vc, vs, hk)
            for i in range(n):
                for h in range(hk * (H // hks), (hk + 1) * (H // hks)):
                    t = cu[b] + i
                    o[t, h], lse[h, t], w[t, h], big[h, t] = attend(q[t, h], k, v, seen[i] & held,
                                                                    scale)
    return o, lse, w, big


def key_weights(q, lse, kc, ks, cu, lens, pages, sums, scale, causal=True, window=-1, sinks=0,
                decay=1.0):
    """(sums, tolerance) after the call, fp64; sums [batch, Hk, capacity].  A
    weight's exponent is off by the score's dx = 2^-15 A, A = scale * sum |q k|,
    and 2^-20 of the score and the LSE; each sum of R weights by (R + 8) 2^-23."""
    T, H, d = q.shape
    hks, cap = sums.shape[1:]
    out, tol = sums.double().clone(), torch.zeros_like(sums, dtype=torch.float64)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        keys = min(max(length, 0), pages.shape[1] * 64, cap)
        if n <= 0 or keys == 0:
            continue
        old = out[b, :, :keys] * decay if decay else torch.zeros((hks, keys), dtype=torch.float64)
        old[:, max(length - n, 0):] = 0
        out[b, :, :keys] = old
        tol[b, :, :keys] = old.abs() * 2.0 ** -22
        for hk in range(hks):
            k, held = plain.keys_of(b, keys, pages, kc, ks, hk)
            for i in range(n):
                seen = seen_keys(i, n, length, keys, causal, window, -1, sinks) & held
                for h in range(hk * (H // hks), (hk + 1) * (H // hks)):
                    row, l = q[cu[b] + i, h].double(), lse[h, cu[b] + i].double()
                    if l == -math.inf or not seen.any():
                        continue
                    x = k[seen] @ row * scale
                    p = torch.exp(x - l)
                    dx = 2.0 ** -15 * scale * (k[seen].abs() @ row.abs())
                    err = 1.1 * dx + 2.0 ** -20 * (x.abs() + l.abs())
                    out[b, hk, :keys][seen] += p
                    tol[b, hk, :keys][seen] += p * (err + (n * (H // hks) + 8) * 2.0 ** -23)
    return out, tol + 1e-37


def select(sums, lens, budget, sinks, recent):
    """(keep, new lengths), by sorting."""
    batch, hk, cap = sums.shape
    keep = torch.full((batch, hk, budget), -1, dtype=torch.int32)
    new = []
    for b, n in enumerate(lens):
        n = min(max(n, 0), cap)
        new.append(min(n, budget))
        for h in range(hk):
            if n <= budget:
                kept = list(range(n))
            else:
                x = [-math.inf if v != v else v for v in sums[b, h, :n].tolist()]
                nan = [v != v for v in sums[b, h, :n].tolist()]
                order = sorted(range(sinks, n - recent), key=lambda j: (nan[j], -x[j], j))
                kept = sorted(list(range(sinks)) + list(range(n - recent, n))
                              + order[:budget - sinks - recent])
            keep[b, h, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
    return keep, torch.tensor(new, dtype=torch.int32)


def compact(codes, scale, pages, keep, first, counts):
    """fp64 codes and scales after the move, page by page from the values
    before it; codes [pages, Hk, 64, d] fp64 (NaN codes as NaN)."""
    num, hks, _, d = codes.shape
    was, factor = codes.clone(), scale.clone()
    codes, scale = codes.clone(), scale.clone()
    width = pages.shape[1]
    for b in range(pages.shape[0]):
        f = max(int(first[b]), 0)
        n = min(max(int(counts[b]), 0), keep.shape[2], max(width * 64 - f, 0))
        for h in range(hks):
            src = keep[b, h if keep.shape[1] > 1 else 0].tolist()
            slot = f
            while slot < f + n:
                off, m = slot % 64, min(64 - slot % 64, f + n - slot)
                page = int(pages[b, slot // 64])
                rows = torch.zeros((m, d), dtype=torch.float64)
                moved = False
                for i in range(m):
                    s = src[slot - f + i]
                    moved |= s != slot + i
                    if s < slot + i or s >= width * 64:
                        continue
                    p = int(pages[b, s // 64])
                    if 0 <= p < num:
                        rows[i] = was[p, h, s % 64] * factor[p, h]
                if moved and 0 <= page < num:
                    mag = torch.where(torch.isnan(rows), 0.0, rows.abs())
                    new = plain.page_scale(mag.amax())
                    if off:
                        new = torch.maximum(new, factor[page, h])
                        if new > factor[page, h]:
                            codes[page, h, :off] = plain.e4m3(was[page, h, :off] * factor[page, h] / new)
                    codes[page, h, off:off + m] = plain.e4m3(rows / new)
                    scale[page, h] = new
                slot += m
    return codes, scale


def move_weights(sums, keep, first, counts, pages, num):
    """Sums after the move; a row of zeros (an entry that names no slot at its
    own or behind it, on a page of the cache) has 0."""
    out = sums.clone()
    batch, hks, cap = sums.shape
    slots = pages.shape[1] * 64
    for b in range(batch):
        f = max(int(first[b]), 0)
        n = min(max(int(counts[b]), 0), keep.shape[2], max(slots - f, 0))
        for h in range(hks):
            src = keep[b, h if keep.shape[1] > 1 else 0].tolist()
            for p0 in range(f // 64 * 64, f + n, 64):
                at = [d for d in range(max(p0, f), min(p0 + 64, f + n))]
                if all(src[d - f] == d for d in at):
                    continue
                for d in at:
                    if d < cap:
                        s = src[d - f]
                        here = d <= s < min(cap, slots) and 0 <= int(pages[b, s // 64]) < num
                        out[b, h, d] = sums[b, h, s] if here else 0.0
    return out
