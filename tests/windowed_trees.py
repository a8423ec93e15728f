"""Attention of drafted trees as decoding each path token by token would have it,
written from that definition in fp64."""
import torch

import masked_plain as masked
import paged_plain as plain


def path_keys(parents, i, ctx, window, sinks):
    """Slots that node i sees: its path, root first, stands behind the ctx keys of
    the context, each at the next position, and the last one decodes."""
    slots = list(range(ctx)) + [ctx + p for p in masked.path_of(parents, i)[::-1]]
    at = len(slots) - 1
    return [s for position, s in enumerate(slots)
            if window < 0 or position >= at - window or position < sinks]


def windowed_masks(trees, ctxs, words, window, sinks):
    """int32 [nodes of all trees, words]: the nodes among each one's slots."""
    rows = [masked.words_of([s - ctx for s in path_keys(t, i, ctx, window, sinks) if s >= ctx], words)
            for t, ctx in zip(trees, ctxs) for i in range(len(t))]
    return torch.tensor(rows, dtype=torch.int32).reshape(-1, words)


def decoded(q, trees, ctxs, keys, scale, window, sinks):
    """(O, LSE [H, T], sum p |v|, scale sum |q k|) of every node; keys(b, hk) gives
    the fp64 K and V of a sequence's slots."""
    T, H, d = q.shape
    o, lse, w, big = None, torch.zeros((H, T), dtype=torch.float64), None, None
    t = 0
    for b, (tree, ctx) in enumerate(zip(trees, ctxs)):
        for i in range(len(tree)):
            slots = torch.tensor(path_keys(tree, i, ctx, window, sinks))
            for h in range(H):
                k, v = keys(b, h)
                if o is None:
                    o = torch.zeros((T, H, v.shape[1]), dtype=torch.float64)
                    w, big = o.clone(), lse.clone()
                seen = torch.ones(len(slots), dtype=torch.bool)
                o[t, h], lse[h, t], w[t, h], big[h, t] = masked.attend(q[t, h], k[slots], v[slots],
                                                                       seen, scale)
            t += 1
    return o, lse, w, big


def cached(pages, kc, ks, vc, vs, lens, group):
    """keys() of a paged cache."""
    held = {}

    def keys(b, h):
        if (b, h // group) not in held:
            held[b, h // group] = tuple(plain.keys_of(b, lens[b], pages, c, s, h // group)[0]
                                        for c, s in ((kc, ks), (vc, vs)))
        return held[b, h // group]
    return keys
