"""Measured cases of the masks and the eviction of the paged 8-bit cache:

  tree     a tree of drafted tokens: its ancestor masks and positions from the
           parents, then attention of all its nodes over the cache
  sink     decode attention with a sliding window and the first tokens of each
           sequence, which stay visible
  prompt   the same mask in the packed prompt forward
  weights  attention weights of a step's rows, summed for each key and kv head
  evict    the keys to keep by those sums, and the cache moved together in place
  commit   the accepted path of each drafted tree moved behind its context

`run` computes them in plain fp32 torch, or, with `own` set, through the
library's entry points.  `exact` computes them from their definition in fp64.

Shapes: head counts and head dims of the repository's workloads (32 query
heads over 8 or 4, head dims 64 to 128, 128 heads of 192 / 128), contexts up
to 32768 tokens, prompts of about 4096 with windows of 1024.  Inputs are
normal, with one channel in 16 of the cached keys eight times larger, as keys
of trained models have.
"""
import math
import random

import torch

own = False

PAGE = 64
E4M3_MAX = 448.0
NEG = float("-inf")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One request whose draft model proposes 16 tokens: latency counts.
        dict(name="tree one 16", op="tree", batch=1, q_lo=16, q_hi=16, len_lo=4112, len_hi=4112,
             heads=32, heads_k=8, dim=128, window=-1, sinks=0),
        # A batch of requests with large trees.
        dict(name="tree 24 x 33-64", op="tree", batch=24, q_lo=33, q_hi=64, len_lo=517,
             len_hi=5000, heads=32, heads_k=8, dim=128, window=-1, sinks=0),
        # Small ragged trees in a sliding window with sinks.
        dict(name="tree d64 window", op="tree", batch=32, q_lo=3, q_hi=24, len_lo=100, len_hi=8192,
             heads=32, heads_k=4, dim=64, window=1024, sinks=4),
        # A decode step of a mixed batch, the window shorter than most contexts.
        dict(name="sink step 64", op="sink", batch=64, q_lo=1, q_hi=1, len_lo=100, len_hi=16384,
             heads=32, heads_k=4, dim=128, window=4095, sinks=4),
        # Long windows: the rate at which the cache streams.
        dict(name="sink long 32x32768", op="sink", batch=32, q_lo=1, q_hi=1, len_lo=30001,
             len_hi=32768, heads=32, heads_k=8, dim=128, window=16383, sinks=70),
        # Prompts of a model with a sliding window, grouped heads.
        dict(name="prompt 4x4096", op="prompt", batch=4, q_lo=3900, q_hi=4096, len_lo=3900,
             len_hi=4096, heads=32, heads_k=8, dim=128, dim_v=128, window=1024, sinks=4),
        # The latent-attention prefill shape, ragged.
        dict(name="prompt d192 ragged", op="prompt", batch=5, q_lo=1, q_hi=4001, len_lo=1001,
             len_hi=4001, heads=128, heads_k=128, dim=192, dim_v=128, window=1023, sinks=130),
        # Weights of one decode step of a mixed batch, added to the sums so far.
        dict(name="weights step 64", op="weights", batch=64, q_lo=1, q_hi=1, len_lo=100,
             len_hi=8192, heads=32, heads_k=4, dim=128, window=-1, sinks=0, decay=1.0),
        # The last rows of long prompts look back once, for the first eviction.
        dict(name="weights prompt end", op="weights", batch=4, q_lo=32, q_hi=32, len_lo=20001,
             len_hi=32768, heads=32, heads_k=8, dim=128, window=-1, sinks=0, decay=0.0),
        # A batch whose caches are cut to a quarter.
        dict(name="evict 64 x 8192", op="evict", batch=64, len_lo=1000, len_hi=8192, heads_k=8,
             dim=128, budget=2048, sinks=4, recent=256),
        # One long context cut down, odd sizes.
        dict(name="evict one 32768", op="evict", batch=1, len_lo=32768, len_hi=32768, heads_k=8,
             dim=96, budget=4097, sinks=1, recent=100),
        # After a step of the second tree case: paths of one to six tokens stay.
        dict(name="commit 24 trees", op="commit", batch=24, q_lo=33, q_hi=64, len_lo=517,
             len_hi=5000, heads_k=8, dim=128, most=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "sink", "prompt", "weights", "evict", "commit"))
    dim = rng.choice((64, 80, 96, 128))
    heads_k = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 3, 4, 8))
    window = rng.choice((-1, _log(rng, 16, 8192)))
    sinks = rng.choice((0, 1, 4, 64, 131))
    if op == "tree":
        batch = _log(rng, 1, 48)
        hi = min(16384, _log(rng, 80, (1 << 17) // batch))
        q_hi = _log(rng, 2, max(2, min(64, 4096 // (batch * group))))
        return dict(op=op, batch=batch, q_lo=rng.choice((1, q_hi)), q_hi=q_hi,
                    len_lo=max(q_hi, rng.choice((hi // 8, hi))), len_hi=max(q_hi, hi),
                    heads=heads_k * group, heads_k=heads_k, dim=dim, window=window, sinks=sinks)
    if op == "sink":
        batch = _log(rng, 1, 128)
        hi = min(32768, _log(rng, 1, (1 << 20) // batch))
        return dict(op=op, batch=batch, q_lo=1, q_hi=min(hi, rng.choice((1, 1, 4))),
                    len_lo=max(4, rng.choice((hi // 8, hi))), len_hi=max(4, hi),
                    heads=heads_k * group, heads_k=heads_k, dim=dim,
                    window=_log(rng, 1, max(2, hi)), sinks=sinks)
    if op == "prompt":
        batch = _log(rng, 1, 24)
        hi = _log(rng, 1, min(4096, 16384 // batch))
        dim = rng.choice((64, 72, 80, 96, 128, 192))
        if dim == 192:
            group = 1
        ctx = rng.choice((0, _log(rng, 1, 2048)))
        return dict(op=op, batch=batch, q_lo=rng.choice((1, hi)), q_hi=hi,
                    len_lo=hi + rng.choice((0, ctx)), len_hi=hi + ctx, heads=heads_k * group,
                    heads_k=heads_k, dim=dim, dim_v=min(dim, 128), window=_log(rng, 1, 2048),
                    sinks=sinks)
    if op == "weights":
        batch = _log(rng, 1, 64)
        hi = min(32768, _log(rng, 64, (1 << 18) // batch))
        q_hi = rng.choice((1, 1, 4, 16, 32))
        return dict(op=op, batch=batch, q_lo=rng.choice((1, q_hi)), q_hi=q_hi,
                    len_lo=max(q_hi, rng.choice((hi // 8, hi))), len_hi=max(q_hi, hi),
                    heads=heads_k * group, heads_k=heads_k, dim=dim, window=window, sinks=sinks,
                    decay=rng.choice((0.0, 0.5, 1.0)))
    if op == "evict":
        batch = _log(rng, 1, 64)
        hi = min(32768, _log(rng, 16, (1 << 19) // batch))
        budget = _log(rng, 8, hi)
        sinks = min(sinks, budget // 4)
        return dict(op=op, batch=batch, len_lo=rng.choice((1, hi // 2, hi)), len_hi=hi,
                    heads_k=heads_k, dim=dim, budget=budget, sinks=sinks,
                    recent=rng.randint(0, budget // 2))
    batch = _log(rng, 1, 64)
    hi = min(16384, _log(rng, 80, (1 << 18) // batch))
    return dict(op=op, batch=batch, q_lo=1, q_hi=rng.randint(2, 64), len_lo=64, len_hi=hi,
                heads_k=heads_k, dim=dim, most=rng.randint(1, 12))


def _spread(lo, hi, n, phase=0.0):
    """n whole numbers in [lo, hi], both ends among them where n allows, in no order."""
    if n == 1:
        return [hi]
    mixed = sorted(range(n), key=lambda i: (i * 0.6180339887498949 + phase) % 1.0)
    return [lo + (hi - lo) * i // (n - 1) for i in mixed]


def _lengths(case):
    """(query rows, length with them) of each sequence."""
    n = case["batch"]
    lens = _spread(case["len_lo"], case["len_hi"], n)
    if "q_hi" not in case:
        return [0] * n, lens
    rows = _spread(case["q_lo"], case["q_hi"], n, 0.37)
    return [min(r, m) for r, m in zip(rows, lens)], lens


# ------------------------------------------------------------------ inputs
def _cum(lens, device):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=device)


def _normal(shape, gen, loud=False):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    if loud:
        x[..., 5::16] *= 8
    return x


def _power_above(x):
    """Smallest power of two s >= x, within 2^-64 .. 2^64 (x >= 0)."""
    m, e = torch.frexp(x)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(x > 0, e, torch.full_like(e, -64)).clamp(-64, 64)
    return torch.ldexp(torch.ones_like(x), e)


def _cache(pages, heads, dim, gen, loud):
    """A quantised cache of random values and its power-of-two scales."""
    codes = torch.empty((pages, heads, PAGE, dim), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((pages, heads), device="cuda")
    step = max(1, (1 << 27) // (heads * PAGE * dim))
    for p in range(0, pages, step):
        x = _normal((min(step, pages - p), heads, PAGE, dim), gen, loud).float()
        # (Texts have loud and quiet stretches.)
        x *= torch.exp2(torch.randint(-2, 3, (x.shape[0], 1, 1, 1), generator=gen, device="cuda"))
        s = _power_above(x.abs().amax((2, 3)) / E4M3_MAX)
        codes[p:p + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        scale[p:p + step] = s
    return codes, scale


def _parents(rows, seed):
    """Parents (within its tree, -1: a root) of every node, as a draft model's
    best-first expansion leaves them."""
    rng = random.Random(seed)
    out = []
    for n in rows:
        for i in range(n):
            out.append(-1 if i == 0 or rng.random() < 0.03 else int(i * rng.random() ** 1.5))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    rows, lens = _lengths(case)
    batch, hk, d = case["batch"], case["heads_k"], case["dim"]
    st = dict(case=case, rows=rows, most_q=max(rows), most=max(lens))
    st["cu"] = _cum(rows, "cuda")
    total = sum(rows)
    if op == "prompt":
        h, dv = case["heads"], case["dim_v"]
        st["cu_k"] = _cum(lens, "cuda")
        st["q"] = _normal((total, h, d), gen)
        st["k"] = _normal((sum(lens), hk, d), gen)
        st["v"] = _normal((sum(lens), hk, dv), gen)
        st["scale"] = d ** -0.5
        return st
    width = max(-(-n // PAGE) for n in lens)
    pages = sum(-(-n // PAGE) for n in lens) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    used = 0
    for b, n in enumerate(lens):
        m = -(-n // PAGE)
        table[b, :m] = perm[used:used + m]
        used += m
    st["page_table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["kc"], st["ks"] = _cache(pages, hk, d, gen, True)
    if op != "weights":
        st["vc"], st["vs"] = _cache(pages, hk, d, gen, False)
    if op in ("tree", "commit"):
        st["parents"] = torch.tensor(_parents(rows, seed), dtype=torch.int32, device="cuda")
    if op in ("tree", "sink", "weights"):
        st["q"] = _normal((total, case["heads"], d), gen)
        st["scale"] = d ** -0.5
    if op == "weights":
        # What the attention of the same rows returned, and the sums so far.
        st["lse"] = _row_lse(st)
        st["sums"] = torch.rand((batch, hk, width * PAGE), generator=gen, device="cuda")
        st["sums"] *= st["sums"] ** 8
    if op == "evict":
        # Sums as decode steps leave them: few keys hold most of the weight.
        x = torch.randn((batch, hk, width * PAGE), generator=gen, device="cuda")
        st["sums"] = torch.exp(3 * x)
        st["sums"][torch.rand(x.shape, generator=gen, device="cuda") < 0.2] = 0
    if op == "commit":
        # The verified path: from a root down, as far as the target model agreed.
        rng = random.Random(seed + 1)
        keep = torch.zeros((batch, 1, case["most"]), dtype=torch.int32)
        first, count = [], []
        flat, at = _parents(rows, seed), 0
        for b, n in enumerate(rows):
            par = flat[at:at + n]
            at += n
            node = rng.randrange(n)
            path = []
            while node >= 0:
                path.append(node)
                node = par[node]
            path = path[::-1][:case["most"]]
            ctx = lens[b] - n
            keep[b, 0, :len(path)] = torch.tensor([ctx + p for p in path])
            first.append(ctx)
            count.append(len(path))
        st["keep"] = keep.cuda()
        st["first"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        st["count"] = torch.tensor(count, dtype=torch.int32, device="cuda")
    return st


def _row_lse(st):
    """fp32 LSE [heads, rows] of the case's rows, causal, with its mask."""
    case = st["case"]
    h, hk, d = case["heads"], case["heads_k"], case["dim"]
    lse = torch.empty((h, st["q"].shape[0]), device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(st["rows"], st["lens"].tolist())):
        pages = st["page_table"][b, :-(-length // PAGE)].long()
        k = (st["kc"][pages].float() * st["ks"][pages][..., None, None]).transpose(0, 1)
        k = k.reshape(hk, -1, d)[:, :length]
        q = st["q"][at:at + n].float().reshape(n, hk, h // hk, d).permute(1, 0, 2, 3)
        s = torch.matmul(q.reshape(hk, -1, d), k.transpose(1, 2)) * st["scale"]
        s = s.reshape(hk, n, h // hk, length)
        s.masked_fill_(~_causal_seen(case, n, length)[None, :, None], NEG)
        lse[:, at:at + n] = torch.logsumexp(s, -1).permute(0, 2, 1).reshape(h, n)
        at += n
    return lse


# -------------------------------------------------------------- plain forms
def _causal_seen(case, n, length):
    """[n, length] truth values: key j of row i, which stands at length - n + i."""
    at = torch.arange(length - n, length, device="cuda")[:, None]
    j = torch.arange(length, device="cuda")[None]
    seen = j <= at
    if case["window"] >= 0:
        seen &= (j >= at - case["window"]) | (j < case["sinks"])
    return seen


def _plain_tree(st):
    """Ancestor masks as 32-bit words and the nodes' positions."""
    parents, cu = st["parents"].long(), st["cu"].long()
    n_seq, most = cu.numel() - 1, st["most_q"]
    words = -(-most // 32)
    nodes = parents.numel()
    seq = torch.repeat_interleave(torch.arange(n_seq, device="cuda"), cu[1:] - cu[:-1],
                                  output_size=nodes)
    at = torch.arange(nodes, device="cuda") - cu[seq]
    bits = torch.zeros((nodes, words * 32), dtype=torch.bool, device="cuda")
    depth = torch.full((nodes,), -1, device="cuda")
    node = at
    for _ in range(most):
        live = node >= 0
        safe = node.clamp(min=0)
        bits.scatter_(1, safe[:, None], bits.gather(1, safe[:, None]) | live[:, None])
        depth = depth + live
        node = torch.where(live, parents[cu[seq] + safe], node)
    weight = torch.ones(32, dtype=torch.long, device="cuda") << torch.arange(32, device="cuda")
    packed = (bits.reshape(nodes, words, 32) * weight).sum(-1)
    packed = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).int()
    positions = (st["lens"].long()[seq] - (cu[1:] - cu[:-1])[seq] + depth).int()
    return packed, positions


def _unpack(mask):
    """[T, words] int32 to [T, 32 words] truth values."""
    shift = torch.arange(32, device=mask.device)
    return ((mask.long()[..., None] >> shift) & 1).bool().flatten(-2)


def _plain_attn(st, mask=None):
    """Attention of the case's rows over the cache, all sequences padded."""
    case = st["case"]
    q, table, lens = st["q"].float(), st["page_table"].long(), st["lens"].long()
    cu = st["cu"].long()
    b, hk = table.shape[0], st["kc"].shape[1]
    d, g = q.shape[2], q.shape[1] // hk
    width, most_q = -(-st["most"] // PAGE), st["most_q"]
    table = table[:, :width].clamp(min=0)
    k = (st["kc"][table].float() * st["ks"][table][..., None, None]).transpose(1, 2)
    v = (st["vc"][table].float() * st["vs"][table][..., None, None]).transpose(1, 2)
    k, v = k.reshape(b, hk, width * PAGE, d), v.reshape(b, hk, width * PAGE, d)
    nq = cu[1:] - cu[:-1]
    i = torch.arange(most_q, device=q.device)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    rows = q[row].reshape(b, most_q, hk, g, d).transpose(1, 2).reshape(b, hk, most_q * g, d)
    s = torch.matmul(rows, k.transpose(2, 3)) * st["scale"]
    j = torch.arange(width * PAGE, device=q.device)
    ctx = (lens - nq)[:, None, None]
    if mask is None:
        stand = ctx + i[None, :, None]
        seen = (j <= stand) & (j < lens[:, None, None])
        recent = j >= stand - case["window"]
    else:
        bits = _unpack(mask)[row]                     # [B, most_q, 32 words]
        stand = ctx + bits.sum(-1, keepdim=True) - 1
        node = (j - ctx).clamp(0, bits.shape[2] - 1).expand(b, most_q, -1)
        drafted = (j >= ctx) & (j < lens[:, None, None])
        seen = (j < ctx) | (drafted & bits.gather(2, node))
        recent = (j >= stand - case["window"]) | (j >= ctx)
    if case["window"] >= 0:
        seen &= recent | (j < case["sinks"])
    s = s.masked_fill_(~seen.repeat_interleave(g, dim=1)[:, None], NEG)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    del s
    sums = p.sum(-1, keepdim=True)
    o = (torch.matmul(p, v) / sums).reshape(b, hk, most_q, g, d).transpose(1, 2)
    lse = (top + torch.log(sums)).reshape(b, hk, most_q, g).transpose(1, 2)
    real = i < nq[:, None]
    o = o.reshape(b, most_q, hk * g, d)[real].to(torch.bfloat16)
    return o, lse.reshape(b, most_q, hk * g)[real].t().contiguous()


def _plain_prompt(st):
    case = st["case"]
    h, hk, dv = case["heads"], case["heads_k"], case["dim_v"]
    q, k, v = st["q"], st["k"], st["v"]
    o = torch.empty((q.shape[0], h, dv), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((h, q.shape[0]), device="cuda")
    lens = _lengths(case)[1]
    q0 = k0 = 0
    for n, length in zip(st["rows"], lens):
        seen = _causal_seen(case, n, length)
        step = max(1, (1 << 30) // (n * length))      # heads at once
        for a in range(0, h, step):
            e = min(h, a + step)
            kv = torch.arange(a, e, device="cuda") // (h // hk)
            x = q[q0:q0 + n, a:e].float().transpose(0, 1)
            y = k[k0:k0 + length].float().transpose(0, 1)[kv]
            s = (torch.matmul(x, y.transpose(1, 2)) * st["scale"]).masked_fill_(~seen, NEG)
            top = s.amax(-1, keepdim=True)
            p = torch.exp_(s.sub_(top))
            sums = p.sum(-1, keepdim=True)
            z = torch.matmul(p, v[k0:k0 + length].float().transpose(0, 1)[kv]) / sums
            o[q0:q0 + n, a:e] = z.transpose(0, 1).to(torch.bfloat16)
            lse[a:e, q0:q0 + n] = (top + torch.log(sums))[..., 0]
        q0, k0 = q0 + n, k0 + length
    return o, lse


def _plain_weights(st):
    case = st["case"]
    h, hk, d = case["heads"], case["heads_k"], case["dim"]
    sums = st["sums"]
    at = 0
    lens = _lengths(case)[1]
    for b, (n, length) in enumerate(zip(st["rows"], lens)):
        pages = st["page_table"][b, :-(-length // PAGE)].long()
        k = (st["kc"][pages].float() * st["ks"][pages][..., None, None]).transpose(0, 1)
        k = k.reshape(hk, -1, d)[:, :length]
        q = st["q"][at:at + n].float().reshape(n, hk, h // hk, d).permute(1, 0, 2, 3)
        s = torch.matmul(q.reshape(hk, -1, d), k.transpose(1, 2)) * st["scale"]
        lse = st["lse"][:, at:at + n].reshape(hk, h // hk, n).transpose(1, 2)
        p = torch.exp(s.reshape(hk, n, h // hk, length) - lse[..., None])
        p *= _causal_seen(case, n, length)[None, :, None]
        p = p.sum((1, 2))
        p[:, :length - n] += case["decay"] * sums[b, :, :length - n]
        sums[b, :, :length] = p
        at += n
    return sums


def _plain_select(st):
    """Kept positions [B, heads, budget] in order (-1 behind the last) and lengths."""
    case = st["case"]
    sums, lens = st["sums"], st["lens"].long()
    budget, n = case["budget"], sums.shape[2]
    j = torch.arange(n, device="cuda")
    length = lens[:, None, None]
    fixed = (j < case["sinks"]) | (j >= length - case["recent"])
    key = torch.where(fixed, torch.inf, sums)
    key = torch.where(j < length, key, -torch.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    if n < budget:
        pad = torch.full((*order.shape[:2], budget - n), n, device="cuda")
        order = torch.cat([order, pad], -1)
    held = lens.clamp(max=budget)
    kept = order[..., :budget]
    kept = torch.where(j.new_tensor(range(budget)) < held[:, None, None], kept, 1 << 30)
    kept = torch.sort(kept, dim=-1).values
    return torch.where(kept == 1 << 30, -1, kept).int(), held.int()


def _plain_move(codes, scale, table, keep, first, count):
    """Rows keep[b, h, j], j < count[b], to the slots first[b] + j of sequence b."""
    batch, m = keep.shape[0], keep.shape[2]
    pages, hk, _, d = codes.shape
    keep = keep.long().expand(batch, hk, m)
    first, count = first.long(), count.long()
    b = torch.arange(batch, device="cuda")[:, None, None]
    h = torch.arange(hk, device="cuda")[None, :, None]
    j = torch.arange(m, device="cuda")
    live = (j < count[:, None])[:, None]                       # [B, 1, m]
    dst = (first[:, None] + j)[:, None].expand(batch, hk, m)
    src = keep.clamp(min=0)
    page = table.long()[b, src // PAGE].clamp(min=0)
    rows = codes[page, h, src % PAGE].float() * scale[page, h][..., None]
    n_pages = (PAGE - 1 + m - 1) // PAGE + 1
    p = dst // PAGE - (first // PAGE)[:, None, None]           # page of the move
    top = torch.where(live, rows.abs().amax(-1), 0.0)
    amax = torch.zeros((batch, hk, n_pages), device="cuda").scatter_reduce_(2, p, top, "amax")
    moved = torch.zeros((batch, hk, n_pages), device="cuda").scatter_reduce_(
        2, p, ((src != dst) & live).float(), "amax") > 0
    at = (first // PAGE)[:, None] + torch.arange(n_pages, device="cuda")
    cell_page = table.long().gather(1, at.clamp(max=table.shape[1] - 1)).clamp(min=0)
    cell_page = cell_page[:, None].expand(batch, hk, n_pages)
    slot0 = torch.where(at == (first // PAGE)[:, None], (first % PAGE)[:, None], 0)[:, None]
    old = scale[cell_page, h]
    new = _power_above(amax / E4M3_MAX)
    new = torch.where(slot0 > 0, torch.maximum(new, old), new)
    # Codes before the first slot follow a scale that has grown.
    ratio = torch.where(slot0 > 0, old / new, 1.0)
    pb, ph, pp = torch.nonzero(moved, as_tuple=True)
    held = codes[cell_page[pb, ph, pp], ph].float()
    before = torch.arange(PAGE, device="cuda") < slot0.expand(batch, hk, n_pages)[pb, ph, pp][:, None]
    held = torch.where(before[..., None], held * ratio[pb, ph, pp][:, None, None], held)
    index = torch.full((batch, hk, n_pages), -1, device="cuda")
    index[pb, ph, pp] = torch.arange(pb.numel(), device="cuda")
    where = index.gather(2, p)
    go = live & (where >= 0)
    values = rows / new.gather(2, p)[..., None]
    held[where[go], dst[go] % PAGE] = values[go].clamp(-E4M3_MAX, E4M3_MAX)
    codes[cell_page[pb, ph, pp], ph] = held.to(torch.float8_e4m3fn)
    scale[cell_page[pb, ph, pp], ph] = new[pb, ph, pp]


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import varlen_flashattention_forward_gb300 as fa
        if op == "prompt":
            o, lse = fa.fa_varlen_fwd(st["q"], st["k"], st["v"], st["cu"], st["cu_k"],
                                      st["most_q"], st["most"], st["scale"], causal=True,
                                      window_left=case["window"], sink_tokens=case["sinks"],
                                      return_lse=True)
            return dict(o=o, lse=lse)
        if op == "tree":
            mask, positions = fa.fa_draft_tree(st["parents"], st["cu"], st["lens"],
                                               max_nodes=st["most_q"])
            o, lse = fa.fa_paged_attn(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["cu"],
                                      st["lens"], st["page_table"], max_seqlen_q=st["most_q"],
                                      max_seqlen_k=st["most"], softmax_scale=st["scale"],
                                      window_left=case["window"], sink_tokens=case["sinks"],
                                      tree_mask=mask, return_lse=True)
            return dict(mask=mask, positions=positions, o=o, lse=lse)
        if op == "sink":
            o, lse = fa.fa_paged_attn(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["cu"],
                                      st["lens"], st["page_table"], max_seqlen_q=st["most_q"],
                                      max_seqlen_k=st["most"], softmax_scale=st["scale"],
                                      window_left=case["window"], sink_tokens=case["sinks"],
                                      return_lse=True)
            return dict(o=o, lse=lse)
        if op == "weights":
            fa.fa_paged_key_weights(st["q"], st["lse"], st["kc"], st["ks"], st["cu"], st["lens"],
                                    st["page_table"], st["sums"], softmax_scale=st["scale"],
                                    window_left=case["window"], sink_tokens=case["sinks"],
                                    decay=case["decay"])
            return dict(sums=st["sums"])
        if op == "evict":
            keep, lens = fa.fa_paged_kv_select(st["sums"], st["lens"], case["budget"],
                                               sink_tokens=case["sinks"],
                                               recent_tokens=case["recent"])
            fa.fa_paged_kv_compact(st["kc"], st["vc"], st["ks"], st["vs"], st["page_table"], keep,
                                   lens, weights=st["sums"])
            return dict(keep=keep, lens=lens, k=st["kc"], v=st["vc"], k_scale=st["ks"],
                        v_scale=st["vs"], sums=st["sums"])
        fa.fa_paged_kv_compact(st["kc"], st["vc"], st["ks"], st["vs"], st["page_table"],
                               st["keep"], st["count"], first=st["first"])
        return dict(k=st["kc"], v=st["vc"], k_scale=st["ks"], v_scale=st["vs"])
    if op == "prompt":
        o, lse = _plain_prompt(st)
        return dict(o=o, lse=lse)
    if op == "tree":
        mask, positions = _plain_tree(st)
        o, lse = _plain_attn(st, mask)
        return dict(mask=mask, positions=positions, o=o, lse=lse)
    if op == "sink":
        o, lse = _plain_attn(st)
        return dict(o=o, lse=lse)
    if op == "weights":
        return dict(sums=_plain_weights(st))
    if op == "evict":
        keep, lens = _plain_select(st)
        first = torch.zeros_like(lens)
        _plain_move(st["kc"], st["ks"], st["page_table"], keep, first, lens)
        _plain_move(st["vc"], st["vs"], st["page_table"], keep, first, lens)
        live = keep >= 0
        moved = st["sums"].gather(2, keep.long().clamp(min=0))
        n = min(keep.shape[2], st["sums"].shape[2])
        st["sums"][..., :n] = torch.where(live, moved, 0.0)[..., :n] \
            + torch.where(live[..., :n], 0.0, st["sums"][..., :n])
        return dict(keep=keep, lens=lens, k=st["kc"], v=st["vc"], k_scale=st["ks"],
                    v_scale=st["vs"], sums=st["sums"])
    _plain_move(st["kc"], st["ks"], st["page_table"], st["keep"], st["first"], st["count"])
    _plain_move(st["vc"], st["vs"], st["page_table"], st["keep"], st["first"], st["count"])
    return dict(k=st["kc"], v=st["vc"], k_scale=st["ks"], v_scale=st["vs"])


# --------------------------------------------------------------------- work
def _seen_keys(case, n, length):
    """(keys that some row sees, pairs of a row and a key it sees), causal."""
    w, s = case["window"], case["sinks"]
    keys = length
    if w >= 0:
        lo = max(0, length - n - w)
        keys = length - lo + min(s, lo)
    pairs = 0
    for at in range(length - n, length):
        lo = max(0, at - w) if w >= 0 else 0
        pairs += at + 1 - lo + min(s, lo)
    return keys, pairs


def work(case):
    op, d, hk = case["op"], case["dim"], case["heads_k"]
    rows, lens = _lengths(case)
    table = sum(-(-n // PAGE) for n in lens) * (4 + 8 * hk)
    if op in ("evict", "commit"):
        # Codes of the rows that move are read and written, keys and values.
        n = sum(min(m, case["budget"]) for m in lens) if op == "evict" \
            else sum(min(m, case["most"]) for m in rows)
        sums = 4 * hk * sum(lens) + 12 * hk * n if op == "evict" else 4 * n
        return dict(bytes=4 * n * hk * d + sums, flops=4 * n * hk * d)
    h = case["heads"]
    seen = [_seen_keys(case, n, m) for n, m in zip(rows, lens)]
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    if op == "prompt":
        dv = case["dim_v"]
        return dict(bytes=sum(rows) * h * (2 * d + 2 * dv + 4) + keys * hk * 2 * (d + dv),
                    flops=pairs * h * 2 * (d + dv))
    if op == "weights":
        moved = sum(lens) * hk * (8 if case["decay"] else 4)
        return dict(bytes=keys * hk * d + table // 2 + sum(rows) * h * (2 * d + 4) + moved,
                    flops=pairs * h * 2 * d)
    tree = 12 * sum(rows) if op == "tree" else 0
    return dict(bytes=keys * hk * d * 2 + keys // PAGE * (4 + 8 * hk) + sum(rows) * h * (d * 4 + 4)
                + tree, flops=pairs * h * d * 4)


# -------------------------------------------------------------------- exact
def _e4m3(x):
    """x (fp64) rounded to the nearest e4m3 value, ties to even, within +-448."""
    m, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _held(st, b, n, codes, scale):
    """fp64 rows [heads, n, d] of sequence b's first n positions."""
    pages = st["page_table"][b, :-(-n // PAGE)].long()
    x = codes[pages].double() * scale[pages].double()[:, :, None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_move(st, codes, scale, keep, first, count):
    """Pages one after another, each from its values before the move."""
    codes, scale = codes.double(), scale.double()
    was, factor = codes.clone(), scale.clone()
    pt = st["page_table"].tolist()
    hk = codes.shape[1]
    head = torch.arange(hk, device="cuda")[:, None]
    for b, (f, c) in enumerate(zip(first, count)):
        table = st["page_table"][b].long()
        slot = f
        while slot < f + c:
            off, m = slot % PAGE, min(PAGE - slot % PAGE, f + c - slot)
            src = keep[b, :, slot - f:slot - f + m].long().expand(hk, m)
            page = pt[b][slot // PAGE]
            stays = (src == torch.arange(slot, slot + m, device="cuda")).all(1)
            from_page = table[src // PAGE]
            rows = was[from_page, head, src % PAGE] * factor[from_page, head][..., None]
            top = rows.abs().amax((1, 2))
            s = torch.full_like(top, 2.0 ** -64)
            for _ in range(128):
                s = torch.where((top > E4M3_MAX * s) & (s < 2.0 ** 64), 2 * s, s)
            if off:
                s = torch.maximum(s, factor[page])
            new = codes[page].clone()
            if off:
                new[:, :off] = _e4m3(new[:, :off] * (factor[page] / s)[:, None, None])
            new[:, off:off + m] = _e4m3(rows / s[:, None, None])
            codes[page] = torch.where(stays[:, None, None], codes[page], new)
            scale[page] = torch.where(stays, scale[page], s)
            slot += m
    return codes, scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    rows, lens = _lengths(case)
    hk, d = case["heads_k"], case["dim"]
    if op in ("evict", "commit"):
        if op == "commit":
            keep, out = st["keep"], {}
            first, count = st["first"].tolist(), st["count"].tolist()
        else:
            first, count = [0] * len(lens), [min(n, case["budget"]) for n in lens]
            keep = torch.full((len(lens), hk, case["budget"]), -1, dtype=torch.int32, device="cuda")
            sums = st["sums"].double()
            for b, n in enumerate(lens):
                lo, hi = case["sinks"], n - case["recent"]
                if n <= case["budget"]:
                    keep[b, :, :n] = torch.arange(n, device="cuda")
                    continue
                m = case["budget"] - lo - case["recent"]
                # The m-th largest value, all above it, and its first few ties.
                x = sums[b, :, lo:hi]
                mine = torch.zeros_like(x, dtype=torch.bool)
                if m:
                    edge = torch.sort(x, -1).values[:, hi - lo - m][:, None]
                    mine = x > edge
                    ties = x == edge
                    mine |= ties & (ties.cumsum(-1) <= m - mine.sum(-1, keepdim=True))
                chosen = torch.ones((hk, n), dtype=torch.bool, device="cuda")
                chosen[:, lo:hi] = mine
                keep[b] = chosen.nonzero()[:, 1].reshape(hk, -1)
            for b, n in enumerate(count):
                sums[b, :, :n] = sums[b].gather(1, keep[b, :, :n].long())
            out = dict(keep=keep, lens=torch.tensor(count, dtype=torch.int32, device="cuda"))
        k, ks = _exact_move(st, st["kc"], st["ks"], keep, first, count)
        v, vs = _exact_move(st, st["vc"], st["vs"], keep, first, count)
        out.update(k=k, v=v, k_scale=ks, v_scale=vs)
        if op == "evict":
            out["sums"] = sums
        return out
    h = case["heads"]
    g = h // hk
    total = sum(rows)
    if op == "weights":
        sums = st["sums"].double()
        at = 0
        for b, (n, length) in enumerate(zip(rows, lens)):
            k = _held(st, b, length, st["kc"], st["ks"])
            new = torch.zeros((hk, length), dtype=torch.float64, device="cuda")
            for i in range(n):
                hi = length - n + i + 1
                lo = max(0, hi - 1 - case["window"]) if case["window"] >= 0 else 0
                x = k[:, :hi] @ st["q"][at + i].double().reshape(hk, g, d).transpose(1, 2)
                p = torch.exp(x * st["scale"] - st["lse"][:, at + i].double().reshape(hk, 1, g))
                p[:, min(case["sinks"], lo):lo] = 0
                new[:, :hi] += p.sum(-1)
            new[:, :length - n] += case["decay"] * sums[b, :, :length - n]
            sums[b, :, :length] = new
            at += n
        return dict(sums=sums)
    dv = case.get("dim_v", d)
    o = torch.zeros((total, h, dv), dtype=torch.float64, device="cuda")
    lse = torch.full((h, total), NEG, dtype=torch.float64, device="cuda")
    out = {}
    if op == "tree":
        flat, words = st["parents"].tolist(), -(-max(rows) // 32)
        paths, positions = [], []
        at = 0
        for n, length in zip(rows, lens):
            for i in range(n):
                path, node = [], i
                while node >= 0:
                    path.append(node)
                    node = flat[at + node]
                paths.append(path)
                positions.append(length - n + len(path) - 1)
            at += n
        mask = [[sum(1 << (p % 32) for p in path if p // 32 == w) for w in range(words)]
                for path in paths]
        mask = [[w - (1 << 32) if w >> 31 else w for w in row] for row in mask]
        out = dict(mask=torch.tensor(mask, dtype=torch.int32, device="cuda"),
                   positions=torch.tensor(positions, dtype=torch.int32, device="cuda"))
    at = k0 = 0
    for b, (n, length) in enumerate(zip(rows, lens)):
        if op == "prompt":
            k = st["k"][k0:k0 + length].double().transpose(0, 1)
            v = st["v"][k0:k0 + length].double().transpose(0, 1)
            k0 += length
        else:
            k = _held(st, b, length, st["kc"], st["ks"])
            v = _held(st, b, length, st["vc"], st["vs"])
        step = 256 if op == "prompt" else 1
        for i in range(0, n, step):
            m = min(step, n - i)
            if op == "tree":
                pos = positions[at + i]
                ctx = length - n
                lo = max(0, pos - case["window"]) if case["window"] >= 0 else 0
                lo = min(lo, ctx)
                cols = list(range(min(case["sinks"], lo))) + list(range(lo, ctx))
                cols += sorted(ctx + p for p in paths[at + i])
                cols = torch.tensor(cols, device="cuda")
                hidden = None
            else:
                # Columns of the block: the sinks, then what its windows span.
                p0 = length - n + i
                lo = max(0, p0 - case["window"]) if case["window"] >= 0 else 0
                sinks = torch.arange(min(case["sinks"], lo), device="cuda")
                cols = torch.cat([sinks, torch.arange(lo, p0 + m, device="cuda")])
                pos = p0 + torch.arange(m, device="cuda")[:, None]
                hidden = cols > pos
                if case["window"] >= 0:
                    hidden |= (cols < pos - case["window"]) & (cols >= case["sinks"])
            x = st["q"][at + i:at + i + m].double().reshape(m, hk, g, d).permute(1, 2, 0, 3)
            x = torch.matmul(x.reshape(hk, g * m, d), k[:, cols].transpose(1, 2)) * st["scale"]
            x = x.reshape(hk, g, m, -1)
            if hidden is not None:
                x.masked_fill_(hidden, NEG)
            l = torch.logsumexp(x, dim=-1)
            p = torch.exp(x - l[..., None]).reshape(hk, g * m, -1)
            y = torch.matmul(p, v[:, cols]).reshape(hk, g, m, dv).permute(2, 0, 1, 3)
            o[at + i:at + i + m] = y.reshape(m, h, dv)
            lse[:, at + i:at + i + m] = l.reshape(h, m)
        at += n
    out.update(o=o, lse=lse)
    return out
