"""Measured cases of the serving operators around the attention forward:

  norm_rope  per-head RMS norm of queries and keys with the position rotation
  append     new keys and values into the paged 8-bit cache
  attn       attention of a few query rows per sequence over that cache
  gather     the cache back to packed bf16 keys and values

`run` computes them in plain fp32 torch, or, with `own` set, through the
library's entry points.  `exact` computes them from their definition in fp64.

Shapes: head counts and head dims of the repository's workloads (32 query
heads over 8 or 4, head dims 64, 80, 96, 128, prompts of a few thousand
tokens, contexts up to 65536).  Inputs are normal, with one channel in 16 of
the keys eight times larger, as keys of trained models have.
"""
import math
import random

import torch

own = False

PAGE = 64
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of 64 requests: latency counts.
        dict(name="norm_rope step 64", op="norm_rope", tokens=64, heads=32, heads_k=8, dim=128,
             rot=128, interleaved=False),
        # A packed batch of prompts, q and k taken out of a fused projection.
        dict(name="norm_rope prompt 8192", op="norm_rope", tokens=8192, heads=32, heads_k=8,
             dim=128, rot=128, interleaved=False),
        # Odd token count, partial rotation of neighbouring pairs.
        dict(name="norm_rope odd d96", op="norm_rope", tokens=5003, heads=28, heads_k=4, dim=96,
             rot=48, interleaved=True),
        # One decode step of 256 requests: every token lands in a page that holds others.
        dict(name="append step 256", op="append", batch=256, new_lo=1, new_hi=1, ctx_lo=1,
             ctx_hi=4095, heads_k=8, dim=128, rot=128, norm=True, interleaved=False),
        # Prompts of about 2048 tokens written into empty caches.
        dict(name="append prompt 4x2048", op="append", batch=4, new_lo=1900, new_hi=2048, ctx_lo=0,
             ctx_hi=0, heads_k=8, dim=128, rot=128, norm=True, interleaved=False),
        # Ragged chunks behind ragged contexts, keys already rotated.
        dict(name="append ragged d64", op="append", batch=37, new_lo=1, new_hi=700, ctx_lo=3,
             ctx_hi=1500, heads_k=4, dim=64, rot=0, norm=False, interleaved=False),
        # One request of 8192 tokens: the latency of a lone user.
        dict(name="attn one 8192", op="attn", batch=1, q_lo=1, q_hi=1, len_lo=8192, len_hi=8192,
             heads=32, heads_k=8, dim=128, window=-1),
        # A decode step of a mixed batch.
        dict(name="attn step 64", op="attn", batch=64, q_lo=1, q_hi=1, len_lo=100, len_hi=8192,
             heads=32, heads_k=4, dim=128, window=-1),
        # Long contexts: the rate at which the cache streams.
        dict(name="attn long 32x32768", op="attn", batch=32, q_lo=1, q_hi=1, len_lo=30001,
             len_hi=32768, heads=32, heads_k=8, dim=128, window=-1),
        # Drafts of several tokens checked at once, in a sliding window.
        dict(name="attn drafts d64 window", op="attn", batch=24, q_lo=2, q_hi=7, len_lo=517,
             len_hi=9001, heads=32, heads_k=8, dim=64, window=4096),
        # Context of two long chunks, for the prompt kernel.
        dict(name="gather 2x32768", op="gather", batch=2, len_lo=30000, len_hi=32768, heads_k=8,
             dim=128),
        # Short ragged contexts.
        dict(name="gather ragged d96", op="gather", batch=21, len_lo=1, len_hi=1300, heads_k=4,
             dim=96),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "attn", "attn", "gather"))
    dim = rng.choice((64, 80, 96, 128))
    if op == "norm_rope":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.choice((8, 16, 28, 32)),
                    heads_k=rng.choice((1, 4, 8)), dim=dim, rot=16 * rng.randint(0, dim // 16),
                    interleaved=rng.random() < 0.5)
    heads_k = rng.choice((1, 2, 4, 8))
    if op == "append":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, 8192 // batch))
        ctx = rng.choice((0, _log(rng, 1, 4095)))
        return dict(op=op, batch=batch, new_lo=min(hi, rng.choice((0, 1, hi))), new_hi=hi,
                    ctx_lo=min(ctx, rng.choice((0, ctx))), ctx_hi=ctx, heads_k=heads_k, dim=dim,
                    rot=rng.choice((0, 16 * (dim // 16))), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5)
    if op == "gather":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, 65536 // batch)
        return dict(op=op, batch=batch, len_lo=rng.choice((0, hi // 2, hi)), len_hi=hi,
                    heads_k=heads_k, dim=dim)
    batch = _log(rng, 1, 128)
    hi = min(65536, _log(rng, 1, (1 << 20) // batch))
    q_hi = min(hi, rng.choice((1, 1, 1, 2, 5, 8)))
    return dict(op=op, batch=batch, q_lo=rng.choice((1, q_hi)), q_hi=q_hi,
                len_lo=max(q_hi, rng.choice((hi // 8, hi))), len_hi=hi,
                heads=heads_k * rng.choice((1, 3, 4, 8, 16)), heads_k=heads_k, dim=dim,
                window=rng.choice((-1, -1, _log(rng, 1, hi))))


def _spread(lo, hi, n, phase=0.0):
    """n whole numbers in [lo, hi], both ends among them where n allows, in no order."""
    if n == 1:
        return [hi]
    mixed = sorted(range(n), key=lambda i: (i * 0.6180339887498949 + phase) % 1.0)
    return [lo + (hi - lo) * i // (n - 1) for i in mixed]


def _lengths(case):
    """(new or query tokens, total length after them) of each sequence."""
    op, n = case["op"], case["batch"]
    if op == "append":
        new = _spread(case["new_lo"], case["new_hi"], n)
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], n, 0.37)
        return new, [a + b for a, b in zip(new, ctx)]
    if op == "attn":
        return (_spread(case["q_lo"], case["q_hi"], n, 0.37),
                _spread(case["len_lo"], case["len_hi"], n))
    lens = _spread(case["len_lo"], case["len_hi"], n)
    return lens, lens


# ------------------------------------------------------------------ inputs
def _table(positions, rot, device):
    """cos and sin of the first `positions` positions, angles in fp64."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


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


def _cache(pages, heads, dim, gen, loud):
    """A quantised cache of random values and its power-of-two scales."""
    codes = torch.empty((pages, heads, PAGE, dim), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((pages, heads), device="cuda")
    step = max(1, (1 << 27) // (heads * PAGE * dim))
    for p in range(0, pages, step):
        x = _normal((min(step, pages - p), heads, PAGE, dim), gen, loud).float()
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX)))
        codes[p:p + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
        scale[p:p + step] = s
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "norm_rope":
        t, h, hk, d = case["tokens"], case["heads"], case["heads_k"], case["dim"]
        qkv = _normal((t, h + 2 * hk, d), gen)
        st["q"], st["k"] = qkv[:, :h], qkv[:, h:h + hk]
        st["qw"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
        st["kw"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
        st["positions"] = torch.randint(0, 65536, (t,), generator=gen, device="cuda",
                                        dtype=torch.int32)
        st["table"] = _table(65536, case["rot"], "cuda") if case["rot"] else None
        return st
    new, lens = _lengths(case)
    width = max(1, max(-(-n // PAGE) for n in lens))
    pages = sum(-(-n // PAGE) for n in lens) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    used = 0
    rows = []
    for b, n in enumerate(lens):
        m = -(-n // PAGE)
        rows.append((b, used, m))
        used += m
    table = table.cuda()
    for b, at, m in rows:
        table[b, :m] = perm[at:at + m]
    st["page_table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    hk, d = case["heads_k"], case["dim"]
    st["kc"], st["ks"] = _cache(pages, hk, d, gen, True)
    st["vc"], st["vs"] = _cache(pages, hk, d, gen, False)
    st["cu"] = _cum(new, "cuda")
    st["most_new"], st["most"] = max(new), max(lens)
    total = sum(new)
    if op == "append":
        kv = _normal((total, 2 * hk, d), gen)
        st["k"], st["v"] = kv[:, :hk], kv[:, hk:]
        st["k"][..., 5::16] *= 8
        st["kw"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if case["norm"] else None
        st["table"] = _table(width * PAGE, case["rot"], "cuda") if case["rot"] else None
        # Where each new token goes, as a scheduler has it.
        seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
        at = torch.arange(total, device="cuda") - st["cu"][:-1].long()[seq]
        st["pos"] = st["lens"].long()[seq] - torch.tensor(new, device="cuda")[seq] + at
        st["page"] = table[seq, st["pos"] // PAGE].long()
    elif op == "attn":
        st["q"] = _normal((total, case["heads"], d), gen)
        st["scale"] = d ** -0.5
    else:
        st["total"] = total
        seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
        st["pos"] = torch.arange(total, device="cuda") - st["cu"][:-1].long()[seq]
        st["page"] = table[seq, st["pos"] // PAGE].long()
    return st


# -------------------------------------------------------------- plain forms
def _plain_norm(x, w):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return x


def _plain_rotate(x, rows, interleaved):
    """x [T, H, d] fp32, rows [T, rot] cos then sin; the first rot dims turn."""
    half = rows.shape[1] // 2
    cos, sin = rows[:, None, :half], rows[:, None, half:]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_store(y, page, pos, codes, scale):
    """Puts y [T, Hk, d] fp32 at (page, pos % 64), growing the pages' scales."""
    pages, inv = torch.unique(page, return_inverse=True)
    n, off = pages.numel(), pos % PAGE
    amax = torch.zeros((n, y.shape[1]), device=y.device)
    amax.index_reduce_(0, inv, y.abs().amax(-1), "amax")
    s = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(-64, 64))
    first = torch.full((n,), PAGE, device=y.device, dtype=off.dtype)
    first.index_reduce_(0, inv, off, "amin")
    old = scale[pages]
    s = torch.where((first > 0)[:, None], torch.maximum(s, old), s)
    ratio = torch.where((first > 0)[:, None], old / s, 1.0)
    held = codes[pages].float()
    # Slots behind the new tokens keep their codes; those before follow the scale.
    before = torch.arange(PAGE, device=y.device)[None, :] < first[:, None]
    held = torch.where(before[:, None, :, None], held * ratio[:, :, None, None], held)
    held[inv, :, off] = (y / s[inv][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes[pages] = held.to(torch.float8_e4m3fn)
    scale[pages] = s


def _plain_attn(st):
    q, table, lens = st["q"].float(), st["page_table"].long(), st["lens"].long()
    cu = st["cu"].long()
    b, hk = table.shape[0], st["kc"].shape[1]
    d, g = q.shape[2], q.shape[1] // hk
    width, most_q = -(-st["most"] // PAGE), st["most_new"]
    table = table[:, :width].clamp(min=0)
    k = (st["kc"][table].float() * st["ks"][table][..., None, None]).transpose(1, 2)
    v = (st["vc"][table].float() * st["vs"][table][..., None, None]).transpose(1, 2)
    k, v = k.reshape(b, hk, width * PAGE, d), v.reshape(b, hk, width * PAGE, d)
    nq = cu[1:] - cu[:-1]
    i = torch.arange(most_q, device=q.device)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    # [B, Hk, most_q * g, d]
    rows = q[row].reshape(b, most_q, hk, g, d).transpose(1, 2).reshape(b, hk, most_q * g, d)
    s = torch.matmul(rows, k.transpose(2, 3)) * st["scale"]
    last = lens[:, None] - nq[:, None] + i          # the key at each row's own position
    j = torch.arange(width * PAGE, device=q.device)
    seen = j <= last[:, :, None]
    if st["case"]["window"] >= 0:
        seen &= j >= last[:, :, None] - st["case"]["window"]
    seen = seen.repeat_interleave(g, dim=1)[:, None]
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    sums = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(j[None, :, None] < lens[:, None, None], 1.0, 0.0)[:, None] * v)
    o = (o / sums).reshape(b, hk, most_q, g, d).transpose(1, 2).reshape(b, most_q, hk * g, d)
    lse = (top + torch.log(sums)).reshape(b, hk, most_q, g).transpose(1, 2)
    lse = lse.reshape(b, most_q, hk * g)
    real = i < nq[:, None]
    return o[real].to(torch.bfloat16), lse[real].t().contiguous()


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import varlen_flashattention_forward_gb300 as fa
        if op == "norm_rope":
            q, k = fa.fa_qk_norm_rope(st["q"], st["k"], st["positions"], st["table"], st["qw"],
                                      st["kw"], eps=EPS, interleaved=case["interleaved"])
            return dict(q=q, k=k)
        if op == "append":
            fa.fa_paged_kv_append(st["k"], st["v"], st["cu"], st["lens"], st["page_table"],
                                  st["kc"], st["vc"], st["ks"], st["vs"], cos_sin=st["table"],
                                  k_weight=st["kw"], eps=EPS, interleaved=case["interleaved"])
            return dict(k=st["kc"], v=st["vc"], k_scale=st["ks"], v_scale=st["vs"])
        if op == "attn":
            o, lse = fa.fa_paged_attn(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["cu"],
                                      st["lens"], st["page_table"], max_seqlen_q=st["most_new"],
                                      max_seqlen_k=st["most"], softmax_scale=st["scale"],
                                      causal=True, window_left=case["window"], return_lse=True)
            return dict(o=o, lse=lse)
        k, v = fa.fa_paged_kv_gather(st["kc"], st["vc"], st["ks"], st["vs"], st["cu"],
                                     st["page_table"], st["total"])
        return dict(k=k, v=v)
    if op == "norm_rope":
        q, k = _plain_norm(st["q"], st["qw"]), _plain_norm(st["k"], st["kw"])
        if st["table"] is not None:
            rows = st["table"][st["positions"].long()]
            q = _plain_rotate(q, rows, case["interleaved"])
            k = _plain_rotate(k, rows, case["interleaved"])
        return dict(q=q.to(torch.bfloat16), k=k.to(torch.bfloat16))
    if op == "append":
        k = _plain_norm(st["k"], st["kw"])
        if st["table"] is not None:
            k = _plain_rotate(k, st["table"][st["pos"]], case["interleaved"])
        _plain_store(k, st["page"], st["pos"], st["kc"], st["ks"])
        _plain_store(st["v"].float(), st["page"], st["pos"], st["vc"], st["vs"])
        return dict(k=st["kc"], v=st["vc"], k_scale=st["ks"], v_scale=st["vs"])
    if op == "attn":
        o, lse = _plain_attn(st)
        return dict(o=o, lse=lse)
    off = st["pos"] % PAGE
    k = st["kc"][st["page"], :, off].float() * st["ks"][st["page"]][..., None]
    v = st["vc"][st["page"], :, off].float() * st["vs"][st["page"]][..., None]
    return dict(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16))


# --------------------------------------------------------------------- work
def work(case):
    op, d = case["op"], case["dim"]
    if op == "norm_rope":
        t, rows = case["tokens"], case["tokens"] * (case["heads"] + case["heads_k"])
        return dict(bytes=rows * d * 4 + t * (4 + 4 * case["rot"]) + 8 * d, flops=rows * d * 7)
    hk = case["heads_k"]
    new, lens = _lengths(case)
    table = sum(-(-n // PAGE) for n in lens) * 4 + 8 * len(lens)
    if op == "append":
        total = sum(new)
        touched = sum(-(-n // PAGE) - (n - m) // PAGE for m, n in zip(new, lens) if m)
        return dict(bytes=total * hk * d * 6 + touched * (4 + 8 * hk) + total * case["rot"] * 4,
                    flops=total * hk * d * 12)
    if op == "gather":
        return dict(bytes=sum(lens) * hk * d * 6 + table * (1 + 2 * hk), flops=sum(lens) * hk * d * 2)
    h, w = case["heads"], case["window"]
    keys = pairs = 0
    for m, n in zip(new, lens):
        lo = max(0, n - m - w) if w >= 0 else 0
        keys += n - lo
        for i in range(n - m, n):
            pairs += i + 1 - (max(0, i - w) if w >= 0 else 0)
    return dict(bytes=keys * hk * d * 2 + keys // PAGE * (4 + 8 * hk) + sum(new) * h * (d * 4 + 4),
                flops=pairs * h * d * 4)


# -------------------------------------------------------------------- exact
def _e4m3(x):
    """x (fp64) rounded to the nearest e4m3 value, ties to even, within +-448."""
    m, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _turned(x, positions, table, interleaved):
    """fp64 rotation, written with complex numbers."""
    half = table.shape[1] // 2
    t = table.double()[positions.long()]
    w = torch.complex(t[:, :half], t[:, half:])[:, None]
    if interleaved:
        z = torch.complex(x[..., 0:2 * half:2].contiguous(), x[..., 1:2 * half:2].contiguous()) * w
        y = torch.stack([z.real, z.imag], dim=-1).flatten(-2)
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * w
        y = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([y, x[..., 2 * half:]], dim=-1)


def _unit(x, w):
    x = x.double()
    return x if w is None else x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        q, k = _unit(st["q"], st["qw"]), _unit(st["k"], st["kw"])
        if st["table"] is not None:
            q = _turned(q, st["positions"], st["table"], case["interleaved"])
            k = _turned(k, st["positions"], st["table"], case["interleaved"])
        return dict(q=q, k=k)
    pt, lens = st["page_table"].tolist(), st["lens"].tolist()
    cu = st["cu"].tolist()
    if op == "append":
        y = _unit(st["k"], st["kw"])
        if st["table"] is not None:
            y = _turned(y, st["pos"], st["table"], case["interleaved"])
        out = {}
        for name, x, codes, scale in (("k", y, st["kc"], st["ks"]), ("v", st["v"].double(), st["vc"], st["vs"])):
            codes, scale = codes.double(), scale.double()
            for b, n in enumerate(lens):
                at = n - (cu[b + 1] - cu[b])
                while at < n:
                    page, off = pt[b][at // PAGE], at % PAGE
                    m = min(PAGE - off, n - at)
                    rows = x[cu[b + 1] - n + at:][:m].transpose(0, 1)
                    s = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / E4M3_MAX)).clamp(-64, 64))
                    if off:
                        s = torch.maximum(s, scale[page])
                        codes[page, :, :off] = _e4m3(codes[page, :, :off] * (scale[page] / s)[:, None, None])
                    codes[page, :, off:off + m] = _e4m3(rows / s[:, None, None])
                    scale[page] = s
                    at += m
            out[name], out[name + "_scale"] = codes, scale
        return out
    if op == "gather":
        ks, vs = [], []
        for b, n in enumerate(lens):
            pages = torch.tensor(pt[b][:-(-n // PAGE)], dtype=torch.long, device="cuda")
            for got, codes, scale in ((ks, st["kc"], st["ks"]), (vs, st["vc"], st["vs"])):
                x = codes[pages].double() * scale[pages].double()[:, :, None, None]
                got.append(x.transpose(1, 2).flatten(0, 1)[:n])
        return dict(k=torch.cat(ks), v=torch.cat(vs))
    h, hk, d = case["heads"], case["heads_k"], case["dim"]
    o = torch.zeros((cu[-1], h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((h, cu[-1]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        pages = torch.tensor(pt[b][:-(-n // PAGE)], dtype=torch.long, device="cuda")
        k, v = ((c[pages].double() * s[pages].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
                for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        for t in range(cu[b], cu[b + 1]):
            hi = n - (cu[b + 1] - t) + 1
            lo = max(0, hi - 1 - case["window"]) if case["window"] >= 0 else 0
            x = st["q"][t].double().reshape(hk, h // hk, d) @ k[:, lo:hi].transpose(1, 2) * st["scale"]
            l = torch.logsumexp(x, dim=-1)
            o[t] = (torch.exp(x - l[..., None]) @ v[:, lo:hi]).reshape(h, d)
            lse[:, t] = l.reshape(h)
    return dict(o=o, lse=lse)
