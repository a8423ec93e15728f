"""Plain fp64 forms of the paged-cache operators, and inputs for their tests.

Everything here is written from the definitions in include/fa_gb300.h, with
loops over sequences, pages and rows, on the CPU; nothing of the library is
used.
"""
import math

import torch

PAGE = 64
E4M3_MAX = 448.0
NAN_CODE = 0x7F


def e4m3(x):
    """x (fp64) rounded to the nearest e4m3 value, ties to even, saturating."""
    m, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    y = (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return torch.where(torch.isnan(x), x, y)


def e4m3_half_step(x):
    """Largest rounding error of a value x that is rounded to e4m3."""
    m, e = torch.frexp(x.abs().clamp(max=E4M3_MAX))
    return torch.exp2((e - 1).clamp(min=-6).double() - 4)


def page_scale(amax):
    """Smallest power of two s with amax <= 448 s, within 2^-64 .. 2^64."""
    s = torch.full_like(amax, 2.0 ** -64)
    for _ in range(128):
        s = torch.where((amax > E4M3_MAX * s) & (s < 2.0 ** 64), 2 * s, s)
    return s


def rms(x, w, eps):
    x = x.double()
    return x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def rotate(y, positions, table, interleaved):
    """y [T, H, d] fp64; the pairs of the first rot dims turn by their angles."""
    if table is None:
        return y
    half = table.shape[1] // 2
    out = y.clone()
    for t, p in enumerate(positions):
        if not 0 <= p < table.shape[0]:
            continue
        c, s = table[p, :half].double(), table[p, half:].double()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[t, :, a] = y[t, :, a] * c[i] - y[t, :, b] * s[i]
            out[t, :, b] = y[t, :, b] * c[i] + y[t, :, a] * s[i]
    return out


def table(positions, rot):
    """cos then sin of every position's angles, from fp64."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def append(y, cu, lens, pages, codes, scale, limit):
    """Stores y [total, Hk, d] fp64 into codes (fp64 values) and scale (fp64),
    both updated; returns a mask of the codes that were written or re-rounded
    and the values (already divided by the scale) that stand there."""
    want = codes.clone()
    touched = torch.zeros_like(codes, dtype=torch.bool)
    for b, n in enumerate(lens):
        new = cu[b + 1] - cu[b]
        at = n - new
        if new <= 0 or at < 0:
            continue
        end = min(n, limit)
        while at < end:
            page, off = int(pages[b, at // PAGE]), at % PAGE
            m = min(PAGE - off, end - at)
            rows = y[cu[b + 1] - n + at:][:m].transpose(0, 1)
            if 0 <= page < codes.shape[0]:
                mag = torch.where(torch.isfinite(rows), rows.abs(), 0.0)
                s = page_scale(mag.amax((1, 2)))
                if off:
                    s = torch.maximum(s, scale[page])
                    grown = (s > scale[page])[:, None, None]
                    again = e4m3(codes[page, :, :off] * (scale[page] / s)[:, None, None])
                    codes[page, :, :off] = torch.where(grown, again, codes[page, :, :off])
                    want[page, :, :off] = codes[page, :, :off]
                    touched[page, :, :off] = grown
                want[page, :, off:off + m] = rows / s[:, None, None]
                codes[page, :, off:off + m] = e4m3(rows / s[:, None, None])
                touched[page, :, off:off + m] = True
                scale[page] = s
            at += m
    return touched, want


def keys_of(b, n, pages, codes, scale, hk):
    """fp64 rows of sequence b's first n positions of one head and which of
    them are on a page of the cache."""
    d = codes.shape[3]
    x = torch.zeros((n, d), dtype=torch.float64)
    held = torch.zeros(n, dtype=torch.bool)
    for j0 in range(0, n, PAGE):
        page = int(pages[b, j0 // PAGE])
        m = min(PAGE, n - j0)
        if 0 <= page < codes.shape[0]:
            x[j0:j0 + m] = codes[page, hk, :m].double() * scale[page, hk].double()
            held[j0:j0 + m] = True
    return x, held


def attention(q, kc, vc, ks, vs, cu, lens, pages, scale, causal, window):
    """(O, LSE [H, T], W, A): W = sum p |v| and A = the largest scale * sum
    |q k| of each row, which the tolerances count in."""
    T, H, d = q.shape
    hks = kc.shape[1]
    o = torch.zeros((T, H, d), dtype=torch.float64)
    w = torch.zeros((T, H, d), dtype=torch.float64)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    big = torch.zeros((H, T), dtype=torch.float64)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        keys = min(max(length, 0), pages.shape[1] * PAGE)
        if n <= 0 or keys == 0:
            continue
        for hk in range(hks):
            k, held = keys_of(b, keys, pages, kc, ks, hk)
            v, _ = keys_of(b, keys, pages, vc, vs, hk)
            for i in range(n):
                at = length - n + i
                j = torch.arange(keys)
                seen = held.clone()
                if causal:
                    seen &= j <= at
                if window >= 0:
                    seen &= j >= at - window
                if not seen.any():
                    continue
                for h in range(hk * (H // hks), (hk + 1) * (H // hks)):
                    row = q[cu[b] + i, h].double()
                    x = k[seen] @ row * scale
                    top = x.max()
                    p = torch.exp(x - top)
                    o[cu[b] + i, h] = p @ v[seen] / p.sum()
                    w[cu[b] + i, h] = p @ v[seen].abs() / p.sum()
                    lse[h, cu[b] + i] = top + torch.log(p.sum())
                    big[h, cu[b] + i] = (k[seen].abs() @ row.abs()).max() * scale
    return o, lse, w, big


# ------------------------------------------------------------------ inputs
def cum(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32)


def make_pages(lens, gen, spare=3, width=None):
    """A page table over scattered pages; entries past a length are -7 (read,
    they would be caught, or far outside the cache)."""
    need = [-(-n // PAGE) for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=gen, dtype=torch.int32)
    t = torch.full((len(lens), width or max(1, max(need))), -7, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        t[b, :m] = perm[at:at + m]
        at += m
    return t, sum(need) + spare


def make_cache(lens, pages, num_pages, hk, d, gen, spread=3, size=1.0):
    """Random codes in the slots the sequences hold, NaN codes and NaN scales
    everywhere else; scales are powers of two `spread` apart at most."""
    codes = torch.full((num_pages, hk, PAGE, d), NAN_CODE, dtype=torch.uint8)
    codes = codes.view(torch.float8_e4m3fn)
    scale = torch.full((num_pages, hk), math.nan)
    for b, n in enumerate(lens):
        for j0 in range(0, n, PAGE):
            page, m = int(pages[b, j0 // PAGE]), min(PAGE, n - j0)
            x = torch.randn((hk, m, d), generator=gen) * size
            s = page_scale(x.abs().amax((1, 2)).double()).float()
            s = s * torch.exp2(torch.randint(0, spread + 1, (hk,), generator=gen).float())
            codes[page, :, :m] = (x / s[:, None, None]).to(torch.float8_e4m3fn)
            scale[page] = s
    return codes, scale
