"""How exact fa_paged_key_weights is, at queries whose bits matter.

A weight is exp(x - lse), x = scale q.k.  Its exponent may be off by

  2^-24 mx scale sum |k|      a row of q is held to 2^-24 of its largest value mx
  2^-18 A, A = scale sum |q k|  sums of products on the tensor core: at most 3 D / 32 = 12
                              steps, each cut once to fp32 (2^-23 of up to 1.13 A, the terms'
                              magnitudes together), the join of two sums, and as much again
  2^-22 (|x| + |lse|)         fp32: the two factors, the LSE in base 2, the difference

and a sum of R weights by (R + 8) 2^-23 of itself (2^-22 of each exponential among it).

The queries have one loud channel, where every key is 0: all of a score comes from
values far below the row's largest.  Two terms of 8 bits, or three of which the second
is e4m3, miss these bounds there (the first tests, on the CPU).
"""
import math

import pytest
import torch

import paged_plain as plain
import varlen_flashattention_forward_gb300 as fa


def e5m2(x):
    """x (fp64) rounded to the nearest e5m2 value, ties to even."""
    m, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-14).double() - 2)
    return torch.round(x / step) * step


def held_as(y, second, third):
    """y, scaled so that its row's largest is in [128, 256), as the sum of an e4m3 term and
    two more (None: none)."""
    total = plain.e4m3(y)
    for f in (second, third):
        if f is not None:
            total = total + f(y - total)
    return total


# --------------------------------------------------------------------- CPU
def every_bf16(lo, hi):
    """All bf16 numbers of [2^lo, 2^hi)."""
    m = 1 + torch.arange(128, dtype=torch.float64) / 128
    return (m[None] * torch.exp2(torch.arange(lo, hi, dtype=torch.float64))[:, None]).flatten()


def test_an_e4m3_and_two_e5m2_terms_hold_a_row_to_24_bits():
    y = every_bf16(-40, 8)
    off = (held_as(y, e5m2, e5m2) - y).abs()
    assert (off <= 2.0 ** -24 * 128).all()
    # Everything from 2^-8 of the row's largest on is held exactly.
    assert (off[y >= 2.0 ** -9] == 0).all()


def test_two_terms_or_an_e4m3_one_in_second_place_do_not():
    y = every_bf16(-40, 8)
    assert ((held_as(y, plain.e4m3, None) - y).abs().max() >= 2.0 ** -18 * 128)
    assert ((held_as(y, plain.e4m3, e5m2) - y).abs().max() >= 2.0 ** -22 * 128)


# ------------------------------------------------------------------ inputs
def inputs(rows, length, Hk, group, d, seed, kind):
    """One sequence: q [rows, Hk * group, d] bf16 and a cache; scale 2^-3."""
    gen = torch.Generator().manual_seed(seed)
    H = Hk * group
    loud = torch.arange(H) % d
    if kind == "same":
        # One value in all channels of a row, of which two e5m2 terms keep the last four
        # bits, one loses them, and two e4m3 terms keep nothing; keys of one sign.
        m = torch.tensor([13, 14, 15, 45, 46, 47, 77, 78, 79])
        m = m[torch.randint(0, 9, (rows, H, 1), generator=gen)]
        y = (2.0 ** -11 * (1 + m / 128)).expand(rows, H, d).clone()
        big = torch.full((rows, H), 128.0)
    else:
        y = torch.exp2(torch.rand((rows, H, d), generator=gen) * 8 - 12)
        y = y * (torch.randint(0, 2, y.shape, generator=gen) * 2 - 1)
        big = 128 + torch.randint(0, 128, (rows, H), generator=gen).float()
    # (Rows of one kv head share its keys, so all of them are loud in one channel.)
    channel = (loud // group * group)[None, :, None].expand(rows, H, 1)
    y.scatter_(2, channel, big[..., None])
    unit = torch.exp2(torch.randint(-3, 2, (rows, H, 1), generator=gen).float())
    q = (y * unit).bfloat16()
    pages = -(-length // 64)
    table = torch.randperm(pages + 2, generator=gen)[:pages].int()[None]
    codes = torch.randint(-448, 449, (pages + 2, Hk, 64, d), generator=gen).float()
    if kind == "same":
        codes = codes.abs()
    for h in range(Hk):
        codes[:, h, :, int(channel[0, h * group, 0])] = 0
    codes = codes.to(torch.float8_e4m3fn)
    scale = torch.exp2(torch.randint(-1, 2, (pages + 2, Hk), generator=gen).float())
    return q, codes, scale, table


def weights_and_tolerance(q, codes, scale, table, length, factor, term=None):
    """(sums [Hk, length], their tolerance, lse [H, rows] fp32), causal, decay 0, q as
    it is or as `term` holds it (the tolerance is that of q itself)."""
    rows, H, d = q.shape
    Hk = codes.shape[1]
    lse = torch.empty((H, rows))
    sums = torch.zeros((Hk, length), dtype=torch.float64)
    tol = torch.zeros_like(sums)
    R = rows * (H // Hk) + 8
    for h in range(H):
        hk = h // (H // Hk)
        k, _ = plain.keys_of(0, length, table, codes, scale, hk)
        for i in range(rows):
            row = q[i, h].double()
            seen = length - rows + i + 1
            x = k[:seen] @ row * factor
            lse[h, i] = torch.logsumexp(x, 0).float()
            L = lse[h, i].double()
            mx = row.abs().max()
            e = (2.0 ** -24 * mx * factor * k[:seen].abs().sum(1)
                 + 2.0 ** -18 * factor * (k[:seen].abs() @ row.abs())
                 + 2.0 ** -22 * (x.abs() + L.abs()))
            p = torch.exp(x - L)
            tol[hk, :seen] += p * (torch.expm1(e) + R * 2.0 ** -23)
            if term is not None:
                up = 2.0 ** (7 - math.floor(math.log2(mx)))
                p = torch.exp(k[:seen] @ (term(row * up) / up) * factor - L)
            sums[hk, :seen] += p
    return sums, tol + 1e-37, lse


CASES = [(1, 1, 4), (1, 2, 16), (7, 2, 4), (16, 2, 4), (40, 1, 4)]  # 4, 16, 28, 64, 160 rows
LENGTH, FACTOR = 300, 0.125


@pytest.mark.parametrize("rows,Hk,group", CASES)
def test_a_term_that_is_missing_exceeds_the_tolerance(rows, Hk, group):
    case = inputs(rows, LENGTH, Hk, group, 64, rows + group, "same")
    want, tol, _ = weights_and_tolerance(*case, LENGTH, FACTOR)

    def worst(*terms):
        got, _, _ = weights_and_tolerance(*case, LENGTH, FACTOR, lambda y: held_as(y, *terms))
        return ((got - want).abs() / tol).max()
    assert worst(e5m2, e5m2) <= 1
    assert worst(e5m2, None) > 2 and worst(plain.e4m3, None) > 2
    assert worst(e5m2, lambda y: -e5m2(y)) > 2    # with the wrong sign
    assert worst(plain.e4m3, e5m2) > 2


# --------------------------------------------------------------------- GPU
def run(q, codes, scale, table, length, lse, factor):
    rows, Hk = q.shape[0], codes.shape[1]
    sums = torch.full((1, Hk, length), torch.nan, device="cuda")
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, rows], [length]))
    fa.fa_paged_key_weights(q.cuda(), lse.cuda(), codes.cuda(), scale.cuda(), cu, lens, table.cuda(),
                            sums, softmax_scale=factor, decay=0.0)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    return sums[0].cpu().double()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["same", "mixed"])
@pytest.mark.parametrize("rows,Hk,group", CASES)
@pytest.mark.parametrize("d", [64, 80, 96, 128])
def test_small_values_beside_a_loud_channel(cuda_device, rows, Hk, group, d, kind):
    case = inputs(rows, LENGTH, Hk, group, d, rows + group + d, kind)
    want, tol, lse = weights_and_tolerance(*case, LENGTH, FACTOR)
    got = run(*case, LENGTH, lse, FACTOR)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,Hk,group", CASES)
@pytest.mark.parametrize("d", [64, 80, 96, 128])
def test_ordinary_queries(cuda_device, rows, Hk, group, d):
    # Normal q, keys with channels eight times louder, scores up to some 40.
    gen = torch.Generator().manual_seed(rows + d)
    lens = [LENGTH]
    pages, num = plain.make_pages(lens, gen)
    codes, scale = plain.make_cache(lens, pages, num, Hk, d, gen, 2)
    q = torch.randn((rows, Hk * group, d), generator=gen)
    q[..., 5::16] *= 4
    q = q.bfloat16()
    want, tol, lse = weights_and_tolerance(q, codes, scale, pages, LENGTH, FACTOR)
    got = run(q, codes, scale, pages, LENGTH, lse, FACTOR)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
