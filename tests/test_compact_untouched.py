"""What fa_paged_kv_compact must leave alone, byte for byte: pages that it does not move,
slots behind the last row, slots before the first one where the page's scale does not
grow.  Codes are any bytes, so that a slot that is written again with the same number
(-0 as 0, one NaN as the other) shows."""
import pytest
import torch

import masked_plain as masked
import paged_plain as plain
import varlen_flashattention_forward_gb300 as fa


def untouched(codes, scale, pages, keep, first, counts):
    """Truth values [pages, Hk, 64] of the slots that keep their bytes and [pages, Hk]
    of the scales that stay; codes fp8, before the move."""
    num, hks = scale.shape
    slots = torch.ones((num, hks, 64), dtype=torch.bool)
    scales = torch.ones((num, hks), dtype=torch.bool)
    _, new = masked.compact(codes.double(), scale.double(), pages, keep, first, counts)
    for b in range(pages.shape[0]):
        f = max(first[b], 0)
        end = f + min(max(counts[b], 0), keep.shape[2], max(pages.shape[1] * 64 - f, 0))
        for h in range(hks):
            src = keep[b, h if keep.shape[1] > 1 else 0].tolist()
            for lo in range(f // 64 * 64, end, 64):
                here = range(max(lo, f), min(lo + 64, end))
                page = int(pages[b, lo // 64])
                if not 0 <= page < num or all(src[s - f] == s for s in here):
                    continue
                scales[page, h] = False
                slots[page, h, here[0] - lo:here[-1] + 1 - lo] = False
                if here[0] > lo and new[page, h] > scale[page, h]:
                    slots[page, h, :here[0] - lo] = False
    return slots, scales


def kept(before, after, slots):
    """Whether the bytes of the slots that must not change are the same."""
    a, b = before.view(torch.uint8), after.view(torch.uint8)
    return torch.equal(a[slots], b[slots])


def case(kind, heads, seed):
    gen = torch.Generator().manual_seed(seed)
    Hk, d = 2, 64
    lens = [300, 130, 70, 64, 191, 40]
    pages, num = plain.make_pages(lens, gen)
    caches = []
    for _ in range(2):
        raw = torch.randint(0, 256, (num, Hk, 64, d), generator=gen).to(torch.uint8)
        raw[torch.rand(raw.shape, generator=gen) < 0.05] = 0x80
        raw[torch.rand(raw.shape, generator=gen) < 0.05] = 0xff
        s = torch.exp2(torch.randint(-3, 4, (num, Hk), generator=gen).float())
        caches.append((raw.view(torch.float8_e4m3fn), s))
    first = [0] * 6 if kind == "evict" else [237, 127, 0, 63, 64, 30]
    n = 150 if kind == "evict" else 7
    keep = torch.full((6, heads, n), -1, dtype=torch.int32)
    counts = [min(n, m - f) for m, f in zip(lens, first)]
    for b, (m, f, c) in enumerate(zip(lens, first, counts)):
        for h in range(heads):
            some = torch.randperm(m - f, generator=gen)[:c].sort().values + f
            if b in (1, 4):  # keeps its first rows, and so whole pages of them
                some = torch.arange(f, f + c)
                if h == 0 and c > 70:
                    some[70:] += m - f - c
            keep[b, h, :c] = some.int()
    if kind == "path":  # a path that starts where it stands, rows behind it stay
        keep[0, :, :7] = torch.tensor([237, 238, 239, 240, 241, 242, 243]).int()
    return gen, pages, caches, keep, first, counts


KINDS = [("evict", 1), ("evict", 2), ("path", 1), ("path", 2)]


@pytest.mark.parametrize("kind,heads", KINDS)
def test_a_slot_that_is_written_again_shows(kind, heads):
    # (The mistakes are planted in a copy, on the CPU.)
    gen, pages, caches, keep, first, counts = case(kind, heads, 1)
    for codes, scale in caches:
        slots, scales = untouched(codes, scale, pages, keep, first, counts)
        assert slots.any() and not slots.all() and scales.any() and not scales.all()
        assert kept(codes, codes.clone(), slots)
        for was, now in ((0x80, 0x00), (0xff, 0x7f)):
            raw = codes.view(torch.uint8).clone()
            at = (raw == was) & slots[..., None]
            assert at.sum() > 100
            raw[tuple(at.nonzero()[0])] = now
            assert not kept(codes, raw.view(torch.float8_e4m3fn), slots)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,heads", KINDS)
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_bytes_that_must_not_change(cuda_device, kind, heads, seed):
    gen, pages, caches, keep, first, counts = case(kind, heads, seed)
    cards = [(c.cuda(), s.cuda()) for c, s in caches]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.fa_paged_kv_compact(cards[0][0], cards[1][0], cards[0][1], cards[1][1], pages.cuda(),
                           keep.cuda(), i32(counts), first=i32(first))
    torch.cuda.synchronize()
    for (codes, scale), (after, new) in zip(caches, cards):
        slots, scales = untouched(codes, scale, pages, keep, first, counts)
        assert kept(codes, after.cpu(), slots)
        assert torch.equal(new.cpu()[scales], scale[scales])
        want, ws = masked.compact(codes.double(), scale.double(), pages, keep, first, counts)
        assert torch.equal(new.cpu().double(), ws)
        assert torch.equal(torch.nan_to_num(after.cpu().double(), 777.0),
                           torch.nan_to_num(want, 777.0))
