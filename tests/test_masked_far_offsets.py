"""GPU: the masked attentions and the eviction where offsets pass 32 bits: the same pages
far behind in a large cache, and rows of weights far behind in a large array, give the
same bits as in small ones."""
import pytest
import torch

import masked_plain as masked
import paged_plain as plain
import varlen_flashattention_forward_gb300 as fa

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_pages_far_behind_in_the_cache(cuda_device):
    gen = torch.Generator().manual_seed(1)
    Hk, H, d, q_lens, lens = 8, 16, 128, [20, 3, 1], [400, 130, 64]
    pages, num = plain.make_pages(lens, gen)
    made = [plain.make_cache(lens, pages, num, Hk, d, gen) for _ in range(2)]
    far = 2 ** 32 // (Hk * 64 * d) + 5           # pages before: their codes pass 2^32 bytes
    mask = masked.tree_masks([masked.random_parents(n, n) for n in q_lens], 1).cuda()
    q = torch.randn((24, H, d), generator=gen).bfloat16().cuda()
    cu, ld = plain.cum(q_lens).cuda(), i32(lens)
    first = i32([350, 100, 10])
    keep = torch.stack([torch.arange(4) * 9 + f for f in (355, 101, 12)]).int()[:, None].cuda()
    got = []
    for ahead in (0, far):
        cache = []
        for codes, scale in made:
            c = torch.zeros((ahead + num, Hk, 64, d), dtype=torch.float8_e4m3fn, device="cuda")
            s = torch.ones((ahead + num, Hk), device="cuda")
            c[ahead:], s[ahead:] = codes.cuda(), torch.nan_to_num(scale, 1.0).cuda()
            cache += [c, s]
        cache = [cache[0], cache[2], cache[1], cache[3]]
        pd = (pages + (pages >= 0) * ahead).int().cuda()
        out = []
        for kw in (dict(max_seqlen_q=20, tree_mask=mask), dict(max_seqlen_q=1, tree_mask=mask),
                   dict(max_seqlen_q=20, window_left=90, sink_tokens=5)):
            out += fa.fa_paged_attn(q, *cache, cu, ld, pd, return_lse=True, **kw)
        lse = out[-1]
        for rows in (24, 3):                      # 40 and 2 rows of a group
            sums = torch.zeros((3, Hk, 500), device="cuda")
            at = cu if rows == 24 else i32([0, 1, 2, 3])
            fa.fa_paged_key_weights(q[:rows], lse[:, :rows].contiguous(), cache[0], cache[2], at,
                                    ld, pd, sums, window_left=90, sink_tokens=5)
            out.append(sums)
        fa.fa_paged_kv_compact(*cache, pd, keep, i32([4, 4, 4]), first=first)
        out += [cache[0][ahead:].view(torch.uint8).clone(), cache[1][ahead:].view(torch.uint8).clone(),
                cache[2][ahead:].clone(), cache[3][ahead:].clone()]
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        got.append(out)
        del cache
    assert all(torch.equal(a.nan_to_num(7), b.nan_to_num(7)) for a, b in zip(*got))


def test_rows_of_weights_far_behind(cuda_device):
    # The last sequence's row starts past 2^31 numbers.
    gen = torch.Generator().manual_seed(2)
    Hk, d, n = 2, 64, 700
    pages, num = plain.make_pages([n], gen)
    made = [plain.make_cache([n], pages, num, Hk, d, gen) for _ in range(2)]
    q = torch.randn((1, 4, d), generator=gen).bfloat16().cuda()
    lse = torch.full((4, 1), 6.0, device="cuda")
    got = []
    for batch, capacity in ((1, 704), (5, 2 ** 28)):
        cache = [c.cuda() for c, _ in made] + [torch.nan_to_num(s, 1.0).cuda() for _, s in made]
        pd = torch.full((batch, pages.shape[1]), -1, dtype=torch.int32, device="cuda")
        pd[-1] = pages[0].cuda()
        lens = i32([0] * (batch - 1) + [n])
        cu = i32([0] * batch + [1])
        sums = torch.zeros((batch, Hk, capacity), device="cuda")
        fa.fa_paged_key_weights(q, lse, cache[0], cache[2], cu, lens, pd, sums)
        was = sums[-1, :, :n].clone()
        keep, new = fa.fa_paged_kv_select(sums, lens, 200, sink_tokens=3, recent_tokens=20)
        fa.fa_paged_kv_compact(*cache, pd, keep, new, weights=sums)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        assert not sums[:-1].any()
        got.append([was, sums[-1, :, :n].clone(), keep[-1], new[-1:], cache[0].view(torch.uint8),
                    cache[1].view(torch.uint8), cache[2], cache[3]])
        del sums
    assert all(torch.equal(a, b) for a, b in zip(*got))
