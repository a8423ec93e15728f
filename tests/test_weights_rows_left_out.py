"""GPU: rows whose LSE is -inf add nothing to fa_paged_key_weights, whatever they hold
(rows of padding, that saw no key, or that the caller leaves out)."""
import math

import pytest
import torch

import paged_plain as plain
import varlen_flashattention_forward_gb300 as fa

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3.0e38])
@pytest.mark.parametrize("rows,group", [(1, 4), (3, 4), (7, 4), (16, 4), (40, 4)])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_rows_without_an_lse_add_nothing(cuda_device, rows, group, d, bad):
    # The same sums, bit by bit, as with zeros in those rows; long enough for tiles
    # that all rows see whole.
    gen = torch.Generator().manual_seed(rows + d)
    Hk, H, lens = 2, 2 * group, [500]
    pages, num = plain.make_pages(lens, gen)
    codes, scale = plain.make_cache(lens, pages, num, Hk, d, gen)
    q = torch.randn((rows, H, d), generator=gen).bfloat16()
    lse = torch.rand((H, rows), generator=gen) * 3 + 5
    lse[torch.rand(lse.shape, generator=gen) < 0.4] = -math.inf
    lse[1, 0], lse[2, 0] = -math.inf, 6.0
    out = torch.isinf(lse).t()
    got = []
    for fill in (0.0, bad):
        filled = q.clone()
        filled[out] = fill
        one = filled.clone()
        one[out] = 0.0
        one[..., d // 2][out] = fill      # one such value in the row
        for x in (filled, one):
            sums = torch.zeros((1, Hk, 500), device="cuda")
            fa.fa_paged_key_weights(x.cuda(), lse.cuda(), codes.cuda(), scale.cuda(), i32([0, rows]),
                                    i32(lens), pages.cuda(), sums)
            torch.cuda.synchronize()
            got.append(sums)
    assert fa.fa_get_device_status() == fa.FA_OK
    assert torch.isfinite(got[0]).all() and (got[0] > 0).any()
    assert all(torch.equal(g, got[0]) for g in got[1:])
