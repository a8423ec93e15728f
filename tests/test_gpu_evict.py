"""GPU: attention weights of cached keys, the choice of the keys to keep, and
the cache moved together, against their plain fp64 forms.

Weights: the tolerance is counted in masked_plain.key_weights.  Choices are
whole numbers and equal.  A move is exact but for codes that a larger scale
rounds again, which are rounded the same way.
"""
import pytest
import torch

import masked_plain as masked
import paged_plain as plain
import varlen_flashattention_forward_gb300 as fa

pytestmark = pytest.mark.gpu


def dev(*ts):
    got = [None if t is None else t.cuda() for t in ts]
    return got if len(got) > 1 else got[0]


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ----------------------------------------------------------------- weights
def check_weights(q_lens, lens, H, Hk, d, causal=True, window=-1, sinks=0, decay=1.0, seed=0,
                  capacity=None, break_pages=None, lens_given=None, stream=None, lse=None, size=1.0,
                  strided=False):
    gen = torch.Generator().manual_seed(seed)
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, Hk, d, gen) for _ in range(2))
    if break_pages:
        break_pages(pages, num)
    cu = plain.cum(q_lens)
    T = int(cu[-1])
    q = (torch.randn((T, H, d), generator=gen) * size).bfloat16()
    given = lens if lens_given is None else lens_given
    capacity = capacity or pages.shape[1] * 64
    sums = torch.rand((len(lens), Hk, capacity), generator=gen)
    for b, (n, m) in enumerate(zip(q_lens, given)):  # what must not be read
        sums[b, :, max(m - n, 0):max(m, 0)] = torch.nan
        if decay == 0 and n:
            sums[b, :, :max(m, 0)] = torch.nan
    wide = torch.empty((T, H + 3, d), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = dev(q)
    qd = wide[:, :H] if strided else dev(q)
    kcd, vcd, ksd, vsd, cud, ld, pd, sd = dev(kc, vc, ks, vs, cu, i32(given), pages, sums)
    if lse is None:
        _, lse = fa.fa_paged_attn(qd, kcd, vcd, ksd, vsd, cud, ld, pd, causal=causal,
                                  window_left=window, sink_tokens=sinks, return_lse=True)
    else:
        lse = dev(lse)
    torch.cuda.synchronize()
    fa.fa_paged_key_weights(qd, lse, kcd, ksd, cud, ld, pd, sd, causal=causal, window_left=window,
                            sink_tokens=sinks, decay=decay, stream=stream)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    want, tol = masked.key_weights(q, lse.cpu(), kc, ks, cu.tolist(), given, pages, sums, d ** -0.5,
                                   causal, window, sinks, decay)
    got = sd.cpu().double()
    for b, (n, m) in enumerate(zip(q_lens, given)):
        m = max(0, min(m, capacity)) if n else 0
        assert ((got[b, :, :m] - want[b, :, :m]).abs() <= tol[b, :, :m]).all(), b
        assert torch.equal(torch.nan_to_num(got[b, :, m:], 7.0),
                           torch.nan_to_num(sums[b, :, m:].double(), 7.0)), b
    return sd


@pytest.mark.parametrize("d", [64, 80, 96, 128])
@pytest.mark.parametrize("H,Hk", [(4, 4), (8, 2), (16, 1), (6, 2)])
@pytest.mark.parametrize("decay", [0.0, 0.75, 1.0])
def test_weights_dims(cuda_device, d, H, Hk, decay):
    check_weights([1, 1, 1], [130, 300, 64], H, Hk, d, decay=decay, seed=d + H)


@pytest.mark.parametrize("q_lens,lens", [
    ([1], [1]), ([1], [2]), ([1, 1], [128, 129]), ([2, 7, 3], [64, 63, 300]), ([17], [100]),
    ([0, 3, 0, 1], [50, 3, 0, 129]), ([40], [200]), ([70, 9], [200, 400]), ([200], [200]),
    ([5, 9], [2, 8]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_weights_many_rows(cuda_device, q_lens, lens, causal):
    check_weights(q_lens, lens, 8, 2, 64, causal=causal, seed=sum(lens))
    check_weights(q_lens, lens, 4, 1, 128, causal=causal, decay=0.0, seed=sum(lens))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 2), (63, 0), (128, 5), (300, 130), (1000, 9)])
@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
def test_weights_windows(cuda_device, window, sinks, decay):
    # Tiles that no row sees only decay; chunks of rows whose windows differ.
    check_weights([1, 3, 90], [900, 129, 700], 4, 2, 64, window=window, sinks=sinks, decay=decay,
                  seed=window)


def test_weights_long_contexts_and_many_sequences(cuda_device):
    check_weights([1, 1], [9000, 5001], 8, 2, 128, seed=31)
    check_weights([32], [20000], 4, 1, 64, decay=0.0, seed=32)
    lens = [1 + 37 * i % 260 for i in range(1100)]  # several launches
    check_weights([1] * 1100, lens, 2, 1, 64, seed=33)


def test_weights_capacity_below_and_above_the_table(cuda_device):
    check_weights([1, 2], [300, 129], 4, 2, 64, capacity=200, seed=34)
    check_weights([1, 2], [300, 129], 4, 2, 64, capacity=1001, seed=35)
    check_weights([1, 2], [130, 64], 4, 2, 64, lens_given=[130, 1000], seed=36)
    check_weights([1, 2], [130, 64], 4, 2, 64, lens_given=[-5, 64], seed=37)


def test_weights_on_missing_pages(cuda_device):
    def break_pages(pages, num):
        pages[0, 0], pages[0, 2], pages[1, 0] = num, -1, 2 ** 31 - 1
    check_weights([1, 3], [300, 64], 8, 2, 128, break_pages=break_pages, seed=38)


def test_weights_given_lse_strided_q_other_stream(cuda_device):
    gen = torch.Generator().manual_seed(39)
    lse = torch.rand((4, 3), generator=gen) * 3
    lse[1, 0], lse[2, 2] = -torch.inf, -torch.inf
    check_weights([1, 2], [200, 129], 4, 2, 64, lse=lse, strided=True, seed=39)
    check_weights([1, 2], [200, 129], 4, 2, 96, stream=torch.cuda.Stream(), seed=40)
    check_weights([1, 2], [200, 129], 4, 2, 96, size=20.0, seed=41)


def test_weights_add_up_to_the_rows(cuda_device):
    # Every row's weights sum to 1 over the keys it sees.
    sums = check_weights([5], [1000], 8, 2, 128, decay=0.0, seed=42)
    assert ((sums.double()[0, :, :1000].sum(-1) - 20).abs() <= 20 * 2.0 ** -10).all()


def test_weights_runs_are_bitwise_the_same_and_malformed_cu_seqlens(cuda_device):
    a = check_weights([3, 40], [5000, 300], 8, 2, 128, seed=43)
    b = check_weights([3, 40], [5000, 300], 8, 2, 128, seed=43)
    assert torch.equal(a.nan_to_num(7), b.nan_to_num(7))
    gen = torch.Generator().manual_seed(44)
    lens = [100, 100, 100]
    pages, num = plain.make_pages(lens, gen)
    kc, ks = plain.make_cache(lens, pages, num, 2, 64, gen)
    q = dev(torch.randn((6, 4, 64), generator=gen).bfloat16())
    lse = torch.zeros((4, 6), device="cuda")
    for cu in ([0, 50, 3, 6], [-9, 2, 4, 2 ** 31 - 1], [5, 4, 3, 2]):
        sums = torch.full((5, 2, 128), 7.0, device="cuda")
        fa.fa_paged_key_weights(q, lse, *dev(kc, ks, i32(cu), i32(lens), pages), sums[1:4])
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        assert (sums[0] == 7).all() and (sums[4] == 7).all() and (sums[1:4, :, 100:] == 7).all()


def test_weights_wait_limit_runs_out_then_recovers(cuda_device):
    gen = torch.Generator().manual_seed(45)
    lens = [3000] * 4
    pages, num = plain.make_pages(lens, gen)
    kc, ks = plain.make_cache(lens, pages, num, 2, 128, gen)
    q = torch.randn((80, 8, 128), generator=gen).bfloat16()
    args = dev(q, torch.full((8, 80), 8.0), kc, ks, plain.cum([20] * 4), i32(lens), pages)

    def call():
        sums = torch.zeros((4, 2, 3008), device="cuda")
        fa.fa_paged_key_weights(*args, sums, decay=0.0)
        return sums
    want = call()
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    fa.fa_set_wait_limit_ns(2000)
    try:
        call()
        assert fa.fa_get_device_status() == fa.FA_ERR_DEVICE_TIMEOUT
    finally:
        fa.fa_set_wait_limit_ns(0)
    got = call()
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK and torch.equal(got, want)


# ------------------------------------------------------------------ select
def check_select(sums, lens, budget, sinks=0, recent=0, stream=None):
    keep, new = fa.fa_paged_kv_select(*dev(sums, i32(lens)), budget, sink_tokens=sinks,
                                      recent_tokens=recent, stream=stream)
    torch.cuda.synchronize()
    want, wn = masked.select(sums, lens, budget, sinks, recent)
    assert torch.equal(new.cpu(), wn)
    assert torch.equal(keep.cpu(), want)


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 1023, 1024, 1025, 2500, 9000])
@pytest.mark.parametrize("budget", [1, 2, 64, 1000])
def test_select_sizes(cuda_device, n, budget):
    gen = torch.Generator().manual_seed(n + budget)
    sums = torch.rand((2, 3, max(n, 1) + 5), generator=gen)
    check_select(sums, [n, n // 2], budget)
    check_select(sums, [n, n + 5], budget, sinks=budget // 3, recent=budget // 2)
    check_select(sums, [n, -3], budget, sinks=budget // 2, recent=budget - budget // 2)


def test_select_ties_and_special_values(cuda_device):
    gen = torch.Generator().manual_seed(1)
    n = 3000
    zero = torch.zeros((1, 1, n))
    check_select(zero, [n], 700, sinks=3, recent=50)
    few = torch.randint(0, 3, (2, 2, n), generator=gen).float()
    check_select(few, [n, 2999], 1500, sinks=4)
    signed = torch.randn((1, 2, n), generator=gen)
    signed[..., ::7] = 0.0
    signed[..., 3::7] = -0.0
    signed[..., 5::11] = torch.nan
    signed[..., 1::13] = -torch.inf
    signed[..., 2::13] = torch.inf
    signed[..., 4::17] = 1e-40
    for budget in (5, 1000, 1800, 2900):
        check_select(signed, [n], budget, recent=2)
    check_select(torch.full((1, 1, n), torch.nan), [n], 10)


def test_select_close_values_long_and_many(cuda_device):
    gen = torch.Generator().manual_seed(2)
    near = (1.0 + torch.randint(0, 4000, (1, 2, 70000), generator=gen).float() * 2.0 ** -23)
    check_select(near, [70000], 30000, sinks=4, recent=1000)
    check_select(torch.rand((300, 2, 200), generator=gen).exp(), [i % 201 for i in range(300)], 77,
                 sinks=1, recent=20)
    check_select(torch.rand((1, 1, 500), generator=gen), [500], 60, stream=torch.cuda.Stream())


def test_select_given_outputs_and_refusals(cuda_device):
    sums = torch.rand((2, 2, 100), device="cuda")
    lens = dev(i32([100, 50]))
    keep = torch.empty((2, 2, 10), dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    got = fa.fa_paged_kv_select(sums, lens, 10, keep=keep, new_lens=new)
    assert got[0] is keep and got[1] is new and new.cpu().tolist() == [10, 10]
    with pytest.raises(ValueError):
        fa.fa_paged_kv_select(sums, lens, 10, new_lens=lens)
    for kw in (dict(budget=0), dict(budget=5, sink_tokens=4, recent_tokens=2),
               dict(budget=5, sink_tokens=-1), dict(budget=5, recent_tokens=2 ** 40)):
        with pytest.raises(fa.FaError):
            fa.fa_paged_kv_select(sums, lens, **kw)


# ----------------------------------------------------------------- compact
def make_both(lens, Hk, d, gen, spread=3, width=None, spare=3):
    pages, num = plain.make_pages(lens, gen, width=width, spare=spare)
    caches = [plain.make_cache(lens, pages, num, Hk, d, gen, spread) for _ in range(2)]
    # (Scales of pages that hold nothing are numbers too where rows may land.)
    return pages, num, [(c, torch.where(torch.isnan(s), 1.0, s)) for c, s in caches]


def check_compact(caches, pages, keep, counts, first=None, sums=None, stream=None):
    cards = [dev(c, s) for c, s in caches]
    sd = None if sums is None else dev(sums)
    fd = None if first is None else dev(i32(first))
    args = dev(pages, keep, i32(counts))
    torch.cuda.synchronize()
    fa.fa_paged_kv_compact(cards[0][0], cards[1][0], cards[0][1], cards[1][1], *args, first=fd,
                           weights=sd, stream=stream)
    torch.cuda.synchronize()
    at = [0] * len(counts) if first is None else first
    for (c, s), (cd, sc) in zip(caches, cards):
        want, ws = masked.compact(c.double(), s.double(), pages, keep, at, counts)
        assert torch.equal(sc.cpu().double(), ws)
        got = cd.cpu().double()
        assert torch.equal(torch.nan_to_num(got, 777.0), torch.nan_to_num(want, 777.0))
        # What does not change keeps its bits.
        same = torch.equal(cd.cpu().view(torch.uint8)[got == c.double()],
                           c.view(torch.uint8)[got == c.double()]) or (got == 0).any()
        assert same
    if sums is not None:
        want = masked.move_weights(sums, keep, at, counts, pages, caches[0][0].shape[0])
        assert torch.equal(sd.cpu(), want)
    return cards


def random_keep(lens, Hk, n, gen, first=None):
    """Ascending distinct slots, n at most of each sequence."""
    keep = torch.full((len(lens), Hk, n), -1, dtype=torch.int32)
    counts = []
    for b, m in enumerate(lens):
        f = 0 if first is None else first[b]
        c = min(n, m - f)
        counts.append(c)
        for h in range(Hk):
            keep[b, h, :c] = (torch.randperm(m - f, generator=gen)[:c].sort().values + f).int()
    return keep, counts


@pytest.mark.parametrize("d", [64, 80, 96, 128])
@pytest.mark.parametrize("n", [1, 63, 64, 65, 200])
def test_compact_dims(cuda_device, d, n):
    gen = torch.Generator().manual_seed(d + n)
    lens = [300, 129, 64, 1]
    pages, num, caches = make_both(lens, 3, d, gen)
    keep, counts = random_keep(lens, 3, n, gen)
    sums = torch.rand((4, 3, pages.shape[1] * 64), generator=gen)
    check_compact(caches, pages, keep, counts, sums=sums)


@pytest.mark.parametrize("heads", [1, 2])
def test_compact_behind_a_first_slot(cuda_device, heads):
    # Paths of drafted trees: earlier slots of the page stay and follow its scale.
    for seed in range(8):
        gen = torch.Generator().manual_seed(seed)
        lens = [300, 130, 70, 64, 191]
        first = [237, 127, 0, 63, 64]
        pages, num, caches = make_both(lens, 2, 64, gen, spread=6)
        keep, counts = random_keep(lens, heads, [1, 3, 9, 64][seed % 4], gen, first)
        sums = torch.rand((5, 2, 250), generator=gen)
        check_compact(caches, pages, keep, counts, first=first, sums=sums)


def test_compact_over_several_rounds_of_a_cluster(cuda_device):
    gen = torch.Generator().manual_seed(3)
    pages, num, caches = make_both([6000], 1, 128, gen)
    keep, counts = random_keep([6000], 1, 4001, gen)
    sums = torch.rand((1, 1, 6016), generator=gen)
    check_compact(caches, pages, keep, counts, sums=sums)
    # ... behind a first slot, and with the rows of the last pages alone.
    keep, counts = random_keep([6000], 1, 1500, gen, [1333])
    check_compact(caches, pages, keep, counts, first=[1333], sums=sums)
    keep = torch.arange(4500, 6000, dtype=torch.int32)[None, None]
    check_compact(caches, pages, keep, [1500], sums=sums)


def test_compact_many_sequences(cuda_device):
    gen = torch.Generator().manual_seed(4)
    lens = [1 + 29 * i % 300 for i in range(400)]
    pages, num, caches = make_both(lens, 2, 64, gen)
    keep, counts = random_keep(lens, 2, 100, gen)
    check_compact(caches, pages, keep, counts)


def test_compact_leaves_pages_whose_rows_stay(cuda_device):
    # With scales that are larger than they need to be, and shared pages.
    gen = torch.Generator().manual_seed(5)
    lens = [200, 250]
    pages, num, caches = make_both(lens, 2, 64, gen, spread=5)
    pages[1, :2] = pages[0, :2]
    keep = torch.arange(200, dtype=torch.int32).repeat(2, 2, 1)
    keep[1, 1, 140:] += 50   # one head of the second sequence moves, behind them
    cards = check_compact(caches, pages, keep, [200, 200])
    for (c, s), (cd, sc) in zip(caches, cards):
        for p in pages[0, :4].tolist() + [int(pages[1, 2])]:
            heads = [0, 1] if p != int(pages[1, 2]) else [0]
            for h in heads:
                assert torch.equal(cd.cpu().view(torch.uint8)[p, h], c.view(torch.uint8)[p, h])
                assert sc.cpu()[p, h] == s[p, h]


def test_compact_of_malformed_lists(cuda_device):
    gen = torch.Generator().manual_seed(6)
    lens = [300, 300]
    pages, num, caches = make_both(lens, 2, 64, gen)
    keep = torch.randint(-400, 800, (2, 2, 150), generator=gen, dtype=torch.int32)
    keep[0, 0, 3], keep[0, 1, 5] = 2 ** 31 - 1, -2 ** 31
    for counts, first in (([150, 2 ** 31 - 1], [0, 100]), ([-7, 150], [5, 2 ** 31 - 1]),
                          ([40, 150], [-9, 300])):
        check_compact(caches, pages, keep, counts, first=first,
                      sums=torch.rand((2, 2, 333), generator=gen))


def test_compact_with_missing_pages(cuda_device):
    gen = torch.Generator().manual_seed(7)
    lens = [300, 200]
    pages, num, caches = make_both(lens, 2, 64, gen)
    pages[0, 1], pages[0, 3], pages[1, 0], pages[1, 2] = num, -1, 2 ** 31 - 1, -2 ** 31
    keep, counts = random_keep(lens, 2, 120, gen)
    check_compact(caches, pages, keep, counts, sums=torch.rand((2, 2, 320), generator=gen))


def test_compact_special_codes_and_scales(cuda_device):
    # NaN codes move as they are and say nothing about the scale; rows of zeros;
    # scales at both ends.
    gen = torch.Generator().manual_seed(8)
    lens = [400]
    pages, num, caches = make_both(lens, 2, 64, gen)
    for c, s in caches:
        raw = c.view(torch.uint8)
        raw[torch.rand(raw.shape, generator=gen) < 0.02] = 0x7f
        raw[torch.rand(raw.shape, generator=gen) < 0.02] = 0xff
        raw[pages[0, 2].long()] = 0
        s[pages[0, 1].long()] = 2.0 ** 60
        s[pages[0, 3].long()] = 2.0 ** -60
        s[pages[0, 4].long()] = 0.0
    keep, counts = random_keep(lens, 2, 200, gen)
    check_compact(caches, pages, keep, counts)
    keep[..., 0] = 0
    check_compact(caches, pages, keep[..., :70].contiguous(), [70])


def test_compact_rows_of_zeros_under_scales_far_apart(cuda_device):
    # Zeros stay zeros whatever the quotient of the scales, past 32 bits too.
    gen = torch.Generator().manual_seed(12)
    pages, num, caches = make_both([256], 2, 64, gen)
    for c, s in caches:
        raw = c.view(torch.uint8)
        raw[pages[0].long()] = 0
        raw[pages[0, 2].long(), :, 5, 3] = 0x7f
        s[pages[0].long()] = 2.0 ** 64
        s[pages[0, 3].long()] = 2.0 ** -64
        raw[pages[0, 3].long(), 1, 9] = 0x31
    keep = torch.tensor([64, 67, 130, 133, 192, 200, 201, 255], dtype=torch.int32)[None, None]
    cards = check_compact(caches, pages, keep, [8])
    assert (cards[0][1].cpu()[pages[0, 0].long()] == 2.0 ** -64).all()


def test_compact_nothing_and_on_another_stream(cuda_device):
    gen = torch.Generator().manual_seed(9)
    pages, num, caches = make_both([100, 90], 2, 96, gen)
    check_compact(caches, pages, torch.empty((2, 1, 0), dtype=torch.int32), [5, 5])
    keep, counts = random_keep([100, 90], 1, 50, gen)
    check_compact(caches, pages, keep, [0, 0])
    check_compact(caches, pages, keep, counts, stream=torch.cuda.Stream())


# ---------------------------------------------------------- runs together
def attend(q, cache, cu, lens, pages, **kw):
    return fa.fa_paged_attn(q, *cache, cu, lens, pages, return_lse=True, **kw)


def held(cache, pages, b, n, which, h):
    """fp64 rows of one head's first n slots, and their page's scale."""
    codes, scale = cache[which].cpu(), cache[which + 2].cpu()
    x, _ = plain.keys_of(b, n, pages, codes, scale, h)
    s = scale[pages[b, torch.arange(n) // 64].long(), h].double()
    return x, s[:, None]


def assert_holds(got, scale, want):
    """Codes that stand for `want`, rounded to e4m3 at most twice under a scale
    no larger than the one they have."""
    assert ((got - want).abs() <= 2 * plain.e4m3_half_step(want / scale) * scale).all()


def assert_attends(o, lse, q, cache, cu, lens, pages, mask=None):
    c = [t.cpu() for t in cache]
    want = masked.paged_attention(q.cpu(), c[0], c[1], c[2], c[3], cu.tolist(), lens.tolist(), pages,
                                  q.shape[2] ** -0.5, mask=mask)
    wo, wl, w, big = want
    dx = 2.0 ** -15 * big  # (the tolerances of the paged attention)
    assert ((o.cpu().double() - wo).abs()
            <= 2.0 ** -8 * wo.abs() + (2 * dx.t()[..., None] + 2.0 ** -10) * w + 1e-30).all()
    assert ((lse.cpu().double() - wl).abs() <= dx + 2.0 ** -20 * (1 + wl.abs())).all()


def test_eviction_run(cuda_device):
    # Prompt, weights of its last rows, eviction, then decode steps with their
    # weights and a second eviction.  After each step the slots hold the tokens
    # that the choices kept, and attention is that over the slots.
    gen = torch.Generator().manual_seed(10)
    Hk, H, d, lens = 2, 8, 64, [500, 333]
    width = 9
    pages = torch.randperm(2 * width + 1, generator=gen)[:2 * width].reshape(2, width).int()
    kc = torch.zeros((2 * width + 1, Hk, 64, d), dtype=torch.float8_e4m3fn, device="cuda")
    cache = [kc, kc.clone(), torch.zeros((2 * width + 1, Hk), device="cuda")]
    cache.append(cache[2].clone())
    pd = dev(pages)
    kv = torch.randn((sum(lens), 2 * Hk, d), generator=gen).bfloat16()
    cu = plain.cum(lens)
    ld = dev(i32(lens))
    kvd = dev(kv)
    fa.fa_paged_kv_append(kvd[:, :Hk], kvd[:, Hk:], dev(cu), ld, pd, *cache)
    tokens = [kv[cu[b]:cu[b + 1]].double() for b in range(2)]  # every token of a sequence
    kept = [[list(range(n)) for _ in range(Hk)] for n in lens]

    def check_slots():
        for b in range(2):
            for h in range(Hk):
                for which in (0, 1):
                    got, scale = held(cache, pages, b, int(ld[b]), which, h)
                    assert_holds(got, scale, tokens[b][kept[b][h], which * Hk + h])
    check_slots()
    rows = 16
    q = torch.randn((2 * rows, H, d), generator=gen).bfloat16()
    cu_q = dev(i32([0, rows, 2 * rows]))
    _, lse = attend(dev(q), cache, cu_q, ld, pd)
    sums = torch.full((2, Hk, width * 64), torch.nan, device="cuda")
    fa.fa_paged_key_weights(dev(q), lse, cache[0], cache[2], cu_q, ld, pd, sums, decay=0.0)
    for budget in (200, 130):
        wk, wn = masked.select(sums.cpu(), ld.cpu().tolist(), budget, 4, 40)
        keep, new = fa.fa_paged_kv_select(sums, ld, budget, sink_tokens=4, recent_tokens=40)
        assert torch.equal(keep.cpu(), wk) and torch.equal(new.cpu(), wn)
        fa.fa_paged_kv_compact(*cache, pd, keep, new, weights=sums)
        ld.copy_(new)
        kept = [[[row[j] for j in wk[b, h].tolist() if j >= 0] for h, row in enumerate(kept[b])]
                for b in range(2)]
        check_slots()
        for step in range(3):
            one = torch.randn((2, H + 2 * Hk, d), generator=gen).bfloat16()
            od = dev(one)
            cu_1 = dev(i32([0, 1, 2]))
            ld += 1
            fa.fa_paged_kv_append(od[:, H:H + Hk], od[:, H + Hk:], cu_1, ld, pd, *cache)
            qs = od[:, :H].contiguous()
            o, lse = attend(qs, cache, cu_1, ld, pd)
            fa.fa_paged_key_weights(qs, lse, cache[0], cache[2], cu_1, ld, pd, sums)
            torch.cuda.synchronize()
            assert fa.fa_get_device_status() == fa.FA_OK
            for b in range(2):
                for h in range(Hk):
                    kept[b][h].append(len(tokens[b]))
                tokens[b] = torch.cat([tokens[b], one[b, H:][None].double()])
            check_slots()
            assert_attends(o, lse, qs, cache, cu_1.cpu(), ld.cpu(), pages)
            assert torch.isfinite(sums[0, :, :int(ld[0])]).all()


def test_drafted_tree_run(cuda_device):
    # Masks and positions, rotation, append, attention of the tree, and the
    # accepted path moved behind the context: the slots then hold the path's
    # tokens, and causal attention over them sees what the tree's rows saw.
    gen = torch.Generator().manual_seed(11)
    Hk, H, d, ctx, nodes = 2, 8, 128, [190, 64], [21, 40]
    lens = [c + n for c, n in zip(ctx, nodes)]
    trees = [masked.random_parents(n, 60 + n) for n in nodes]
    pages, num = plain.make_pages(lens, gen)
    made = [plain.make_cache(ctx, pages, num, Hk, d, gen, 0) for _ in range(2)]
    cache = [dev(made[0][0]), dev(made[1][0]), dev(made[0][1]), dev(made[1][1])]
    context = {(b, w, h): held(cache, pages, b, ctx[b], w, h)[0]
               for b in range(2) for w in range(2) for h in range(Hk)}
    tab = dev(plain.table(400, d))
    qkv = dev(torch.randn((sum(nodes), H + 2 * Hk, d), generator=gen).bfloat16())
    cu, ld, pd = dev(plain.cum(nodes), i32(lens), pages)
    parents = dev(i32([p for t in trees for p in t]))
    mask, pos = fa.fa_draft_tree(parents, cu, ld, max_nodes=40)
    q, k = fa.fa_qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hk], pos, tab)
    v = qkv[:, H + Hk:]
    fa.fa_paged_kv_append(k, v, cu, ld, pd, *cache)
    o, lse = attend(q, cache, cu, ld, pd, tree_mask=mask)
    torch.cuda.synchronize()
    assert_attends(o, lse, q, cache, cu.cpu(), ld.cpu(), pages, masked.tree_masks(trees, 2))
    # The deepest node's path is accepted.
    paths = [max((masked.path_of(t, i)[::-1] for i in range(n)), key=len)
             for t, n in zip(trees, nodes)]
    assert all(len(p) > 2 for p in paths)
    keep = torch.full((2, 1, max(map(len, paths))), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        keep[b, 0, :len(p)] = i32([ctx[b] + x for x in p])
    fa.fa_paged_kv_compact(*cache, pd, *dev(keep, i32([len(p) for p in paths])), first=dev(i32(ctx)))
    new = i32([c + len(p) for c, p in zip(ctx, paths)])
    at = torch.tensor([int(cu[b]) + x for b, p in enumerate(paths) for x in p])
    cu_p = plain.cum([len(p) for p in paths])
    po, pl = attend(q[at.cuda()], cache, *dev(cu_p, new), pd)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    assert_attends(po, pl, q[at.cuda()], cache, cu_p, new, pages)
    for b in range(2):
        for h in range(Hk):
            for w, x in ((0, k), (1, v)):
                got, scale = held(cache, pages, b, int(new[b]), w, h)
                mine = x.cpu()[at[cu_p[b]:cu_p[b + 1]], h].double()
                assert_holds(got, scale, torch.cat([context[b, w, h], mine]))


def test_eviction_in_a_graph(cuda_device):
    # Captured once, replayed on other sums and lengths in place.
    gen = torch.Generator().manual_seed(12)
    lens = [400, 300]
    pages, num, caches = make_both(lens, 2, 64, gen)
    cards = [dev(c, s) for c, s in caches]
    sums = torch.rand((2, 2, 448), generator=gen)
    sd, ld, pd = dev(sums, i32(lens), pages)

    def step():
        keep, new = fa.fa_paged_kv_select(sd, ld, 150, sink_tokens=4, recent_tokens=30)
        fa.fa_paged_kv_compact(cards[0][0], cards[1][0], cards[0][1], cards[1][1], pd, keep, new,
                               weights=sd)
        return keep, new
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        keep, new = step()
    for now in ([400, 300], [149, 151]):
        for (c, s), (cd, sc) in zip(caches, cards):
            cd.copy_(c)
            sc.copy_(s)
        sums = torch.rand((2, 2, 448), generator=gen)
        sd.copy_(sums)
        ld.copy_(i32(now))
        g.replay()
        torch.cuda.synchronize()
        wk, wn = masked.select(sums, now, 150, 4, 30)
        assert torch.equal(keep.cpu(), wk) and torch.equal(new.cpu(), wn)
        for (c, s), (cd, sc) in zip(caches, cards):
            want, ws = masked.compact(c.double(), s.double(), pages, wk, [0, 0], wn.tolist())
            assert torch.equal(sc.cpu().double(), ws)
            assert torch.equal(torch.nan_to_num(cd.cpu().double(), 777.0),
                               torch.nan_to_num(want, 777.0))
        assert torch.equal(sd.cpu(), masked.move_weights(sums, wk, [0, 0], wn.tolist(), pages, num))
