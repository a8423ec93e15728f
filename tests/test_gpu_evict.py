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
