"""GPU: the serving operators around the attention forward (q/k norm with
rotation, paged 8-bit cache) against their plain fp64 forms.

Tolerances count roundings.  u = 2^-24 is half a step of fp32, 2^-8 of bf16
(relative), and e4m3's half step is taken at each value.

  norm and rotation  one bf16 rounding of the result, and fp32 arithmetic
      before it: the sum of d squares, the root, two products and a sum, at
      most (d + 16) u of the larger of the pair.
  append  one e4m3 rounding, the same fp32 arithmetic before it; codes that
      are rounded again are compared bit for bit.
  attention  the score is a sum of d products in fp32 (q is held in two e4m3
      terms, exact to 2^-18 of its row's largest value): off by at most
      dx = 2^-15 A, A = scale * sum |q k|, and 2^-20 |x| more from the
      products with the scales; p is off by dx relatively, is rounded to at
      least 11 bits for the product with v, and O once to bf16:
      2^-8 |O| + (2 dx + 2^-10) sum p |v|.  LSE: dx + 2^-20 (1 + |LSE|).
"""
import math

import pytest
import torch

import paged_plain as plain
import varlen_flashattention_forward_gb300 as fa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def dev(*ts):
    got = [None if t is None else t.cuda() for t in ts]
    return got if len(got) > 1 else got[0]


# ------------------------------------------------------- norm and rotation
def norm_tolerance(y, d):
    """y: the exact result; the pair's other member is bounded by the row's
    largest value."""
    return 2.0 ** -8 * y.abs() + 2 * (d + 16) * U * y.abs().amax(-1, keepdim=True) + 1e-37


def check_norm_rope(T, H, Hk, d, rot, interleaved, norm, seed, max_pos=300, fused=True):
    gen = torch.Generator().manual_seed(seed)
    buf = torch.randn((T, H + 2 * Hk, d), generator=gen).bfloat16()
    q, k = buf[:, :H], buf[:, H:H + Hk]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    qw = torch.randn(d, generator=gen) if norm else None
    kw = torch.randn(d, generator=gen) if norm else None
    pos = torch.randint(0, max_pos, (T,), generator=gen, dtype=torch.int32)
    tab = plain.table(max_pos, rot) if rot else None
    bd = dev(buf)
    qd, kd = (bd[:, :H], bd[:, H:H + Hk]) if fused else (bd[:, :H].contiguous(),
                                                         bd[:, H:H + Hk].contiguous())
    qo, ko = fa.fa_qk_norm_rope(qd, kd, dev(pos), dev(tab), dev(qw), dev(kw), eps=1e-5,
                                interleaved=interleaved)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want = plain.rotate(plain.rms(x, w, 1e-5), pos.tolist(), tab, interleaved)
        assert got.is_contiguous()
        assert ((got.cpu().double() - want).abs() <= norm_tolerance(want, d)).all()


@pytest.mark.parametrize("d,rot", [(64, 64), (72, 64), (80, 80), (96, 48), (128, 128), (128, 0),
                                   (192, 64), (256, 256), (8, 0), (16, 16), (136, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_dims(cuda_device, d, rot, interleaved):
    check_norm_rope(37, 6, 2, d, rot, interleaved, True, seed=d + rot)


@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (1, 32, 8), (3, 5, 1), (257, 7, 7), (2000, 3, 1)])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_counts(cuda_device, T, H, Hk, norm):
    check_norm_rope(T, H, Hk, 128, 128, False, norm, seed=T, fused=T % 2 == 1)


def test_norm_rope_one_side_in_place_and_skipped_tokens(cuda_device):
    gen = torch.Generator().manual_seed(5)
    x = torch.randn((9, 4, 128), generator=gen).bfloat16()
    pos = torch.tensor([0, -1, 5, 99, 100, 2 ** 31 - 1, -2 ** 31, 7, 1], dtype=torch.int32)
    tab, w = plain.table(100, 128), torch.randn(128, generator=gen)
    want = plain.rotate(plain.rms(x, w, 1e-6), pos.tolist(), tab, False)
    skipped = torch.tensor([not 0 <= p < 100 for p in pos.tolist()])
    for side in (0, 1):
        buf = dev(x)
        got = fa.fa_qk_norm_rope(*((buf, None) if side == 0 else (None, buf)), dev(pos), dev(tab),
                                 **({"q_weight": dev(w), "q_out": buf} if side == 0
                                    else {"k_weight": dev(w), "k_out": buf}))
        assert got[1 - side] is None and got[side].data_ptr() == buf.data_ptr()
        out = buf.cpu()
        assert torch.equal(out[skipped], x[skipped])
        ok = (out.double() - want).abs() <= norm_tolerance(want, 128)
        assert ok[~skipped].all()


def test_norm_rope_in_place_in_a_fused_buffer(cuda_device):
    gen = torch.Generator().manual_seed(6)
    buf = torch.randn((33, 12, 64), generator=gen).bfloat16()
    pos = torch.arange(33, dtype=torch.int32)
    tab = plain.table(33, 64)
    b = dev(buf)
    fa.fa_qk_norm_rope(b[:, :8], b[:, 8:10], dev(pos), dev(tab), q_out=b[:, :8], k_out=b[:, 8:10])
    want = plain.rotate(buf[:, :10].double(), pos.tolist(), tab, False)
    assert ((b[:, :10].cpu().double() - want).abs() <= norm_tolerance(want, 64)).all()
    assert torch.equal(b[:, 10:].cpu(), buf[:, 10:])


def test_norm_rope_no_tokens(cuda_device):
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    qo, ko = fa.fa_qk_norm_rope(q, None, None, None)
    assert qo.shape == (0, 4, 128) and ko is None


# ------------------------------------------------------------------ append
def check_append(new, ctx, Hk, d, rot, norm, seed, interleaved=False, size=1.0, calls=None,
                 bad_page=False, limit=None):
    """Appends `new` tokens of each sequence behind `ctx` cached ones (in
    `calls` portions) and compares codes and scales after each call."""
    gen = torch.Generator().manual_seed(seed)
    final = [a + b for a, b in zip(new, ctx)]
    pages, num = plain.make_pages(final, gen)
    if bad_page:
        pages[0, 0], pages[-1, -1] = num, -2 ** 31
    caches = []
    for _ in range(2):
        codes, scale = plain.make_cache(ctx, pages.clamp(0, num - 1), num, Hk, d, gen)
        caches.append((codes, scale, dev(codes), dev(scale)))
    w = torch.randn(d, generator=gen) if norm else None
    tab = plain.table(limit or pages.shape[1] * 64, rot) if rot else None
    top = min(pages.shape[1] * 64, limit or 1 << 30)
    lens = list(ctx)
    for portion in (calls or [1.0]):
        part = [max(0, min(f - n, math.ceil(a * portion))) for f, n, a in zip(final, lens, new)]
        lens = [n + p for n, p in zip(lens, part)]
        cu = plain.cum(part)
        kv = (torch.randn((int(cu[-1]), 2 * Hk, d), generator=gen) * size).bfloat16()
        k, v = kv[:, :Hk], kv[:, Hk:]
        kvd = dev(kv)
        before = [(c[2].cpu().view(torch.uint8), c[3].cpu()) for c in caches]
        fa.fa_paged_kv_append(kvd[:, :Hk], kvd[:, Hk:], dev(cu),
                              dev(torch.tensor(lens, dtype=torch.int32)), dev(pages),
                              caches[0][2], caches[1][2], caches[0][3], caches[1][3],
                              cos_sin=dev(tab), k_weight=dev(w), eps=1e-6,
                              interleaved=interleaved)
        cul = cu.tolist()
        where = []
        for b in range(len(part)):
            where += [lens[b] - part[b] + i for i in range(part[b])]
        y = plain.rotate(plain.rms(k, w, 1e-6), where, tab, interleaved)
        for (old_codes, old_scale), cache, x, exact in ((before[0], caches[0], y, not (rot or norm)),
                                                        (before[1], caches[1], v.double(), True)):
            codes = old_codes.view(torch.float8_e4m3fn).double()
            scale = old_scale.double()
            touched, want = plain.append(x, cul, lens, pages, codes, scale, top)
            got = cache[2].cpu()
            assert torch.equal(cache[3].cpu().double()[~torch.isnan(scale)],
                               scale[~torch.isnan(scale)])
            same = got.view(torch.uint8) == old_codes
            assert same[~touched].all(), "a slot outside the new tokens changed"
            values = got.double()
            if exact:
                assert torch.equal(torch.nan_to_num(values[touched], 777.0),
                                   torch.nan_to_num(codes[touched], 777.0))
            else:
                # want is the exact quotient; rows within the fp32 error of a
                # border may round to either side.
                slack = (d + 16) * U * 2 * E4M3(want[touched])
                off = (values[touched] - want[touched].clamp(-448, 448)).abs()
                assert (off <= plain.e4m3_half_step(want[touched]) + slack).all()


def E4M3(x):
    """Bound of the pair's other member, in units of the scale."""
    return torch.full_like(x, 448.0)


@pytest.mark.parametrize("d,Hk", [(64, 1), (80, 3), (96, 2), (128, 8)])
@pytest.mark.parametrize("rot,norm", [(0, False), (48, True), (64, False)])
def test_append_dims(cuda_device, d, Hk, rot, norm):
    check_append([5, 1, 130, 64], [0, 63, 30, 64], Hk, d, rot, norm, seed=d + rot)


@pytest.mark.parametrize("new,ctx", [
    ([1], [0]), ([1], [64]), ([1], [63]), ([64], [0]), ([65], [0]), ([63], [1]), ([2], [63]),
    ([1] * 300, [7 * i % 200 for i in range(300)]),          # more sequences than threads
    ([0, 1, 0, 0, 3], [5, 0, 0, 64, 127]),                   # sequences without tokens
    ([700, 1, 1, 1], [0, 100, 200, 300]),                    # a prompt among single tokens
    ([40] * 20, [13 * i % 64 for i in range(20)]),
])
def test_append_lengths(cuda_device, new, ctx):
    check_append(new, ctx, 2, 64, 64, True, seed=len(new) + sum(new), interleaved=True)


def test_append_token_by_token_raises_the_scale(cuda_device):
    # Values grow from call to call, so that earlier codes are rounded again.
    gen = torch.Generator().manual_seed(3)
    Hk, d = 2, 64
    pages = torch.tensor([[1, 0]], dtype=torch.int32)
    kc = torch.zeros((2, Hk, 64, d), dtype=torch.float8_e4m3fn, device="cuda")
    vc, ks, vs = kc.clone(), torch.zeros((2, Hk), device="cuda"), torch.zeros((2, Hk),
                                                                             device="cuda")
    rows = torch.randn((80, 2 * Hk, d), generator=gen) * torch.exp2(torch.arange(80) / 4.0 - 10)[
        torch.randperm(80, generator=gen)][:, None, None]
    rows = rows.bfloat16()
    want_k = torch.zeros((2, Hk, 64, d), dtype=torch.float64)
    want_s = torch.zeros((2, Hk), dtype=torch.float64)
    for t in range(80):
        kv = dev(rows[t:t + 1])
        fa.fa_paged_kv_append(kv[:, :Hk], kv[:, Hk:], dev(plain.cum([1])),
                              dev(torch.tensor([t + 1], dtype=torch.int32)), dev(pages), kc, vc,
                              ks, vs)
        plain.append(rows[t:t + 1, :Hk].double(), [0, 1], [t + 1], pages, want_k, want_s, 128)
        assert torch.equal(ks.cpu().double(), want_s)
        assert torch.equal(kc.cpu().double(), want_k)
    # Written at once, the scales are the same and no value is further off
    # than one more rounding.
    k2, v2, s2, t2 = torch.zeros_like(kc), vc.clone(), torch.zeros_like(ks), torch.zeros_like(vs)
    kv = dev(rows)
    fa.fa_paged_kv_append(kv[:, :Hk], kv[:, Hk:], dev(plain.cum([80])),
                          dev(torch.tensor([80], dtype=torch.int32)), dev(pages), k2, v2, s2, t2)
    assert torch.equal(s2, ks)
    # Codes differ only below the smallest normal value, 2^-6.
    a, b = k2.cpu().double(), kc.cpu().double()
    assert ((a - b).abs() <= torch.where(a.abs() < 2.0 ** -6, 2.0 ** -9, 0.0)).all()


def test_append_in_portions(cuda_device):
    check_append([300, 64, 1, 129], [10, 0, 63, 64], 2, 80, 80, True, seed=11,
                 calls=[0.1, 0.3, 0.02, 1.0])


def test_append_bad_pages_and_lengths(cuda_device):
    check_append([70, 5, 100], [10, 3, 60], 2, 64, 0, False, seed=12, bad_page=True)
    # The rotation table ends before the sequence does.
    check_append([70, 5, 100], [10, 3, 60], 2, 64, 64, True, seed=13, limit=100)


def test_append_malformed_arrays_write_nothing_outside(cuda_device):
    gen = torch.Generator().manual_seed(14)
    kv = dev(torch.randn((20, 4, 64), generator=gen).bfloat16())
    big = 2 ** 31 - 1
    for cu, lens, pages in [
            ([0, 30, 10, 20], [64, 64, 64], [[0], [0], [0]]),      # past the rows, decreasing
            ([-5, 7, 7, 20], [3, 0, big], [[0], [1], [2]]),        # length below, zero, huge
            ([0, 20, 20, 20], [-1, -2 ** 31, 5], [[big], [-1], [3]])]:
        arr = torch.zeros((6, 2, 64, 64), dtype=torch.uint8, device="cuda").fill_(0x38)
        guard = torch.full((6, 2), 1.0, device="cuda")
        kc, vc = arr.view(torch.float8_e4m3fn), arr.clone().view(torch.float8_e4m3fn)
        # Pages 0 and 5 of the storage are guards around a cache of 4.
        fa.fa_paged_kv_append(kv[:, :2], kv[:, 2:], dev(torch.tensor(cu, dtype=torch.int32)),
                              dev(torch.tensor(lens, dtype=torch.int32)),
                              dev(torch.tensor(pages, dtype=torch.int32)), kc[1:5], vc[1:5],
                              guard[1:5], guard.clone()[1:5])
        torch.cuda.synchronize()
        assert (arr[0] == 0x38).all() and (arr[5] == 0x38).all()
        assert (guard[0] == 1).all() and (guard[5] == 1).all()


def test_append_special_values(cuda_device):
    # An infinity and a NaN cost their own places only; zeros get the smallest
    # scale; a value on the border 448 s does not raise the scale.
    inf, nan = math.inf, math.nan
    rows = torch.zeros((64, 2, 64))
    rows[:, 0] = torch.linspace(-1, 1, 64)[:, None]
    rows[3, 0, 5], rows[4, 0, 6], rows[5, 0, 7] = inf, -inf, nan
    rows[:, 1, 0] = 448.0 * 2.0 ** -9
    x = rows.bfloat16()
    kc = torch.zeros((1, 2, 64, 64), dtype=torch.float8_e4m3fn, device="cuda")
    vc, ks, vs = kc.clone(), torch.zeros((1, 2), device="cuda"), torch.ones((1, 2), device="cuda")
    zero = dev(torch.zeros((64, 2, 64)).bfloat16())
    fa.fa_paged_kv_append(dev(x), zero, dev(plain.cum([64])),
                          dev(torch.tensor([64], dtype=torch.int32)),
                          dev(torch.zeros((1, 1), dtype=torch.int32)), kc, vc, ks, vs)
    assert ks[0, 0].item() == 2.0 ** -8 and ks[0, 1].item() == 2.0 ** -9   # 1 / 448 -> 2^-8
    assert (vs == 2.0 ** -64).all() and (vc.float() == 0).all()
    k = kc.cpu().float()[0, 0]
    assert k[3, 5] == 448 and k[4, 6] == -448 and torch.isnan(k[5, 7])
    want = plain.e4m3(x[:, 0].double() * 2.0 ** 8)
    mask = torch.ones((64, 64), dtype=torch.bool)
    mask[3, 5] = mask[4, 6] = mask[5, 7] = False
    assert torch.equal(k.double()[mask], want[mask])


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("d,Hk,lens", [(64, 1, [1]), (80, 3, [0, 64, 65, 0, 1]),
                                       (96, 2, [200, 63, 129]), (128, 8, [1000, 3]),
                                       (64, 2, [i % 70 for i in range(400)])])
def test_gather_is_exact(cuda_device, d, Hk, lens):
    gen = torch.Generator().manual_seed(sum(lens))
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, Hk, d, gen) for _ in range(2))
    total = sum(lens)
    guard = [torch.full((total + 2, Hk, d), 9.0, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    k, v = fa.fa_paged_kv_gather(*dev(kc, vc, ks, vs, plain.cum(lens), pages), total,
                                 k_out=guard[0][1:-1], v_out=guard[1][1:-1])
    for got, codes, scale in ((k, kc, ks), (v, vc, vs)):
        at = 0
        for b, n in enumerate(lens):
            for h in range(Hk):
                want, _ = plain.keys_of(b, n, pages, codes, scale, h)
                assert torch.equal(got[at:at + n, h].cpu().double(), want)
            at += n
    assert all((g[0] == 9).all() and (g[-1] == 9).all() for g in guard)


def test_gather_missing_pages_read_as_zero(cuda_device):
    gen = torch.Generator().manual_seed(1)
    lens = [130, 64, 10]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    pages[0, 1], pages[2, 0] = num, -1
    more = [200, 64, 10]            # and sequence 0 is longer than its table
    k, v = fa.fa_paged_kv_gather(*dev(kc, vc, ks, vs, plain.cum(more), pages), sum(more))
    k = k.cpu().double()
    for h in range(2):
        want, held = plain.keys_of(0, 130, pages, kc, ks, h)
        assert (~held).sum() == 64
        assert torch.equal(k[:130, h], want)
    assert (k[192:200] == 0).all() and (k[264:] == 0).all()


def test_gather_any_scale(cuda_device):
    gen = torch.Generator().manual_seed(2)
    pages, num = plain.make_pages([100], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([100], pages, num, 2, 64, gen) for _ in range(2))
    ks, vs = ks * 1.3, vs * 0.7
    k, _ = fa.fa_paged_kv_gather(*dev(kc, vc, ks, vs, plain.cum([100]), pages), 100)
    for h in range(2):
        want, _ = plain.keys_of(0, 100, pages, kc, ks, h)
        assert ((k[:, h].cpu().double() - want).abs() <= (2.0 ** -8 + 2 * U) * want.abs()).all()


# --------------------------------------------------------------- attention
def check_attn(q_lens, lens, H, Hk, d, causal=True, window=-1, seed=0, size=1.0, pages=None,
               lens_given=None, spread=3, scale=None, strided=False, hints=True, stream=None,
               break_pages=None):
    gen = torch.Generator().manual_seed(seed)
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, Hk, d, gen, spread) for _ in range(2))
    if break_pages:
        break_pages(pages, num)
    cu = plain.cum(q_lens)
    T = int(cu[-1])
    q = (torch.randn((T, H + (3 if strided else 0), d), generator=gen) * size).bfloat16()
    scale = scale or d ** -0.5
    given = lens_given or lens
    out = torch.full((T + 2, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    qd = dev(q)[:, :H]
    o, lse = fa.fa_paged_attn(qd, *dev(kc, vc, ks, vs, cu, torch.tensor(given, dtype=torch.int32),
                                       pages),
                              max_seqlen_q=max(q_lens) if hints else 0,
                              max_seqlen_k=max(lens) if hints else 0, softmax_scale=scale,
                              causal=causal, window_left=window, out=out[1:-1], return_lse=True,
                              stream=stream)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    assert (out[0] == 7).all() and (out[-1] == 7).all()
    wo, wl, w, a = plain.attention(q[:, :H], kc, vc, ks, vs, cu.tolist(), given, pages, scale,
                                   causal, window)
    compare_attn(o.cpu(), lse.cpu(), wo, wl, w, a)
    return o, lse


def compare_attn(o, lse, wo, wl, w, a):
    assert torch.equal(torch.isinf(lse), torch.isinf(wl))
    fin = torch.isfinite(wl)
    dx = 2.0 ** -15 * a + 2.0 ** -20 * a
    off = (lse.double() - wl).abs()[fin]
    assert (off <= dx[fin] + 2.0 ** -20 * (1 + wl[fin].abs())).all(), off.max()
    tol = 2.0 ** -8 * wo.abs() + (2 * dx.t()[..., None] + 2.0 ** -10) * w + 1e-30
    off = (o.double() - wo).abs()
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.parametrize("d", [64, 80, 96, 128])
@pytest.mark.parametrize("H,Hk", [(8, 1), (8, 8), (6, 2), (32, 2), (20, 1)])
def test_attn_single_tokens(cuda_device, d, H, Hk):
    check_attn([1] * 6, [1, 64, 65, 127, 200, 513], H, Hk, d, seed=d + H)


@pytest.mark.parametrize("q_lens,lens", [
    ([2, 5, 1], [2, 130, 64]),
    ([8, 8], [300, 8]),
    ([17], [100]),
    ([0, 3, 0, 1], [50, 3, 0, 129]),       # sequences without query rows
    ([1, 1, 1], [0, 10, 0]),               # sequences without keys
    ([70], [200]),                         # a chunk: several row tiles
])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_many_tokens(cuda_device, q_lens, lens, causal):
    check_attn(q_lens, lens, 8, 2, 64, causal=causal, seed=sum(lens))


def test_attn_more_rows_than_keys(cuda_device):
    # Causal rows that stand before the first key see nothing.
    check_attn([5, 9], [2, 8], 4, 2, 64, seed=21)


@pytest.mark.parametrize("window", [0, 1, 63, 64, 100, 1000])
def test_attn_window(cuda_device, window):
    check_attn([1, 3, 8], [700, 129, 64], 4, 2, 128, window=window, seed=window)
    check_attn([1, 3], [300, 129], 4, 2, 64, causal=False, window=window, seed=window + 1)


def test_attn_long_contexts(cuda_device):
    check_attn([1, 1], [9000, 5001], 8, 2, 128, seed=31)
    check_attn([4], [20000], 4, 1, 64, seed=32)


def test_attn_many_sequences(cuda_device):
    lens = [1 + 37 * i % 260 for i in range(600)]
    check_attn([1] * 600, lens, 4, 1, 64, seed=33)


@pytest.mark.parametrize("size", [0.0, 1e-3, 30.0])
def test_attn_score_ranges(cuda_device, size):
    # Rows of zeros, almost uniform weights, and one key taking all of it.
    check_attn([1, 2], [400, 150], 8, 2, 128, size=size, seed=41)


def test_attn_scales_far_apart(cuda_device):
    check_attn([1, 1], [900, 300], 4, 2, 64, spread=12, seed=42)


def test_attn_strided_q_no_hints_other_stream(cuda_device):
    check_attn([1, 2, 1], [64, 100, 300], 8, 4, 96, strided=True, hints=False, seed=43)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check_attn([1, 2, 1], [64, 100, 300], 8, 4, 96, seed=44, stream=s)


def test_attn_missing_pages_are_skipped(cuda_device):
    def break_some(pages, num):
        pages[0, 0], pages[0, 2], pages[1, 0], pages[2, 1] = num, -1, 2 ** 31 - 1, -2 ** 31
    check_attn([1, 1, 3], [300, 64, 130], 8, 2, 128, seed=45, break_pages=break_some)


def test_attn_lengths_past_the_table(cuda_device):
    check_attn([1, 2], [130, 64], 4, 2, 64, lens_given=[130, 1000], seed=46)
    check_attn([1, 2], [130, 64], 4, 2, 64, lens_given=[-5, 64], seed=47)


def test_attn_malformed_cu_seqlens(cuda_device):
    gen = torch.Generator().manual_seed(48)
    lens = [100, 100, 100]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    q = dev(torch.randn((6, 4, 64), generator=gen).bfloat16())
    for cu in ([0, 50, 3, 6], [-9, 2, 4, 2 ** 31 - 1], [5, 4, 3, 2]):
        out = torch.full((8, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        fa.fa_paged_attn(q, *dev(kc, vc, ks, vs, torch.tensor(cu, dtype=torch.int32),
                                 torch.tensor(lens, dtype=torch.int32), pages), out=out[1:-1])
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        assert (out[0] == 7).all() and (out[-1] == 7).all()


def test_attn_rows_behind_the_last_sequence_stay(cuda_device):
    gen = torch.Generator().manual_seed(49)
    pages, num = plain.make_pages([100], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([100], pages, num, 2, 64, gen) for _ in range(2))
    q = dev(torch.randn((5, 4, 64), generator=gen).bfloat16())
    out = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 5), 7.0, device="cuda")
    fa.fa_paged_attn(q, *dev(kc, vc, ks, vs, torch.tensor([0, 2], dtype=torch.int32),
                             torch.tensor([100], dtype=torch.int32), pages), out=out, lse=lse)
    assert (out[2:] == 7).all() and (lse[:, 2:] == 7).all() and not (out[:2] == 7).any()


def test_attn_no_rows(cuda_device):
    gen = torch.Generator().manual_seed(50)
    pages, num = plain.make_pages([100], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([100], pages, num, 2, 64, gen) for _ in range(2))
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    o = fa.fa_paged_attn(q, *dev(kc, vc, ks, vs, torch.tensor([0, 0], dtype=torch.int32),
                                 torch.tensor([100], dtype=torch.int32), pages))
    assert o.shape == (0, 4, 64)


def test_attn_runs_are_bitwise_the_same(cuda_device):
    a = check_attn([1, 3, 1], [2000, 700, 64], 8, 2, 128, seed=51)
    b = check_attn([1, 3, 1], [2000, 700, 64], 8, 2, 128, seed=51)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attn_nan_and_infinite_values_reach_their_rows(cuda_device):
    # A NaN code of a visible key makes its dim NaN; of a key or page nobody
    # sees (make_cache fills those with NaN) it does nothing.
    gen = torch.Generator().manual_seed(52)
    pages, num = plain.make_pages([100, 50], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([100, 50], pages, num, 1, 64, gen) for _ in range(2))
    page = int(pages[0, 1])
    vc.view(torch.uint8)[page, 0, 3, 17] = plain.NAN_CODE
    q = torch.randn((2, 2, 64), generator=gen).bfloat16()
    o = fa.fa_paged_attn(*dev(q, kc, vc, ks, vs, plain.cum([1, 1]),
                              torch.tensor([100, 50], dtype=torch.int32), pages)).cpu()
    assert torch.isnan(o[0, :, 17]).all()
    keep = torch.arange(64) != 17
    assert torch.isfinite(o[0][:, keep]).all() and torch.isfinite(o[1]).all()


# ------------------------------------------------------------ used together
def test_serving_run(cuda_device):
    """A prompt in two parts, then decode steps: norm and rotation, append,
    attention; each step against plain attention over the values the cache
    stands for, with the chunk's attention also through the gather and
    fa_varlen_fwd, and through a merge of context and own keys."""
    gen = torch.Generator().manual_seed(60)
    H, Hk, d, B = 8, 2, 128, 3
    final = [150, 40, 300]
    pages, num = plain.make_pages([n + 8 for n in final], gen)
    tab = dev(plain.table(512, d))
    qw, kw = torch.rand(d, generator=gen) + 0.5, torch.rand(d, generator=gen) + 0.5
    kc = torch.zeros((num, Hk, 64, d), dtype=torch.float8_e4m3fn, device="cuda")
    vc, ks, vs = kc.clone(), torch.zeros((num, Hk), device="cuda"), torch.zeros((num, Hk),
                                                                               device="cuda")
    scale, have = d ** -0.5, [0] * B
    steps = [[n // 3 for n in final], [n - n // 3 for n in final], [1] * B, [1, 0, 1], [4, 2, 3]]
    for step, part in enumerate(steps):
        have = [a + b for a, b in zip(have, part)]
        cu = plain.cum(part)
        T = int(cu[-1])
        qkv = dev(torch.randn((T, H + 2 * Hk, d), generator=gen).bfloat16())
        pos = torch.cat([torch.arange(n - p, n) for n, p in zip(have, part)]).int()
        lens = torch.tensor(have, dtype=torch.int32)
        q, k = fa.fa_qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hk], dev(pos), tab, dev(qw), dev(kw))
        fa.fa_paged_kv_append(qkv[:, H:H + Hk], qkv[:, H + Hk:], *dev(cu, lens, pages), kc, vc, ks,
                              vs, cos_sin=tab, k_weight=dev(kw))
        o, lse = fa.fa_paged_attn(q, kc, vc, ks, vs, *dev(cu, lens, pages),
                                  max_seqlen_q=max(part), return_lse=True)
        kcc, vcc, ksc, vsc = kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu()
        want = plain.attention(q.cpu(), kcc, vcc, ksc, vsc, cu.tolist(), have, pages, scale, True,
                               -1)
        compare_attn(o.cpu(), lse.cpu(), *want)
        # What the cache stands for is the normed and rotated key within its
        # rounding (half an e4m3 step of the page's scale).
        cuk = plain.cum(have)
        gk, gv = fa.fa_paged_kv_gather(kc, vc, ks, vs, *dev(cuk, pages), int(cuk[-1]))
        for b in range(B):
            if part[b]:
                mine = gk[int(cuk[b + 1]) - part[b]:int(cuk[b + 1])].cpu().double()
                true = k[int(cu[b]):int(cu[b + 1])].cpu().double()
                top = ksc[pages[b, :-(-have[b] // 64)].long()].double().amax(0)[:, None]
                assert ((mine - true).abs() <= (2.0 ** -4 + 2.0 ** -7) * true.abs()
                        + 2.0 ** -9 * top).all()
        ov, lv = fa.fa_varlen_fwd(q, gk, gv, dev(cu), dev(cuk), max(part), max(have), scale, True,
                                  return_lse=True)
        # fa_varlen_fwd rounds p to bf16: 2^-8 of sum p |v| more.
        wo, wl, w, a = want
        dx = 2.0 ** -14 * a.t()[..., None]
        assert ((ov.cpu().double() - wo).abs()
                <= 2.0 ** -8 * wo.abs() + (2 * dx + 2.0 ** -7) * w + 1e-30).all()
        assert ((lv.cpu().double() - wl).abs() <= 2.0 ** -14 * a + 2.0 ** -18 * (1 + wl.abs())).all()
        # Context from the cache, own keys unquantised, merged.
        if step == 1:
            ctx = torch.tensor([n - p for n, p in zip(have, part)], dtype=torch.int32)
            oc, lc = fa.fa_paged_attn(q, kc, vc, ks, vs, *dev(cu, ctx, pages), causal=False,
                                      return_lse=True)
            v = qkv[:, H + Hk:]
            on, ln = fa.fa_varlen_fwd(q, k, v, dev(cu), dev(cu), max(part), max(part), scale, True,
                                      return_lse=True)
            om, lm = fa.fa_merge_attn_states(oc, lc, on, ln)
            # The own keys differ from the cached ones by their e4m3 rounding:
            # compare with plain attention over exactly these keys.
            for b in range(B):
                g = H // Hk
                for h in (0, H - 1):
                    kctx, _ = plain.keys_of(b, int(ctx[b]), pages, kcc, ksc, h // g)
                    vctx, _ = plain.keys_of(b, int(ctx[b]), pages, vcc, vsc, h // g)
                    rows = slice(int(cu[b]), int(cu[b + 1]))
                    ka = torch.cat([kctx, k[rows, h // g].cpu().double()])
                    va = torch.cat([vctx, v[rows, h // g].cpu().double()])
                    x = q[rows, h].cpu().double() @ ka.t() * scale
                    i = torch.arange(part[b])[:, None]
                    x = x.masked_fill(torch.arange(have[b])[None] > int(ctx[b]) + i, -math.inf)
                    p = torch.softmax(x, 1)
                    off = (om[rows, h].cpu().double() - p @ va).abs()
                    # Two parts rounded to bf16 and their mix once more.
                    assert (off <= 2.0 ** -6 * (p @ va.abs()) + 1e-30).all()
    assert fa.fa_get_device_status() == fa.FA_OK


def test_decode_step_in_a_graph(cuda_device):
    """Append and attention captured once and replayed on new tokens."""
    gen = torch.Generator().manual_seed(61)
    H, Hk, d, lens0 = 8, 2, 64, [63, 200, 5]
    pages, num = plain.make_pages([n + 8 for n in lens0], gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens0, pages, num, Hk, d, gen) for _ in range(2))
    kcd, vcd, ksd, vsd, pd = dev(kc, vc, ks, vs, pages)
    cu = dev(plain.cum([1] * 3))
    lens = torch.tensor([n + 1 for n in lens0], dtype=torch.int32).cuda()
    qkv = torch.zeros((3, H + 2 * Hk, d), dtype=torch.bfloat16, device="cuda")
    tab = dev(plain.table(512, d))
    pos = (lens - 1).contiguous()

    def step():
        q, _ = fa.fa_qk_norm_rope(qkv[:, :H], None, pos, tab)
        fa.fa_paged_kv_append(qkv[:, H:H + Hk], qkv[:, H + Hk:], cu, lens, pd, kcd, vcd, ksd, vsd,
                              cos_sin=tab)
        return q, *fa.fa_paged_attn(q, kcd, vcd, ksd, vsd, cu, lens, pd, max_seqlen_q=1,
                                    return_lse=True)

    first = torch.randn((3, H + 2 * Hk, d), generator=gen).bfloat16()
    qkv.copy_(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        q, o, lse = step()
    for n in range(1, 5):
        qkv.copy_(torch.randn((3, H + 2 * Hk, d), generator=gen).bfloat16())
        lens.copy_(torch.tensor([x + n for x in lens0], dtype=torch.int32))
        pos.copy_(lens - 1)
        graph.replay()
        torch.cuda.synchronize()
        want = plain.attention(q.cpu(), kcd.cpu(), vcd.cpu(), ksd.cpu(), vsd.cpu(), [0, 1, 2, 3],
                               lens.tolist(), pages, d ** -0.5, True, -1)
        compare_attn(o.cpu(), lse.cpu(), *want)
    assert fa.fa_get_device_status() == fa.FA_OK


def test_two_streams_at_once(cuda_device):
    """Calls on two streams without a wait between them, each with the
    workspace it allocates."""
    gen = torch.Generator().manual_seed(62)
    cases = []
    for i in range(2):
        lens = [3000 + 100 * i, 500]
        pages, num = plain.make_pages(lens, gen)
        (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
        q = torch.randn((2, 8, 64), generator=gen).bfloat16()
        cpu = (q, kc, vc, ks, vs, plain.cum([1, 1]), torch.tensor(lens, dtype=torch.int32), pages)
        cases.append((cpu, dev(*cpu), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (_, g, s) in enumerate(cases):
            got[i].append(fa.fa_paged_attn(*g, return_lse=True, stream=s))
    torch.cuda.synchronize()
    for i, (c, _, _) in enumerate(cases):
        q, kc, vc, ks, vs, cu, lens, pages = c
        want = plain.attention(q, kc, vc, ks, vs, cu.tolist(), lens.tolist(), pages, 64 ** -0.5,
                               True, -1)
        for o, lse in got[i]:
            compare_attn(o.cpu(), lse.cpu(), *want)


# ------------------------------------------------- shapes of tiles and calls
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("tokens,rows", [(1, 16), (7, 32), (13, 32)])
def test_attn_row_tiles(cuda_device, d, tokens, rows):
    assert fa.fa_paged_attn_plan(2, 2 * tokens, 8, 2, d, tokens)[1] == rows
    check_attn([tokens, max(1, tokens - 2)], [700, 260], 8, 2, d, seed=d + tokens)
    check_attn([tokens, 1], [300, 70], 8, 2, d, window=100, seed=d + tokens + 1)


@pytest.mark.parametrize("hint", [1, 3, 1000])
def test_attn_wrong_hints_do_not_matter(cuda_device, hint):
    gen = torch.Generator().manual_seed(53)
    lens, q_lens = [200, 65], [5, 2]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    q = torch.randn((7, 8, 64), generator=gen).bfloat16()
    cpu = (q, kc, vc, ks, vs, plain.cum(q_lens), torch.tensor(lens, dtype=torch.int32), pages)
    o, lse = fa.fa_paged_attn(*dev(*cpu), max_seqlen_q=hint, max_seqlen_k=hint, return_lse=True)
    want = plain.attention(q, kc, vc, ks, vs, [0, 5, 7], lens, pages, 0.125, True, -1)
    compare_attn(o.cpu(), lse.cpu(), *want)


def test_attn_batches_of_several_launches(cuda_device):
    # 1024 sequences to a launch.
    lens = [1 + 29 * i % 130 for i in range(1300)]
    check_attn([1] * 1300, lens, 2, 1, 64, seed=54)
    lens = [9 + 29 * i % 130 for i in range(700)]
    check_attn([1 + i % 9 for i in range(700)], lens, 8, 1, 64, seed=55)


def test_attn_given_workspace(cuda_device):
    gen = torch.Generator().manual_seed(56)
    lens = [3000, 129]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    q = torch.randn((2, 8, 64), generator=gen).bfloat16()
    args = dev(q, kc, vc, ks, vs, plain.cum([1, 1]), torch.tensor(lens, dtype=torch.int32), pages)
    need = fa.fa_paged_attn_plan(2, 2, 8, 2, 64, 1)[2]
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")  # NaN as fp32
    want = plain.attention(q, kc, vc, ks, vs, [0, 1, 2], lens, pages, 0.125, True, -1)
    for _ in range(2):
        o, lse = fa.fa_paged_attn(*args, max_seqlen_q=1, return_lse=True, workspace=ws[:need])
        compare_attn(o.cpu(), lse.cpu(), *want)
    assert (ws[need:] == 255).all()
    for bad in (ws[:need - 16], ws[8:need + 8]):
        with pytest.raises(fa.FaError) as e:
            fa.fa_paged_attn(*args, max_seqlen_q=1, workspace=bad)
        assert e.value.status == fa.FA_ERR_INVALID_ARG


def test_attn_special_queries_and_scales(cuda_device):
    # A NaN or an infinity in a row of q makes that row NaN and no other; a
    # page whose V scale is 0 adds zeros, not NaN.
    gen = torch.Generator().manual_seed(57)
    lens = [200]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 1, 64, gen) for _ in range(2))
    vs[pages[0, 1]] = 0.0
    q = torch.randn((2, 4, 64), generator=gen).bfloat16()
    q[0, 1, 3], q[1, 2, 60], q[1, 0] = math.nan, math.inf, 0.0
    cpu = (q, kc, vc, ks, vs, plain.cum([2]), torch.tensor(lens, dtype=torch.int32), pages)
    o, lse = (t.cpu() for t in fa.fa_paged_attn(*dev(*cpu), return_lse=True))
    bad = torch.zeros((2, 4), dtype=torch.bool)
    bad[0, 1] = bad[1, 2] = True
    assert torch.isnan(o[bad]).all() and torch.isnan(lse.t()[bad]).all()
    q[bad] = 0.0
    wo, wl, w, a = plain.attention(q, kc, vc, ks, vs, [0, 2], lens, pages, 0.125, True, -1)
    o[bad], wo[bad], lse.t()[bad], wl.t()[bad] = 0.0, 0.0, 0.0, 0.0
    compare_attn(o, lse, wo, wl, w, a)


def test_attn_nan_keys_behind_a_row_do_not_reach_it(cuda_device):
    gen = torch.Generator().manual_seed(58)
    lens = [130]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 1, 64, gen) for _ in range(2))
    kc.view(torch.uint8)[pages[0, 2], 0, 1] = plain.NAN_CODE  # the key of the last row
    q = torch.randn((3, 4, 64), generator=gen).bfloat16()
    cpu = (q, kc, vc, ks, vs, plain.cum([3]), torch.tensor(lens, dtype=torch.int32), pages)
    o, lse = (t.cpu() for t in fa.fa_paged_attn(*dev(*cpu), return_lse=True))
    assert torch.isnan(o[2]).all() and torch.isnan(lse[:, 2]).all()
    # The first two rows, against a cache without that key.
    wo, wl, w, a = plain.attention(q[:2], kc, vc, ks, vs, [0, 2], [129], pages, 0.125, True, -1)
    compare_attn(o[:2], lse[:, :2], wo, wl, w, a)


def test_attn_shared_pages(cuda_device):
    # Sequences with a common prefix name the same pages.
    gen = torch.Generator().manual_seed(59)
    lens = [300, 300, 192]
    pages, num = plain.make_pages(lens, gen)
    pages[1, :3] = pages[0, :3]
    pages[2, :3] = pages[0, :3]
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 128, gen) for _ in range(2))
    q = torch.randn((3, 8, 128), generator=gen).bfloat16()
    cpu = (q, kc, vc, ks, vs, plain.cum([1, 1, 1]), torch.tensor(lens, dtype=torch.int32), pages)
    o, lse = fa.fa_paged_attn(*dev(*cpu), return_lse=True)
    want = plain.attention(q, kc, vc, ks, vs, [0, 1, 2, 3], lens, pages, 128 ** -0.5, True, -1)
    compare_attn(o.cpu(), lse.cpu(), *want)


def test_two_graphs_replayed_at_once(cuda_device):
    """Each captured call has the workspace of its own capture."""
    gen = torch.Generator().manual_seed(63)
    graphs = []
    for i in range(2):
        lens = [4000 - 700 * i, 300]
        pages, num = plain.make_pages(lens, gen)
        (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
        q = torch.randn((2, 8, 64), generator=gen).bfloat16()
        cpu = (q, kc, vc, ks, vs, plain.cum([1, 1]), torch.tensor(lens, dtype=torch.int32), pages)
        args, s, g = dev(*cpu), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            fa.fa_paged_attn(*args, return_lse=True)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            out = fa.fa_paged_attn(*args, return_lse=True)
        graphs.append((cpu, args, s, g, out))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, _, s, g, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (q, kc, vc, ks, vs, cu, lens, pages), _, _, _, (o, lse) in graphs:
        want = plain.attention(q, kc, vc, ks, vs, cu.tolist(), lens.tolist(), pages, 0.125, True, -1)
        compare_attn(o.cpu(), lse.cpu(), *want)


def test_attn_wait_limit_runs_out_then_recovers(cuda_device):
    """Under a 1 us limit the kernel's waits run out: it reports the timeout,
    unwinds and returns, and the same call then succeeds under the default."""
    assert fa.fa_get_device_status() == fa.FA_OK
    gen = torch.Generator().manual_seed(64)
    lens = [3000, 200, 64]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 128, gen) for _ in range(2))
    q = torch.randn((4, 8, 128), generator=gen).bfloat16()
    cpu = (q, kc, vc, ks, vs, plain.cum([1, 2, 1]), torch.tensor(lens, dtype=torch.int32), pages)
    args = dev(*cpu)
    try:
        fa.fa_set_wait_limit_ns(1000)
        fa.fa_paged_attn(*args, return_lse=True)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_ERR_DEVICE_TIMEOUT
    finally:
        fa.fa_set_wait_limit_ns(0)
    assert fa.fa_get_device_status() == fa.FA_OK
    o, lse = fa.fa_paged_attn(*args, return_lse=True)
    want = plain.attention(q, kc, vc, ks, vs, [0, 1, 3, 4], lens, pages, 128 ** -0.5, True, -1)
    compare_attn(o.cpu(), lse.cpu(), *want)
    assert fa.fa_get_device_status() == fa.FA_OK


def test_append_then_attend_on_a_given_stream(cuda_device):
    """Append and attention of one cache on one side stream, given by hand."""
    gen = torch.Generator().manual_seed(65)
    pages, num = plain.make_pages([200, 70], gen)
    kc = torch.zeros((num, 2, 64, 64), dtype=torch.float8_e4m3fn, device="cuda")
    vc, ks, vs = kc.clone(), torch.zeros((num, 2), device="cuda"), torch.zeros((num, 2),
                                                                             device="cuda")
    kv = torch.randn((270, 4, 64), generator=gen).bfloat16()
    q = torch.randn((2, 4, 64), generator=gen).bfloat16()
    cu, lens = plain.cum([200, 70]), torch.tensor([200, 70], dtype=torch.int32)
    kvd, qd, cud, lensd, pd, one = dev(kv, q, cu, lens, pages, plain.cum([1, 1]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fa.fa_paged_kv_append(kvd[:, :2], kvd[:, 2:], cud, lensd, pd, kc, vc, ks, vs, stream=s)
    o, lse = fa.fa_paged_attn(qd, kc, vc, ks, vs, one, lensd, pd, return_lse=True, stream=s)
    s.synchronize()
    want = plain.attention(q, kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu(), [0, 1, 2], [200, 70], pages,
                           0.125, True, -1)
    compare_attn(o.cpu(), lse.cpu(), *want)


@pytest.mark.parametrize("d", [64, 80, 128])
def test_append_by_either_kernel(cuda_device, d):
    # Both kernels (few tokens a sequence, many) on the same positions.
    check_append([100] + [0] * 30, [20] + [5] * 30, 2, d, 16 * (d // 16), True, seed=66 + d)
    check_append([100, 30], [20, 5], 2, d, 16 * (d // 16), True, seed=67 + d)


@pytest.mark.parametrize("d,Hk", [(64, 3), (96, 1), (128, 9)])
def test_append_of_prompts_and_single_tokens(cuda_device, d, Hk):
    # Single tokens of many sequences with longer pieces among them, on both
    # sides of the 16 tokens that one warp takes, behind part-filled pages.
    check_append([1] * 30 + [150, 16, 17, 1, 0, 64], [37 * i % 130 for i in range(36)], Hk, d,
                 16 * (d // 32), True, seed=70 + d, interleaved=d == 96)
    # Many tokens: blocks that take several heads, an odd one left over.
    check_append([1900, 640], [0, 33], Hk, d, 16 * (d // 32), True, seed=71 + d)


def test_gather_outputs_aligned_to_16_bytes_only(cuda_device):
    gen = torch.Generator().manual_seed(68)
    pages, num = plain.make_pages([100], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([100], pages, num, 2, 64, gen) for _ in range(2))
    buf = torch.zeros((2, 100 * 2 * 64 + 8), dtype=torch.bfloat16, device="cuda")
    outs = [b[8:].view(100, 2, 64) for b in buf]
    assert outs[0].data_ptr() % 32 == 16
    k, v = fa.fa_paged_kv_gather(*dev(kc, vc, ks, vs, plain.cum([100]), pages), 100, k_out=outs[0],
                                 v_out=outs[1])
    assert (buf[:, :8] == 0).all()
    for got, codes, scale in ((k, kc, ks), (v, vc, vs)):
        for h in range(2):
            want, _ = plain.keys_of(0, 100, pages, codes, scale, h)
            assert torch.equal(got[:, h].cpu().double(), want)


@pytest.mark.parametrize("d,H,causal", [(64, 128, True), (128, 96, False)])
def test_attn_groups_wider_than_a_row_tile(cuda_device, d, H, causal):
    # One kv head for all: the heads of a token fill more than one tile.
    check_attn([1, 3, 0, 2], [130, 400, 64, 1], H, 1, d, causal=causal, seed=H)


def test_cache_past_32_bit_offsets(cuda_device):
    # The pages at the end of caches of 4.6 GB give what the first ones give.
    gen = torch.Generator().manual_seed(72)
    Hk, d, many = 8, 128, 70001
    counts, lens = [100, 1], [150, 129]
    pages = torch.tensor([[3, 1, 0], [2, 5, 4]], dtype=torch.int32)
    kv = torch.randn((101, 2 * Hk, d), generator=gen).bfloat16().cuda()
    q = torch.randn((2, 32, d), generator=gen).bfloat16().cuda()
    tab = dev(plain.table(192, d))
    first = torch.randint(0, 256, (2, 6, Hk, 64, d), generator=gen, dtype=torch.uint8)
    first[(first & 127) == 127] = 0                              # no NaN
    got = []
    for num, ids in ((6, pages), (many, many - 1 - pages)):
        rows = ids.flatten().long().cuda()
        kc, vc = (torch.empty((num, Hk, 64, d), dtype=torch.uint8, device="cuda") for _ in "kv")
        for c, x in ((kc, first[0]), (vc, first[1])):
            c[rows] = x[pages.flatten().long()].cuda()
        ks, vs = (torch.full((num, Hk), 2.0 ** -5, device="cuda") for _ in "kv")
        cache = (kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs)
        lend, idd = dev(torch.tensor(lens, dtype=torch.int32), ids)
        fa.fa_paged_kv_append(kv[:, :Hk], kv[:, Hk:], dev(plain.cum(counts)), lend, idd, *cache,
                              cos_sin=tab)
        o, lse = fa.fa_paged_attn(q, *cache, dev(plain.cum([1, 1])), lend, idd, return_lse=True)
        k, v = fa.fa_paged_kv_gather(*cache, dev(plain.cum(lens)), idd, sum(lens))
        got.append([t.cpu() for t in (kc[rows], vc[rows], ks[rows], vs[rows], o, lse, k, v)])
    assert fa.fa_get_device_status() == fa.FA_OK
    assert torch.isfinite(got[0][4]).all()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_more_sequences_than_a_block_has_threads(cuda_device):
    check_append([1] * 1100, [i % 130 for i in range(1100)], 1, 64, 0, False, seed=73)
    check_append([17] * 300, [i % 130 for i in range(300)], 1, 128, 0, False, seed=74)
    test_gather_is_exact(cuda_device, 64, 1, [i % 3 for i in range(700)])


# ------------------------------------------------------- V scales far apart
def check_far_scales(scales, tiles, batch, tops=None, hi=1.0, d=64, H=4, seed=80):
    """`batch` sequences of 128-key tiles whose pages' V scales are scales[t]
    for tile t (a pair: its two pages), scores 0, or tops[t] (base 2) for all
    keys of tile t."""
    gen = torch.Generator().manual_seed(seed)
    n = 128 * tiles
    pages, num = plain.make_pages([n] * batch, gen)
    kc = torch.zeros((num, 1, 64, d), dtype=torch.float8_e4m3fn)
    vc = (torch.randn((num, 1, 64, d), generator=gen) * hi).to(torch.float8_e4m3fn)
    ks, vs = torch.ones((num, 1)), torch.zeros((num, 1))
    q = torch.ones((batch, H, d)).bfloat16()
    scale = math.log(2) / d
    for t in range(tiles):
        pair = scales[t % len(scales)]
        for i, s in enumerate(pair if isinstance(pair, tuple) else (pair, pair)):
            vs[pages[:, 2 * t + i].long()] = s
            if tops:   # score = scale * d * top * ln 2 / ln 2
                kc.view(torch.uint8)[pages[:, 2 * t + i].long()] = torch.tensor(
                    tops[t % len(tops)]).to(torch.float8_e4m3fn).view(torch.uint8)
    o, lse = fa.fa_paged_attn(*dev(q, kc, vc, ks, vs, plain.cum([1] * batch),
                                   torch.full((batch,), n, dtype=torch.int32), pages),
                              max_seqlen_q=1, softmax_scale=scale, return_lse=True)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    want = plain.attention(q, kc, vc, ks, vs, list(range(batch + 1)), [n] * batch, pages, scale,
                           True, -1)
    compare_attn(o.cpu(), lse.cpu(), *want)


LO, HI = 2.0 ** -64, 2.0 ** 64


@pytest.mark.parametrize("batch,tiles", [(1, 2), (1, 8), (300, 2), (300, 5)])
@pytest.mark.parametrize("scales", [(LO, HI), (HI, LO), (0.0, HI), (HI, 0.0), ((LO, HI), (HI, LO)),
                                    (LO, LO, HI, HI), (HI, HI, LO, LO), (LO, 1.0, HI)])
def test_attn_v_scales_at_both_ends(cuda_device, scales, batch, tiles):
    """Keys whose V scale is 2^128 below another's (an all-zero page has 2^-64)
    keep their share of the softmax, whichever tile, warpgroup or CTA they are
    in.  A key of the small scale adds at most 448 * 2^-25 to an output of at
    least 2^7 sum |code| of the large one's, far inside the tolerance's 2^-10."""
    check_far_scales(scales, tiles, batch)


@pytest.mark.parametrize("batch,tiles", [(1, 4), (300, 4)])
@pytest.mark.parametrize("turn", [False, True])
def test_attn_large_values_under_small_weights(cuda_device, batch, tiles, turn):
    """Weights of 2^-128 and values of 2^64 beside weights of 1 and values of
    2^-64: both sides are about half of the output.  (128 is an e4m3 number.)"""
    scales, tops = (HI, HI, LO, LO), (0.0, 0.0, 128.0, 128.0)
    if turn:
        scales, tops = scales[::-1], tops[::-1]
    check_far_scales(scales, tiles, batch, tops=tops)


# ---------------------------------------------- views with strides of no use
def turned(x):
    """x [1, H, d] as the torch-contiguous tensor with the strides (d, d, 1)."""
    y = torch.empty((x.shape[1], 1, x.shape[2]), dtype=x.dtype, device=x.device).transpose(0, 1)
    y.copy_(x)
    assert y.is_contiguous() and y.stride()[:2] == (x.shape[2], x.shape[2])
    return y


@pytest.mark.parametrize("d", [64, 80, 128])
def test_one_row_turned_round(cuda_device, d):
    gen = torch.Generator().manual_seed(90 + d)
    H, Hk = 8, 2
    q, k, v = dev(*(torch.randn((1, h, d), generator=gen).bfloat16() for h in (H, Hk, Hk)))
    tab, w, pos = dev(plain.table(200, d), torch.rand(d, generator=gen),
                      torch.tensor([129], dtype=torch.int32))
    qo, ko = fa.fa_qk_norm_rope(q, k, pos, tab, w, w)
    out = [turned(torch.zeros_like(t)) for t in (q, k)]
    got = fa.fa_qk_norm_rope(turned(q), turned(k), pos, tab, w, w, q_out=out[0], k_out=out[1])
    assert torch.equal(got[0], qo) and torch.equal(got[1], ko)
    assert got[0].data_ptr() == out[0].data_ptr()
    pages, num = plain.make_pages([130], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([129], pages, num, Hk, d, gen, 0) for _ in range(2))
    lens, cu = dev(torch.tensor([130], dtype=torch.int32), plain.cum([1]))
    res = []
    for kk, vv, qq in ((k, v, qo), (turned(k), turned(v), turned(qo))):
        c = dev(kc.clone(), vc.clone(), ks.clone(), vs.clone())
        fa.fa_paged_kv_append(kk, vv, cu, lens, dev(pages), *c, cos_sin=tab)
        o, lse = fa.fa_paged_attn(qq, *c, cu, lens, dev(pages), return_lse=True)
        res.append((c[0].view(torch.uint8), c[1].view(torch.uint8), o, lse))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    # Beside a strided tensor fa_varlen_fwd takes its strides too.
    kv = dev(torch.randn((40, 2 * Hk, d), generator=gen).bfloat16())
    cuk = dev(plain.cum([40]))
    a, b = (fa.fa_varlen_fwd(t, kv[:, :Hk], kv[:, Hk:], cu, cuk) for t in (q, turned(q)))
    assert torch.equal(a, b)
    q3, cu3 = dev(torch.randn((3, 2 * H, d), generator=gen).bfloat16(), plain.cum([3]))
    a, b = (fa.fa_varlen_fwd(q3[:, :H], t, u, cu3, cu) for t, u in ((k, v), (turned(k), turned(v))))
    assert torch.equal(a, b)


def test_one_head_with_any_head_stride(cuda_device):
    gen = torch.Generator().manual_seed(94)
    T, d = 70, 64
    buf = dev(torch.randn((T, 3 * d), generator=gen).bfloat16())
    odd = [buf[:, i * d:(i + 1) * d].as_strided((T, 1, d), (3 * d, 5, 1), i * d) for i in range(3)]
    plainly = [t.contiguous() for t in odd]
    tab, pos = dev(plain.table(T, d), torch.arange(T, dtype=torch.int32))
    pages, num = plain.make_pages([T], gen)
    lens, cu = dev(torch.tensor([T], dtype=torch.int32), plain.cum([T]))
    res = []
    for q, k, v in (odd, plainly):
        c = [torch.zeros((num, 1, 64, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in "kv"]
        c += [torch.zeros((num, 1), device="cuda") for _ in "kv"]
        qn, kn = fa.fa_qk_norm_rope(q, k, pos, tab)
        fa.fa_paged_kv_append(k, v, cu, lens, dev(pages), *c, cos_sin=tab)
        o = fa.fa_paged_attn(q, *c, cu, lens, dev(pages))
        f = fa.fa_varlen_fwd(q, k, v, cu, cu)
        res.append((qn, kn, c[0].view(torch.uint8), c[1].view(torch.uint8), o, f))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_attn_hint_that_changes_in_place(cuda_device):
    # A hint may be anything with an integer value; one object may hold
    # another value in the next call, for which another workspace is needed.
    gen = torch.Generator().manual_seed(95)
    pages, num = plain.make_pages([200], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([200], pages, num, 2, 64, gen) for _ in range(2))
    q = torch.randn((9, 8, 64), generator=gen).bfloat16()
    cpu = (q, kc, vc, ks, vs, plain.cum([9]), torch.tensor([200], dtype=torch.int32), pages)
    args, most = dev(*cpu), torch.tensor(1)
    want = plain.attention(q, kc, vc, ks, vs, [0, 9], [200], pages, 0.125, True, -1)
    for hint in (1, 9, 1):
        most.fill_(hint)
        o, lse = fa.fa_paged_attn(*args, max_seqlen_q=most, max_seqlen_k=most, return_lse=True)
        compare_attn(o.cpu(), lse.cpu(), *want)


@pytest.mark.parametrize("size", [2 ** 30 - 1, 2 ** 31 - 1, 2 ** 32, 2 ** 32 + 3, 2 ** 70])
def test_windows_past_every_position(cuda_device, size):
    gen = torch.Generator().manual_seed(96)
    lens, q_lens = [200, 70], [3, 90]     # the second has rows before its first key
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    q = torch.randn((93, 8, 64), generator=gen).bfloat16()
    args = dev(q, kc, vc, ks, vs, plain.cum(q_lens), torch.tensor(lens, dtype=torch.int32), pages)
    k, v = dev(*(torch.randn((270, 2, 64), generator=gen).bfloat16() for _ in "kv"))
    cu, cuk = args[5], dev(plain.cum(lens))
    for causal in (True, False):
        a, b = (fa.fa_paged_attn(*args, causal=causal, window_left=w, return_lse=True)
                for w in (-1, size))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert (a[0] != 0).any(-1).sum() > 500   # (rows of both sequences see keys)
        for win in ((size, -1), (-1, size), (size, size)):
            a, b = (fa.fa_varlen_fwd(args[0], k, v, cu, cuk, 90, 200, causal=causal, window_left=l,
                                     window_right=r, return_lse=True)
                    for l, r in ((-1, -1), win))
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("loud", [1.0, 100.0, 1e4])
def test_attn_queries_with_a_loud_channel(cuda_device, loud):
    """A row of q is held to 2^-17 of its largest value, here one that meets keys
    of 0: the scores may be off by 2^-17 max |q| sum |k| scale more."""
    gen = torch.Generator().manual_seed(97)
    H, Hk, d, n = 8, 2, 64, 300
    pages, num = plain.make_pages([n], gen)
    (kc, ks), (vc, vs) = (plain.make_cache([n], pages, num, Hk, d, gen) for _ in range(2))
    kc.view(torch.uint8)[:, :, :, 5] = 0
    q = torch.randn((1, H, d), generator=gen).bfloat16()
    q[..., 5] = loud
    cpu = (q, kc, vc, ks, vs, plain.cum([1]), torch.tensor([n], dtype=torch.int32), pages)
    o, lse = fa.fa_paged_attn(*dev(*cpu), return_lse=True)
    wo, wl, w, a = plain.attention(q, kc, vc, ks, vs, [0, 1], [n], pages, 0.125, True, -1)
    for h in range(H):
        k, _ = plain.keys_of(0, n, pages, kc, ks, h // (H // Hk))
        # compare_attn takes 2^-15 of a.
        a[h, 0] += 2.0 ** -2 * 0.125 * float(q[0, h].abs().max()) * float(k.abs().sum(1).max())
    compare_attn(o.cpu(), lse.cpu(), wo, wl, w, a)
