"""GPU: sinks behind a sliding window and trees of drafted tokens, over the
paged cache, against their plain fp64 forms.

Tolerances are those of the attention over the paged cache, counted in
roundings: a score is off by at most dx = 2^-15 A, A = scale * sum |q k|, and
2^-20 |x| more; a weight is rounded to at least 11 bits for the product with v,
and O once to bf16: 2^-8 |O| + (2 dx + 2^-10) sum p |v|.  LSE: dx + 2^-20 (1 +
|LSE|).  Masks and positions are whole numbers, and equal.
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


def assert_close(o, lse, want):
    """o, lse against (O, LSE, W, A) of the plain form."""
    wo, wl, w, big = want
    dx = 2.0 ** -15 * big
    tol = 2.0 ** -8 * wo.abs() + (2 * dx.t()[..., None] + 2.0 ** -10) * w + 1e-30
    assert ((o.cpu().double() - wo).abs() <= tol).all()
    if lse is None:
        return
    got = lse.cpu().double()
    empty = torch.isinf(wl)
    assert (got[empty] == wl[empty]).all()
    assert ((got - wl).abs()[~empty] <= (dx + 2.0 ** -20 * (1 + wl.abs()))[~empty]).all()


def check(q_lens, lens, H, Hk, d, causal=True, window=-1, sinks=0, trees=None, words=None, mask=None,
          seed=0, size=1.0, spread=3, break_pages=None, lens_given=None, hints=True, stream=None,
          poison=None):
    gen = torch.Generator().manual_seed(seed)
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, Hk, d, gen, spread) for _ in range(2))
    if poison is not None:
        for c in (kc, vc):
            poison(c.view(torch.uint8), pages)
    if break_pages:
        break_pages(pages, num)
    cu = plain.cum(q_lens)
    q = (torch.randn((int(cu[-1]), H, d), generator=gen) * size).bfloat16()
    if trees is not None:
        mask = masked.tree_masks(trees, words or max(1, -(-max(q_lens) // 32)))
    given = lens if lens_given is None else lens_given
    args = dev(q, kc, vc, ks, vs, cu, i32(given), pages)
    md = None if mask is None else dev(mask)
    if stream is not None:
        torch.cuda.synchronize()
    o, lse = fa.fa_paged_attn(*args, max_seqlen_q=max(q_lens) if hints else 0, causal=causal,
                              window_left=window, sink_tokens=sinks, tree_mask=md, return_lse=True,
                              stream=stream)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    want = masked.paged_attention(q, kc, vc, ks, vs, cu.tolist(), given, pages, d ** -0.5, causal,
                                  window, sinks, mask)
    assert_close(o, lse, want)
    return o, lse


# ------------------------------------------------------------------- sinks
@pytest.mark.parametrize("d", [64, 80, 96, 128])
@pytest.mark.parametrize("sinks", [1, 4, 70, 128, 131, 300])
def test_sinks_dims(cuda_device, d, sinks):
    check([1, 1, 1], [1000, 129, 700], 8, 2, d, window=100, sinks=sinks, seed=d + sinks)


@pytest.mark.parametrize("window", [0, 1, 63, 127, 128, 255, 700])
def test_sinks_windows(cuda_device, window):
    check([1, 3, 9], [900, 129, 400], 4, 2, 64, window=window, sinks=5, seed=window)


@pytest.mark.parametrize("causal", [True, False])
def test_sinks_of_chunks(cuda_device, causal):
    # Several row tiles, whose windows start in different tiles.
    check([70, 1], [600, 300], 8, 2, 64, causal=causal, window=150, sinks=3, seed=1)
    check([33], [33], 4, 1, 128, causal=causal, window=4, sinks=2, seed=2)


def test_sinks_of_lengths_around_them(cuda_device):
    # Shorter than the sinks, as long, one more, and empty.
    check([1, 1, 1, 1, 0, 2], [1, 4, 5, 0, 50, 7], 4, 2, 64, window=1, sinks=4, seed=3)
    check([4, 5], [2, 300], 4, 2, 64, window=2, sinks=2, seed=4)  # more rows than keys


def test_sinks_without_a_window_say_nothing(cuda_device):
    a = check([1, 2], [300, 129], 4, 2, 64, sinks=7, seed=5)
    b = check([1, 2], [300, 129], 4, 2, 64, sinks=0, seed=5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_sinks_as_long_as_everything_are_no_window(cuda_device):
    a = check([1, 2], [300, 1129], 4, 2, 64, window=50, sinks=2 ** 40, seed=6)
    b = check([1, 2], [300, 1129], 4, 2, 64, seed=6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_sinks_over_many_ctas(cuda_device):
    # Units that several CTAs share, gaps inside and at the ends of parts.
    check([1, 1], [20000, 9001], 8, 2, 128, window=6000, sinks=2000, seed=7)
    check([1] * 300, [1 + 53 * i % 1900 for i in range(300)], 4, 1, 64, window=300, sinks=9, seed=8)


def test_pages_between_sinks_and_window_are_not_read(cuda_device):
    def poison(codes, pages):
        # NaN in every page of the gap, and its id taken away in the other run.
        codes[pages[0, 1:9].long()] = plain.NAN_CODE

    def break_pages(pages, num):
        pages[0, 1:9] = -1
    for kw in (dict(poison=poison), dict(break_pages=break_pages)):
        o, lse = check([1], [1000], 4, 2, 128, window=300, sinks=64, seed=9, **kw)
        assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


def test_keys_between_sinks_and_window_in_their_pages(cuda_device):
    # NaN keys in the sinks' page behind them, and in the window's first page.
    def poison(codes, pages):
        codes[pages[0, 0].long(), :, 5:] = plain.NAN_CODE
        codes[pages[0, 10].long(), :, :20] = plain.NAN_CODE
    o, lse = check([1], [1000], 4, 2, 64, window=1000 - 1 - 660, sinks=5, seed=10, poison=poison)
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()


def test_sinks_on_missing_pages(cuda_device):
    def break_pages(pages, num):
        pages[0, 0], pages[1, -1] = -1, num
    check([1, 1], [700, 640], 4, 2, 64, window=100, sinks=70, seed=11, break_pages=break_pages)


def test_sinks_of_lengths_past_the_table(cuda_device):
    # The window lies past the keys that are held: the sinks alone are seen.
    check([1, 1], [130, 700], 4, 2, 64, window=64, sinks=6, seed=12, lens_given=[130, 5000])


# ------------------------------------------------------------------- trees
def trees_of(q_lens, seed, **kw):
    return [masked.random_parents(n, seed + i, **kw) for i, n in enumerate(q_lens)]


@pytest.mark.parametrize("q_lens", [[1], [5], [31], [32], [33], [64], [65, 2], [100], [0, 7, 0]])
def test_draft_tree(cuda_device, q_lens):
    trees = trees_of(q_lens, sum(q_lens))
    lens = [n + 13 * i for i, n in enumerate(q_lens)]
    parents = i32([p for t in trees for p in t])
    mask, pos = fa.fa_draft_tree(*dev(parents, plain.cum(q_lens), i32(lens)), max_nodes=max(q_lens))
    words = -(-max(q_lens) // 32)
    want = masked.tree_masks(trees, words)
    assert mask.dtype == torch.int32 and torch.equal(mask.cpu(), want)
    depths = [lens[b] - n + len(masked.path_of(trees[b], i)) - 1
              for b, n in enumerate(q_lens) for i in range(n)]
    assert pos.cpu().tolist() == depths
    # Fewer words than the nodes: those past them have no bit.
    if words > 1:
        short, again = fa.fa_draft_tree(*dev(parents, plain.cum(q_lens), i32(lens)), max_nodes=3)
        assert torch.equal(short.cpu(), want[:, :1]) and torch.equal(again, pos)


def test_draft_tree_malformed_parents_rows_behind_and_given_outputs(cuda_device):
    parents = i32([-1, 5, 1, -7, 3, 2 ** 31 - 1, 5])
    mask = torch.full((9, 2), 7, dtype=torch.int32, device="cuda")
    pos = torch.full((7,), 7, dtype=torch.int32, device="cuda")
    got = fa.fa_draft_tree(*dev(parents, i32([0, 6]), i32([6])), tree_mask=mask[1:8], positions=pos)
    assert got[0].data_ptr() == mask[1:8].data_ptr() and got[1] is pos
    tree = [-1, -1, 1, -1, 3, -1]
    assert torch.equal(mask[1:7].cpu(), masked.tree_masks([tree], 2))
    assert (mask[0] == 7).all() and (mask[7:] == 7).all() and pos[6] == 7
    assert pos[:6].cpu().tolist() == [0, 0, 1, 0, 1, 0]
    for cu in ([0, 50], [-9, 3], [5, 2]):
        fa.fa_draft_tree(*dev(parents, i32(cu), i32([-2 ** 31])), tree_mask=mask[1:8], positions=pos)
        torch.cuda.synchronize()
        assert (mask[0] == 7).all() and (mask[8] == 7).all()


def test_draft_tree_many_sequences_and_long_chains(cuda_device):
    q_lens = [1 + i % 3 for i in range(70000)]
    trees = [[-1, 0, 0][:n] for n in q_lens]
    parents = i32([p for t in trees for p in t])
    mask, pos = fa.fa_draft_tree(*dev(parents, plain.cum(q_lens), i32(q_lens)), max_nodes=3)
    rows = {0: 1, 1: 3, 2: 5}
    assert mask[:, 0].cpu().tolist() == [rows[i] for n in q_lens for i in range(n)]
    n = 5000
    chain = torch.arange(-1, n - 1, dtype=torch.int32)
    mask, pos = fa.fa_draft_tree(*dev(chain, i32([0, n]), i32([n + 10])), max_nodes=n)
    assert pos.cpu().tolist() == list(range(10, n + 10))
    assert torch.equal(mask.cpu()[[0, 1, 31, 32, n - 1]],
                       i32([masked.words_of(range(i + 1), 157) for i in (0, 1, 31, 32, n - 1)]))


@pytest.mark.parametrize("d", [64, 80, 96, 128])
@pytest.mark.parametrize("H,Hk", [(4, 4), (8, 2), (16, 1), (6, 2)])
def test_tree_dims(cuda_device, d, H, Hk):
    q_lens = [3, 17, 1]
    check(q_lens, [130, 300, 64], H, Hk, d, trees=trees_of(q_lens, d + H), seed=d + H)


@pytest.mark.parametrize("n", [1, 2, 16, 31, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 97, 127, 128, 300])
def test_tree_sizes(cuda_device, n, ctx):
    check([n], [ctx + n], 4, 2, 64, trees=trees_of([n], n + ctx), seed=n + ctx)


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 3), (64, 1), (130, 70), (3000, 2)])
def test_tree_windows(cuda_device, window, sinks):
    # Deep trees, so that the rows' windows differ.
    q_lens = [40, 9, 21]
    trees = trees_of(q_lens, window, chain=0.9)
    check(q_lens, [900, 64, 150], 4, 2, 64, window=window, sinks=sinks, trees=trees, seed=window)
    check(q_lens, [900, 64, 150], 16, 2, 128, window=window, sinks=sinks, trees=trees, seed=window)


def test_tree_over_many_ctas(cuda_device):
    q_lens = [20, 7]
    check(q_lens, [15000, 8001], 8, 2, 128, trees=trees_of(q_lens, 1), seed=21)
    q_lens = [1 + i % 9 for i in range(200)]
    check(q_lens, [n + 41 * i % 500 for i, n in enumerate(q_lens)], 4, 1, 64,
          trees=trees_of(q_lens, 2), seed=22)


def test_tree_that_is_a_chain_is_causal(cuda_device):
    q_lens, lens = [9, 33], [200, 97]
    a = check(q_lens, lens, 8, 2, 64, trees=[list(range(-1, n - 1)) for n in q_lens], seed=23)
    b = check(q_lens, lens, 8, 2, 64, seed=23)
    # (Two kernels, which round P apart: 2^-8 of O and 2^-10 of sum p |v| each.)
    assert ((a[0].float() - b[0].float()).abs() <= 2.0 ** -7 * (1 + b[0].float().abs())).all()
    small = [4, 3]  # 16 rows a sequence: one kernel
    a = check(small, lens, 8, 2, 64, trees=[list(range(-1, n - 1)) for n in small], seed=25)
    b = check(small, lens, 8, 2, 64, seed=25)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = check(q_lens, lens, 8, 2, 64, trees=[list(range(-1, n - 1)) for n in q_lens], window=20,
              sinks=3, seed=24)
    b = check(q_lens, lens, 8, 2, 64, window=20, sinks=3, seed=24)
    # (Nodes name the nodes they see: the window bounds the keys before them
    # alone, so that rows deeper than the window see more than causal ones.)
    same = torch.tensor([i <= 20 for n in q_lens for i in range(n)])
    diff = ((a[0].float() - b[0].float()).abs() <= 2.0 ** -7 * (1 + b[0].float().abs())).cpu()
    assert diff[same].all() and not diff[~same].all()


def test_masks_of_any_bits(cuda_device):
    # Not trees: no bit (an empty row where there is no context), all bits,
    # bits past the last node, more words than nodes, fewer.
    gen = torch.Generator().manual_seed(25)
    q_lens = [5, 40, 3]
    for words in (1, 2, 5):
        mask = torch.randint(-2 ** 31, 2 ** 31, (48, words), generator=gen).int()
        mask[0], mask[1], mask[45] = 0, -1, 0
        for window in (-1, 30):
            check(q_lens, [5, 300, 3], 4, 2, 64, mask=mask, window=window, sinks=2, seed=26)


def test_tree_more_nodes_than_keys(cuda_device):
    # Nodes whose keys would stand before the first one have none.
    check([6, 4], [3, 300], 4, 2, 64, trees=trees_of([6, 4], 3), seed=27)
    check([6], [6], 4, 2, 64, trees=trees_of([6], 3), seed=28, lens_given=[-4])


def test_tree_without_hints_and_on_another_stream(cuda_device):
    q_lens = [12, 1, 30]
    s = torch.cuda.Stream()
    check(q_lens, [100, 64, 333], 8, 4, 96, trees=trees_of(q_lens, 4), seed=29, hints=False)
    check(q_lens, [100, 64, 333], 8, 4, 96, trees=trees_of(q_lens, 4), seed=30, stream=s)


def test_tree_rows_behind_the_last_sequence_and_malformed_cu_seqlens(cuda_device):
    gen = torch.Generator().manual_seed(31)
    lens = [100, 100, 100]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    q = dev(torch.randn((6, 4, 64), generator=gen).bfloat16())
    mask = dev(torch.randint(-2 ** 31, 2 ** 31, (6, 2), generator=gen).int())
    for cu in ([0, 50, 3, 6], [-9, 2, 4, 2 ** 31 - 1], [5, 4, 3, 2], [0, 1, 2, 2]):
        out = torch.full((8, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        fa.fa_paged_attn(q, *dev(kc, vc, ks, vs, i32(cu), i32(lens), pages), out=out[1:-1],
                         window_left=10, sink_tokens=3, tree_mask=mask)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_OK
        assert (out[0] == 7).all() and (out[-1] == 7).all()
    assert (out[3:] == 7).all() and not (out[1:3] == 7).any()


@pytest.mark.parametrize("d", [64, 80, 128])
def test_masked_runs_are_bitwise_the_same(cuda_device, d):
    # Many short units, so that a CTA goes from one to the next under way, its
    # warps apart; whole ones and parts.
    gen = torch.Generator().manual_seed(37)
    q_lens = [1 + i % 9 for i in range(200)]
    lens = [n + 41 * i % 500 for i, n in enumerate(q_lens)]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, d, gen) for _ in range(2))
    q = torch.randn((sum(q_lens), 8, d), generator=gen).bfloat16()
    mask = masked.tree_masks(trees_of(q_lens, 9), 1)
    args = dev(q, kc, vc, ks, vs, plain.cum(q_lens), i32(lens), pages)
    for kw in (dict(tree_mask=dev(mask)), dict(window_left=100, sink_tokens=3)):
        want = fa.fa_paged_attn(*args, max_seqlen_q=9, return_lse=True, **kw)
        for _ in range(15):
            got = fa.fa_paged_attn(*args, max_seqlen_q=9, return_lse=True, **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.fa_get_device_status() == fa.FA_OK


def test_masked_wait_limit_runs_out_then_recovers(cuda_device):
    gen = torch.Generator().manual_seed(32)
    lens = [3000] * 4
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 128, gen) for _ in range(2))
    q = torch.randn((4, 8, 128), generator=gen).bfloat16()
    args = dev(q, kc, vc, ks, vs, plain.cum([1] * 4), i32(lens), pages)
    kw = dict(window_left=500, sink_tokens=4)
    want = fa.fa_paged_attn(*args, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    fa.fa_set_wait_limit_ns(2000)
    try:
        fa.fa_paged_attn(*args, **kw)
        assert fa.fa_get_device_status() == fa.FA_ERR_DEVICE_TIMEOUT
    finally:
        fa.fa_set_wait_limit_ns(0)
    got = fa.fa_paged_attn(*args, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK and torch.equal(got, want)


def test_wide_wait_limit_runs_out_then_recovers(cuda_device):
    # (As above, of a tree with more rows than the 16 of a narrow tile.)
    gen = torch.Generator().manual_seed(38)
    q_lens, lens = [40, 9, 30], [3000, 2000, 2500]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 128, gen) for _ in range(2))
    q = torch.randn((79, 8, 128), generator=gen).bfloat16()
    args = dev(q, kc, vc, ks, vs, plain.cum(q_lens), i32(lens), pages)
    kw = dict(max_seqlen_q=40, tree_mask=dev(masked.tree_masks(trees_of(q_lens, 6), 2)))
    want = fa.fa_paged_attn(*args, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    fa.fa_set_wait_limit_ns(2000)
    try:
        fa.fa_paged_attn(*args, **kw)
        assert fa.fa_get_device_status() == fa.FA_ERR_DEVICE_TIMEOUT
    finally:
        fa.fa_set_wait_limit_ns(0)
    got = fa.fa_paged_attn(*args, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK and torch.equal(got, want)


def test_masked_calls_with_a_given_workspace(cuda_device):
    # The plan's bytes do, one fewer is refused, before anything is launched.
    gen = torch.Generator().manual_seed(39)
    q_lens, lens = [40, 2], [900, 300]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    q = torch.randn((42, 4, 64), generator=gen).bfloat16()
    mask = masked.tree_masks(trees_of(q_lens, 7), 2)
    args = dev(q, kc, vc, ks, vs, plain.cum(q_lens), i32(lens), pages)
    grid, rows, need = fa.fa_paged_attn_plan(2, 42, 4, 2, 64, 40, masked=True)
    assert rows == 256 and need > fa.fa_paged_attn_plan(2, 42, 4, 2, 64, 40)[2]
    for kw in (dict(tree_mask=dev(mask)), dict(window_left=90, sink_tokens=7)):
        want = fa.fa_paged_attn(*args, max_seqlen_q=40, **kw)
        held = torch.full((need + 16,), 0xa5, dtype=torch.uint8, device="cuda")
        got = fa.fa_paged_attn(*args, max_seqlen_q=40, workspace=held[:need], **kw)
        assert torch.equal(got, want) and (held[need:] == 0xa5).all()
        out = torch.full_like(got, 7.0)
        with pytest.raises(fa.FaError):
            fa.fa_paged_attn(*args, max_seqlen_q=40, workspace=held[:need - 1], out=out, **kw)
        torch.cuda.synchronize()
        assert (out == 7).all()
    assert fa.fa_get_device_status() == fa.FA_OK


def test_two_masked_graphs_at_once(cuda_device):
    # A workspace each: both replay together, on streams of their own.
    gen = torch.Generator().manual_seed(40)
    q_lens, lens = [33, 6, 20], [2000, 700, 1500]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 128, gen) for _ in range(2))
    q = torch.randn((59, 8, 128), generator=gen).bfloat16()
    args = dev(q, kc, vc, ks, vs, plain.cum(q_lens), i32(lens), pages)
    mask = dev(masked.tree_masks(trees_of(q_lens, 8), 2))
    calls = (dict(tree_mask=mask), dict(window_left=200, sink_tokens=5))
    want = [fa.fa_paged_attn(*args, max_seqlen_q=33, **kw) for kw in calls]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in calls]
    for kw in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fa.fa_paged_attn(*args, max_seqlen_q=33, **kw))
    for _ in range(10):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert fa.fa_get_device_status() == fa.FA_OK


def test_masked_calls_in_a_graph(cuda_device):
    # Lengths, trees and queries change in place between replays.
    gen = torch.Generator().manual_seed(33)
    q_lens, lens = [9, 14], [200, 333]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 64, gen) for _ in range(2))
    cu = plain.cum(q_lens)
    q = torch.randn((23, 4, 64), generator=gen).bfloat16()
    qd, cud, ld, pd = dev(q, cu, i32(lens), pages)
    cache = dev(kc, vc, ks, vs)
    parents = dev(i32([p for t in trees_of(q_lens, 5) for p in t]))

    def step():
        mask, pos = fa.fa_draft_tree(parents, cud, ld, max_nodes=14)
        return (pos,) + fa.fa_paged_attn(qd, *cache, cud, ld, pd, max_seqlen_q=14, window_left=100,
                                         sink_tokens=4, tree_mask=mask, return_lse=True)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pos, o, lse = step()
    for trial, now in enumerate(([200, 333], [14, 120])):
        trees = trees_of(q_lens, 50 + trial)
        parents.copy_(i32([p for t in trees for p in t]))
        ld.copy_(i32(now))
        qd.mul_(1 + trial)
        g.replay()
        torch.cuda.synchronize()
        want = masked.paged_attention(qd.cpu(), kc, vc, ks, vs, cu.tolist(), now, pages, 0.125, True,
                                      100, 4, masked.tree_masks(trees, 1))
        assert_close(o, lse, want)
        assert pos.cpu().tolist() == [now[b] - n + len(masked.path_of(trees[b], i)) - 1
                                      for b, n in enumerate(q_lens) for i in range(n)]


# -------------------------------------------- the packed (bf16) attention
def check_packed(q_lens, k_lens, H, Hk, d, dv=None, causal=True, wl=-1, wr=-1, sinks=0, trees=None,
                 words=None, mask=None, seed=0, hints=True, strided=False, size=1.0, only=None):
    """fa_varlen_fwd with the masks.  P is rounded to bf16 there for the
    product with v: 2^-8 sum p |v| more than above.  only: heads compared."""
    gen = torch.Generator().manual_seed(seed)
    dv = dv or d
    cu_q, cu_k = plain.cum(q_lens), plain.cum(k_lens)
    q = (torch.randn((int(cu_q[-1]), H, d), generator=gen) * size).bfloat16()
    kv = torch.randn((int(cu_k[-1]), Hk, d + dv), generator=gen).bfloat16()
    k, v = kv[..., :d], kv[..., d:]
    if trees is not None:
        mask = masked.tree_masks(trees, words or max(1, -(-max(q_lens) // 32)))
    kvd = dev(kv)
    kd, vd = kvd[..., :d], kvd[..., d:]
    if not strided:
        kd, vd = kd.contiguous(), vd.contiguous()
    o, lse = fa.fa_varlen_fwd(dev(q), kd, vd, dev(cu_q), dev(cu_k), max(q_lens) if hints else 0,
                              max(k_lens) if hints else 0, causal=causal, window_left=wl,
                              window_right=wr, sink_tokens=sinks,
                              tree_mask=None if mask is None else dev(mask), return_lse=True)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    rows = None if mask is None else mask.tolist()
    got_o, got_l = o.cpu().double(), lse.cpu().double()
    for b, (n, length) in enumerate(zip(q_lens, k_lens)):
        seen = [masked.seen_keys(i, n, length, length, causal, wl, wr, sinks,
                                 None if rows is None else rows[int(cu_q[b]) + i])
                for i in range(n)]
        if not n:
            continue
        seen = torch.stack(seen)
        for h in range(H) if only is None else only:
            kh = k[cu_k[b]:cu_k[b + 1], h // (H // Hk)].double()
            vh = v[cu_k[b]:cu_k[b + 1], h // (H // Hk)].double()
            qh = q[cu_q[b]:cu_q[b + 1], h].double()
            x = (qh @ kh.t() * d ** -0.5).masked_fill(~seen, -torch.inf)
            l = torch.logsumexp(x, 1) if length else torch.full((n,), -torch.inf)
            empty = ~seen.any(1)
            p = torch.exp(x - torch.where(empty, 0.0, l)[:, None])
            dx = 2.0 ** -15 * ((qh.abs() @ kh.abs().t()) * d ** -0.5).masked_fill(~seen, 0)
            dx = dx.amax(1) if length else torch.zeros(n)
            want, w = p @ vh, p @ vh.abs()
            tol = 2.0 ** -8 * want.abs() + (2 * dx[:, None] + 2.0 ** -8 + 2.0 ** -10) * w + 1e-30
            at = slice(int(cu_q[b]), int(cu_q[b + 1]))
            assert ((got_o[at, h] - want).abs() <= tol).all(), (b, h)
            assert (got_l[h, at][empty] == -torch.inf).all() and (got_o[at, h][empty] == 0).all()
            diff = (got_l[h, at] - l).abs()[~empty]
            assert (diff <= (dx + 2.0 ** -20 * (1 + l.abs()))[~empty]).all(), (b, h)
    return o, lse


DIMS = [(64, 64), (72, 72), (80, 80), (96, 96), (128, 128), (192, 128)]


@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("wl,sinks", [(100, 4), (0, 1), (300, 130), (128, 257), (1, 10000), (90, 64),
                                      (90, 65), (200, 192), (200, 193)])
def test_packed_sinks(cuda_device, d, dv, wl, sinks):
    check_packed([700, 1, 129, 0, 260], [700, 600, 129, 5, 900], 4, 4, d, dv, wl=wl, sinks=sinks,
                 seed=d + wl)


@pytest.mark.parametrize("H,Hk", [(8, 2), (8, 1), (32, 2)])
@pytest.mark.parametrize("q_lens,k_lens", [([1, 1, 3], [900, 64, 500]), ([40, 17], [1000, 17]),
                                           ([200], [777])])
def test_packed_sinks_of_grouped_heads(cuda_device, H, Hk, q_lens, k_lens):
    for d, dv in ((64, 64), (128, 128)):
        check_packed(q_lens, k_lens, H, Hk, d, dv, wl=150, sinks=5, seed=H)


def test_packed_sinks_not_causal(cuda_device):
    for wr in (-1, 0, 40):
        check_packed([300, 65], [300, 900], 2, 2, 80, causal=False, wl=70, wr=wr, sinks=9, seed=wr + 1)


def test_packed_sinks_of_short_segments_and_more_rows_than_keys(cuda_device):
    lens = [1 + 7 * i % 64 for i in range(40)]
    check_packed(lens, lens, 2, 2, 64, wl=9, sinks=3, seed=1)
    check_packed([100, 70], [30, 70], 2, 1, 64, wl=9, sinks=3, seed=2)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
def test_packed_sinks_split_over_clusters(cuda_device, d, dv):
    # One item's key tiles over several CTAs, the gap inside a part or not.
    for wl, sinks in ((8000, 4), (12000, 3000), (2500, 140)):
        assert fa.fa_varlen_fwd_plan(1, 64, 16384, 2, 2, d, dv, 64, 16384, True, wl)[1] > 1
        check_packed([64], [16384], 2, 2, d, dv, wl=wl, sinks=sinks, seed=wl)


def test_packed_sinks_say_nothing_without_a_window(cuda_device):
    a = check_packed([300], [500], 2, 2, 64, sinks=7, seed=3)
    b = check_packed([300], [500], 2, 2, 64, seed=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("wl,sinks", [(-1, 0), (100, 5)])
def test_packed_trees(cuda_device, d, dv, wl, sinks):
    q_lens = [3, 70, 0, 300, 1]
    check_packed(q_lens, [130, 70, 9, 900, 600], 4, 2, d, dv, wl=wl, sinks=sinks,
                 trees=trees_of(q_lens, d, chain=0.7), seed=d, strided=d == 128)


@pytest.mark.parametrize("ctx", [0, 1, 31, 32, 63, 97, 127, 128, 400])
def test_packed_tree_contexts(cuda_device, ctx):
    for n in (2, 33, 64, 150):
        check_packed([n], [ctx + n], 8, 2, 64, trees=trees_of([n], n + ctx), wl=200, sinks=1, seed=n)


def test_packed_masks_of_any_bits(cuda_device):
    gen = torch.Generator().manual_seed(25)
    q_lens = [5, 140, 3]
    for words in (1, 2, 5, 9):
        mask = torch.randint(-2 ** 31, 2 ** 31, (148, words), generator=gen).int()
        mask[0], mask[1], mask[145] = 0, -1, 0
        for wl in (-1, 30):
            check_packed(q_lens, [5, 300, 2], 4, 2, 64, mask=mask, wl=wl, sinks=2, seed=26)


def test_packed_trees_split_over_clusters_and_many_sequences(cuda_device):
    check_packed([60], [16384], 8, 2, 128, trees=trees_of([60], 6), seed=4)
    q_lens = [1 + i % 5 for i in range(2100)]  # two launches
    check_packed(q_lens, [n + 3 * i % 50 for i, n in enumerate(q_lens)], 1, 1, 64,
                 trees=trees_of(q_lens, 7), seed=5)


def test_packed_large_tree_after_the_gather(cuda_device):
    # The path of large trees, against the paged attention of the same rows.
    gen = torch.Generator().manual_seed(34)
    q_lens, lens = [90, 61], [1000, 300]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, 2, 128, gen) for _ in range(2))
    q = torch.randn((151, 8, 128), generator=gen).bfloat16()
    trees = trees_of(q_lens, 8)
    qd, kcd, vcd, ksd, vsd, cu, ld, pd = dev(q, kc, vc, ks, vs, plain.cum(q_lens), i32(lens), pages)
    mask, _ = fa.fa_draft_tree(dev(i32([p for t in trees for p in t])), cu, ld, max_nodes=90)
    cu_k = dev(plain.cum(lens))
    k, v = fa.fa_paged_kv_gather(kcd, vcd, ksd, vsd, cu_k, pd, 1300)
    kw = dict(window_left=400, sink_tokens=3, tree_mask=mask, return_lse=True)
    a = fa.fa_varlen_fwd(qd, k, v, cu, cu_k, 90, 1000, **kw)
    b = fa.fa_paged_attn(qd, kcd, vcd, ksd, vsd, cu, ld, pd, **kw)
    want = masked.paged_attention(q, kc, vc, ks, vs, [0, 90, 151], lens, pages, 128 ** -0.5, True,
                                  400, 3, masked.tree_masks(trees, 3))
    assert_close(*b, want)
    wide = (want[0], want[1], want[2] * 5, want[3])  # (2^-8 sum p |v| more, see check_packed)
    assert_close(*a, wide)


def test_packed_masked_wait_limit_runs_out_then_recovers(cuda_device):
    gen = torch.Generator().manual_seed(35)
    q, k, v = (torch.randn((2000, 4, 64), generator=gen).bfloat16().cuda() for _ in range(3))
    cu = dev(i32([0, 2000]))
    kw = dict(causal=True, window_left=300, sink_tokens=4)
    want = fa.fa_varlen_fwd(q, k, v, cu, cu, 2000, 2000, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    fa.fa_set_wait_limit_ns(2000)
    try:
        fa.fa_varlen_fwd(q, k, v, cu, cu, 2000, 2000, **kw)
        assert fa.fa_get_device_status() == fa.FA_ERR_DEVICE_TIMEOUT
    finally:
        fa.fa_set_wait_limit_ns(0)
    got = fa.fa_varlen_fwd(q, k, v, cu, cu, 2000, 2000, **kw)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK and torch.equal(got, want)


def test_packed_masks_on_another_stream_and_in_a_graph(cuda_device):
    gen = torch.Generator().manual_seed(41)
    q_lens, k_lens = [33, 5], [700, 90]
    q = dev(torch.randn((38, 4, 64), generator=gen).bfloat16())
    k, v = (dev(torch.randn((790, 2, 64), generator=gen).bfloat16()) for _ in range(2))
    cu_q, cu_k = dev(plain.cum(q_lens), plain.cum(k_lens))
    mask = dev(masked.tree_masks(trees_of(q_lens, 10), 2))
    for kw in (dict(tree_mask=mask), dict(window_left=60, sink_tokens=9)):
        call = lambda **more: fa.fa_varlen_fwd(q, k, v, cu_q, cu_k, 33, 700, causal=True,
                                               return_lse=True, **kw, **more)
        want = call()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = call(stream=s)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = call()
        got[0].fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert fa.fa_get_device_status() == fa.FA_OK


def test_packed_rows_behind_the_last_sequence_and_malformed_cu_seqlens(cuda_device):
    gen = torch.Generator().manual_seed(36)
    q, k, v = (torch.randn((200, 2, 64), generator=gen).bfloat16().cuda() for _ in range(3))
    mask = dev(torch.randint(-2 ** 31, 2 ** 31, (200, 3), generator=gen).int())
    for cu_q, cu_k in (([0, 90, 150], [0, 200, 200]), ([-5, 300, 20], [7, 3, 400]),
                       ([50, 20, 60], [0, 2 ** 31 - 1, 9])):
        for tree in (None, mask):
            out = torch.full((202, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
            fa.fa_varlen_fwd(q, k, v, *dev(i32(cu_q), i32(cu_k)), causal=True, window_left=20,
                             sink_tokens=5, tree_mask=tree, out=out[1:-1])
            torch.cuda.synchronize()
            assert fa.fa_get_device_status() == fa.FA_OK
            assert (out[0] == 7).all() and (out[-1] == 7).all()
            if cu_q[0] == 0:
                assert (out[151:] == 7).all()
