"""Trees of drafted tokens under a sliding window: the masks, and attention with them,
against decoding each path token by token.

CPU: the attention's own rule (keys before the nodes' by a position that it counts from
the mask's bits, the nodes' by the bits) applied to these masks names the keys of
that definition, whole numbers, for any tree, window, context and sinks.  GPU: masks
are equal, and outputs within the tolerances of test_gpu_masked (of the packed form,
2^-8 sum p |v| more).
"""
import ctypes
import random

import pytest
import torch

import masked_plain as masked
import paged_plain as plain
import varlen_flashattention_forward_gb300 as fa
import windowed_trees as windowed
from varlen_flashattention_forward_gb300 import build_ext

P = ctypes.c_void_p
INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return fa.load_library()


# --------------------------------------------------------------------- CPU
def test_the_attentions_rule_sees_what_decoding_a_path_sees():
    rng = random.Random(3)
    fell_short = 0
    for trial in range(400):
        n, ctx = rng.choice([1, 2, 9, 40, 70]), rng.choice([0, 1, 3, 30, 200])
        window = rng.choice([-1, 0, 1, 2, 5, 20, 64, 300])
        sinks = rng.choice([0, 1, 4, 5, 33, 500])
        tree = masked.random_parents(n, trial, chain=rng.choice([0.3, 0.9, 1.0]))
        words = -(-n // 32)
        rows = windowed.windowed_masks([tree], [ctx], words, window, sinks).tolist()
        full = masked.tree_masks([tree], words).tolist()
        for i in range(n):
            want = windowed.path_keys(tree, i, ctx, window, sinks)
            seen = masked.seen_keys(i, n, ctx + n, ctx + n, True, window, -1, sinks, rows[i])
            assert seen.nonzero()[:, 0].tolist() == sorted(want), (trial, i)
            old = masked.seen_keys(i, n, ctx + n, ctx + n, True, window, -1, sinks, full[i])
            fell_short += old.nonzero()[:, 0].tolist() != sorted(want)
    assert fell_short > 1000  # masks of all ancestors do not do


def tree(lib, **kw):
    a = dict(par=P(0x1000), cu=P(0x2000), sl=P(0x3000), B=2, T=9, words=1, wl=5, sinks=2,
             mask=P(0x4000), pos=P(0x5000))
    a.update(kw)
    return lib.fa_draft_tree_windowed(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(wl=-2), INV), (dict(sinks=-1), INV), (dict(par=None), INV), (dict(cu=None), INV),
    (dict(sl=None), INV), (dict(mask=None), INV), (dict(B=0), INV), (dict(T=-1), INV),
    (dict(words=0), INV), (dict(par=P(0x1001)), INV), (dict(T=2 ** 20, words=2 ** 12), UNS),
    (dict(T=2 ** 31 - 1), UNS),
])
def test_refusals(lib, kw, expect):
    assert tree(lib, **kw) == expect


def test_valid_calls_fail_only_for_want_of_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert tree(lib) in none and tree(lib, wl=-1, sinks=0, pos=None) in none
    assert tree(lib, wl=2 ** 31 - 1, sinks=2 ** 31 - 1) in none


# --------------------------------------------------------------------- GPU
def dev(*ts):
    got = [t.cuda() for t in ts]
    return got if len(got) > 1 else got[0]


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def parents_of(trees):
    return i32([p for t in trees for p in t])


def masks_of(trees, lens, window, sinks, most, **kw):
    cu = plain.cum([len(t) for t in trees])
    return fa.fa_draft_tree(*dev(parents_of(trees), cu, i32(lens)), max_nodes=most,
                            window_left=window, sink_tokens=sinks, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(-1, 0), (0, 0), (1, 3), (5, 4), (20, 0), (20, 60), (63, 500),
                                          (2 ** 40, 2 ** 40)])
@pytest.mark.parametrize("chain", [0.3, 0.95])
def test_masks(cuda_device, window, sinks, chain):
    nodes, ctxs = [40, 0, 1, 100, 33], [30, 7, 0, 3, 1000]
    trees = [masked.random_parents(n, 7 + n, chain=chain) for n in nodes]
    lens = [c + n for c, n in zip(ctxs, nodes)]
    for words in (1, 2, 4):
        mask, pos = masks_of(trees, lens, window, sinks, 32 * words)
        assert torch.equal(mask.cpu(), windowed.windowed_masks(trees, ctxs, words, window, sinks))
        # Positions are those without a window.
        assert torch.equal(pos, masks_of(trees, lens, -1, 0, 32 * words)[1])


@pytest.mark.gpu
def test_masks_malformed_parents_and_lengths_below_the_nodes(cuda_device):
    # (Sequences shorter than their nodes: positions below 0, and whatever the length.)
    bad = i32([-1, 5, 1, -7, 3, 2 ** 31 - 1])
    tree = [-1, -1, 1, -1, 3, -1]
    for length in (6, 3, -2 ** 31, 2 ** 31 - 1):
        mask = torch.full((8, 1), 7, dtype=torch.int32, device="cuda")
        fa.fa_draft_tree(*dev(bad, i32([0, 6]), i32([length])), tree_mask=mask[1:7], window_left=0,
                         sink_tokens=2)
        torch.cuda.synchronize()
        assert (mask[0] == 7).all() and (mask[7] == 7).all()
        ctx = length - 6
        want = [[p for s, p in enumerate(masked.path_of(tree, i))
                 if s == 0 or ctx + len(masked.path_of(tree, i)) - 1 - s < 2] for i in range(6)]
        assert torch.equal(mask[1:7].cpu(), i32([masked.words_of(w, 1) for w in want]))


def paged_case(nodes, ctxs, Hk, d, chain, seed):
    gen = torch.Generator().manual_seed(seed)
    trees = [masked.random_parents(n, seed + n, chain=chain) for n in nodes]
    lens = [c + n for c, n in zip(ctxs, nodes)]
    pages, num = plain.make_pages(lens, gen)
    (kc, ks), (vc, vs) = (plain.make_cache(lens, pages, num, Hk, d, gen) for _ in range(2))
    return gen, trees, lens, pages, kc, ks, vc, vs


def assert_close(o, lse, want, more=0.0):
    wo, wl, w, big = want
    dx = 2.0 ** -15 * big
    tol = 2.0 ** -8 * wo.abs() + (2 * dx.t()[..., None] + 2.0 ** -10 + more) * w + 1e-30
    assert ((o.cpu().double() - wo).abs() <= tol).all()
    assert ((lse.cpu().double() - wl).abs() <= dx + 2.0 ** -20 * (1 + wl.abs())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("nodes,ctxs", [([4, 3, 1], [200, 0, 2]),      # 16 rows of a group at most
                                        ([40, 9, 21], [860, 2, 130])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 2), (5, 4), (20, 0), (20, 40), (100, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_attention_is_that_of_decoding_each_path(cuda_device, nodes, ctxs, window, sinks, d):
    H, Hk = 8, 2
    gen, trees, lens, pages, kc, ks, vc, vs = paged_case(nodes, ctxs, Hk, d, 0.9, 50 + window)
    q = torch.randn((sum(nodes), H, d), generator=gen).bfloat16()
    mask, _ = masks_of(trees, lens, window, sinks, max(nodes))
    o, lse = fa.fa_paged_attn(*dev(q, kc, vc, ks, vs, plain.cum(nodes), i32(lens), pages),
                              max_seqlen_q=max(nodes), window_left=window, sink_tokens=sinks,
                              tree_mask=mask, return_lse=True)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    keys = windowed.cached(pages, kc, ks, vc, vs, lens, H // Hk)
    assert_close(o, lse, windowed.decoded(q, trees, ctxs, keys, d ** -0.5, window, sinks))


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 4), (20, 40), (100, 5)])
@pytest.mark.parametrize("d,dv", [(64, 64), (80, 80), (128, 128), (192, 128)])
def test_packed_attention_is_that_of_decoding_each_path(cuda_device, window, sinks, d, dv):
    nodes, ctxs, H, Hk = [40, 3, 70], [300, 2, 0], 4, 2
    gen = torch.Generator().manual_seed(60 + window + d)
    trees = [masked.random_parents(n, n, chain=0.9) for n in nodes]
    lens = [c + n for c, n in zip(ctxs, nodes)]
    cu_k = plain.cum(lens)
    q = torch.randn((sum(nodes), H, d), generator=gen).bfloat16()
    k, v = (torch.randn((sum(lens), Hk, x), generator=gen).bfloat16() for x in (d, dv))
    mask, _ = masks_of(trees, lens, window, sinks, max(nodes))
    o, lse = fa.fa_varlen_fwd(*dev(q, k, v, plain.cum(nodes), cu_k), max(nodes), max(lens),
                              window_left=window, sink_tokens=sinks, tree_mask=mask, return_lse=True)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK

    def keys(b, h):
        at = slice(int(cu_k[b]), int(cu_k[b + 1]))
        return k[at, h // (H // Hk)].double(), v[at, h // (H // Hk)].double()
    assert_close(o, lse, windowed.decoded(q, trees, ctxs, keys, d ** -0.5, window, sinks), 2.0 ** -8)


@pytest.mark.gpu
def test_windowed_trees_in_a_graph_and_on_another_stream(cuda_device):
    # Parents, lengths and queries change in place between replays.
    nodes, ctxs, H, Hk, d, window, sinks = [30, 12], [90, 3], 4, 2, 64, 6, 5
    gen, trees, lens, pages, kc, ks, vc, vs = paged_case(nodes, ctxs, Hk, d, 0.9, 70)
    cu = plain.cum(nodes)
    parents, cud, ld, pd, kcd, vcd, ksd, vsd = dev(parents_of(trees), cu, i32(lens), pages, kc, vc, ks, vs)
    q = dev(torch.randn((42, H, d), generator=gen).bfloat16())
    keys = windowed.cached(pages, kc, ks, vc, vs, lens, H // Hk)

    def step(stream=None):
        mask, _ = fa.fa_draft_tree(parents, cud, ld, max_nodes=30, window_left=window,
                                   sink_tokens=sinks, stream=stream)
        return fa.fa_paged_attn(q, kcd, vcd, ksd, vsd, cud, ld, pd, max_seqlen_q=30,
                                window_left=window, sink_tokens=sinks, tree_mask=mask,
                                return_lse=True, stream=stream)
    want = windowed.decoded(q.cpu(), trees, ctxs, keys, d ** -0.5, window, sinks)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(s)
    s.synchronize()
    assert_close(*got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for trial in range(2):
        trees = [masked.random_parents(n, 80 + trial + n, chain=0.9) for n in nodes]
        parents.copy_(parents_of(trees))
        q.mul_(1 + trial)
        g.replay()
        torch.cuda.synchronize()
        assert_close(*got, windowed.decoded(q.cpu(), trees, ctxs, keys, d ** -0.5, window, sinks))
    assert fa.fa_get_device_status() == fa.FA_OK
