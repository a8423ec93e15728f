"""CPU: refusals of the masked attention and drafted-tree entry points, and the
index arithmetic of units whose keys have a gap."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

import varlen_flashattention_forward_gb300 as fa
from varlen_flashattention_forward_gb300 import build_ext

HERE = os.path.dirname(os.path.abspath(__file__))
P = ctypes.c_void_p
INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return fa.load_library()


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("probe") / "masked_index.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-o", so,
                    os.path.join(HERE, "probes", "masked_index_probe.cpp")], check=True)
    return ctypes.CDLL(so)


# ---------------------------------------------------------------- refusals
def attn(lib, **kw):
    a = dict(kc=P(0x1000), vc=P(0x2000), ks=P(0x3000), vs=P(0x4000), cu=P(0x5000), pt=P(0x6000),
             B=2, T=4, Hk=2, d=64, pages=8, width=4, q=P(0x7000), qr=256, qh=64, sl=P(0x8000), H=4,
             mq=1, mk=64, scale=0.125, causal=1, wl=-1, sinks=4, mask=P(0xa000), words=2,
             out=P(0x9000), lse=None, ws=P(0x10000), wsb=1 << 40)
    a.update(kw)
    return lib.fa_paged_attn_masked(*[a[n] for n in (
        "q qr qh kc vc ks vs cu sl pt B T H Hk d pages width mq mk scale causal wl sinks mask words "
        "out lse ws wsb").split()], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(sinks=-1), INV), (dict(words=-1), INV), (dict(mask=None), INV), (dict(mask=P(0xa002)), INV),
    (dict(words=2 ** 30), UNS), (dict(q=None), INV), (dict(sl=None), INV), (dict(wl=-2), INV),
    (dict(d=72), UNS), (dict(H=3), INV), (dict(ws=P(0x10004)), INV),
])
def test_masked_attn_refusals(lib, kw, expect):
    assert attn(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), INV), (dict(T=-1), INV), (dict(H=3), INV), (dict(Hk=0), INV), (dict(d=72), UNS),
    (dict(mq=-1), INV),
])
def test_masked_plan_refusals(lib, kw, expect):
    a = dict(B=2, T=64, H=4, Hk=2, d=64, mq=32)
    a.update(kw)
    grid, rows, need = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
    args = [a[n] for n in "B T H Hk d mq".split()]
    for plan in (lib.fa_paged_attn_masked_plan, lib.fa_paged_attn_plan):
        assert plan(*args, ctypes.byref(grid), ctypes.byref(rows), ctypes.byref(need)) == expect


def tree(lib, **kw):
    a = dict(par=P(0x1000), cu=P(0x2000), sl=P(0x3000), B=2, T=9, words=1, mask=P(0x4000),
             pos=P(0x5000))
    a.update(kw)
    return lib.fa_draft_tree(*[a[n] for n in "par cu sl B T words mask pos".split()], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(par=None), INV), (dict(cu=None), INV), (dict(sl=None), INV), (dict(mask=None), INV),
    (dict(B=0), INV), (dict(T=-1), INV), (dict(words=0), INV), (dict(par=P(0x1001)), INV),
    (dict(mask=P(0x4002)), INV), (dict(pos=P(0x5001)), INV), (dict(cu=P(0x2002)), INV),
    (dict(T=2 ** 20, words=2 ** 12), UNS),
])
def test_draft_tree_refusals(lib, kw, expect):
    assert tree(lib, **kw) == expect


def test_valid_calls_fail_only_for_want_of_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert attn(lib) in none and attn(lib, mask=None, words=0) in none
    assert attn(lib, T=0, q=None, out=None, ws=None, wsb=0, mask=None) in none
    assert tree(lib) in none and tree(lib, pos=None) in none
    assert tree(lib, T=0, par=None, mask=None, pos=None) in none


def tensors():
    kc = torch.zeros((4, 2, 64, 64), dtype=torch.float8_e4m3fn)
    ks = torch.zeros((4, 2))
    return dict(cache=(kc, kc.clone(), ks, ks.clone()),
                cu=torch.tensor([0, 3], dtype=torch.int32),
                pt=torch.zeros((1, 2), dtype=torch.int32),
                lens=torch.tensor([3], dtype=torch.int32),
                q=torch.zeros((3, 4, 64), dtype=torch.bfloat16),
                parents=torch.tensor([-1, 0, 0], dtype=torch.int32),
                mask=torch.zeros((3, 1), dtype=torch.int32))


@pytest.mark.parametrize("mask", [
    torch.zeros((3, 1), dtype=torch.int64), torch.zeros((2, 1), dtype=torch.int32),
    torch.zeros((3,), dtype=torch.int32), torch.zeros((3, 0), dtype=torch.int32),
    torch.zeros((3, 4), dtype=torch.int32)[:, ::2],
])
def test_python_refuses_masks(lib, mask):
    t = tensors()
    with pytest.raises((TypeError, ValueError)):
        fa.fa_paged_attn(t["q"], *t["cache"], t["cu"], t["lens"], t["pt"], tree_mask=mask)
    with pytest.raises((TypeError, ValueError)):
        fa.fa_draft_tree(t["parents"], t["cu"], t["lens"], tree_mask=mask)


@pytest.mark.parametrize("name,bad", [
    ("parents", lambda t: t.long()), ("parents", lambda t: t[None]), ("cu", lambda t: t.long()),
    ("lens", lambda t: t.expand(2)), ("lens", lambda t: t.float()),
])
def test_python_refuses_trees(lib, name, bad):
    t = tensors()
    t[name] = bad(t[name])
    with pytest.raises((TypeError, ValueError)):
        fa.fa_draft_tree(t["parents"], t["cu"], t["lens"])


def test_python_refuses_trees_off_the_gpu_and_without_nodes(lib):
    t = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_draft_tree(t["parents"], t["cu"], t["lens"])
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_paged_attn(t["q"], *t["cache"], t["cu"], t["lens"], t["pt"], tree_mask=t["mask"])


# -------------------------------------------------------------- work split
def walk(probe, q_lens, lens, hk, group, rows, causal, window, held, sinks, tree, ctas):
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    arr = lambda x: (ctypes.c_int * len(x))(*x)  # noqa: E731
    most = 100000
    out = (ctypes.c_int * (8 * most))()
    n = probe.probe_masked_walk(arr(cu), arr(lens), len(lens), cu[-1], hk, group, rows, causal,
                                window, held, sinks, tree, ctas, most, out)
    assert n >= 0
    return [tuple(out[8 * i:8 * i + 8]) for i in range(n)]


def test_segments_cover_every_seen_tile_once(probe):
    rng = random.Random(7)
    for trial in range(500):
        batch = rng.choice([1, 2, 5, 20])
        q_lens = [rng.choice([0, 1, 1, 2, 7, 40]) for _ in range(batch)]
        held = 64 * rng.randrange(1, 60)
        lens = [rng.choice([0, 1, 64, 128, 129, rng.randrange(0, 4000), -3]) for _ in range(batch)]
        hk, group, rows = rng.choice([1, 2]), rng.choice([1, 3, 4]), rng.choice([16, 32])
        causal, window = rng.randrange(2), rng.choice([-1, 0, 1, 100, 1000])
        sinks, tree = rng.choice([0, 1, 4, 127, 128, 129, 700, 2 ** 31 - 1]), rng.randrange(2)
        segs = walk(probe, q_lens, lens, hk, group, rows, causal, window, held, sinks, tree,
                    rng.choice([1, 2, 7, 152]))
        got = {}
        for c, b, h, t, part_lo, count, unit_count, i in segs:
            assert 0 <= part_lo and count > 0 and part_lo + count <= unit_count
            got.setdefault((b, h, t), []).append((part_lo, count, unit_count))
        for b, (n, ln) in enumerate(zip(q_lens, lens)):
            for h in range(hk):
                for t in range(-(-n * group // rows)):
                    parts = sorted(got.pop((b, h, t)))
                    at = 0
                    for lo, count, unit in parts:
                        assert lo == at and unit == parts[0][2]
                        at += count
                    assert at == parts[0][2]
                    # The tiles that hold a key some row of the tile sees.
                    keys = min(max(ln, 0), held)
                    i0, i1 = t * rows // group, (min((t + 1) * rows, n * group) - 1) // group
                    first = ln - n + (0 if tree else i0)
                    hi = min(keys, ln - n + i1 + 1) if causal and not tree else keys
                    lo = max(0, first - window) if window >= 0 else 0
                    need = {j // 128 for j in range(max(hi, 0)) if j >= lo or j < sinks}
                    order = [probe.probe_tile_of(n, ln, t, hk, group, rows, causal, window, held,
                                                 sinks, tree, u) for u in range(at)]
                    assert order == sorted(set(order))
                    if need:
                        assert set(order) == need, (n, ln, window, sinks, held)
                    else:
                        assert at == 1
        assert not got


# ------------------------------------------------------- packed attention
def test_a_place_is_in_the_range_that_holds_it(probe):
    big = 2 ** 31 - 1
    for total in (1, 2, 5, 151, 152, 153, 400, 4567, big - 1, big):
        for ctas in (1, 2, 7, 152, 456):
            starts = [probe.probe_range_start(total, ctas, c) for c in range(ctas + 1)]
            places = {p for s in starts for p in (s - 1, s, s + 1)} | {0, total // 2, total - 1}
            for p in places:
                if 0 <= p < total:
                    c = probe.probe_range_of(total, ctas, p)
                    assert starts[c] <= p < starts[c + 1], (total, ctas, p)


def packed(lib, **kw):
    a = dict(q=P(0x1000), qr=256, qh=64, k=P(0x2000), kr=256, kh=64, v=P(0x3000), vr=256, vh=64,
             cq=P(0x4000), ck=P(0x5000), batch=2, total_q=10, total_k=10, H=4, Hk=4, dqk=64, dv=64,
             mq=0, mk=0, scale=0.125, causal=1, wl=5, wr=-1, sinks=4, mask=P(0x7000), words=1,
             out=P(0x6000), lse=None)
    a.update(kw)
    return lib.fa_varlen_fwd_masked(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(sinks=-1), INV), (dict(words=-1), INV), (dict(mask=None), INV), (dict(mask=P(0x7001)), INV),
    (dict(wr=0), INV), (dict(words=2 ** 30), UNS), (dict(q=None), INV), (dict(wl=-2), INV),
    (dict(dqk=100, dv=100), UNS), (dict(kh=60), INV), (dict(H=6), INV),
])
def test_masked_varlen_refusals(lib, kw, expect):
    assert packed(lib, **kw) == expect


def test_valid_packed_calls_fail_only_for_want_of_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert packed(lib) in none and packed(lib, words=0, mask=None, wr=3) in none
    assert packed(lib, total_q=0, q=None, out=None, mask=None) in none


def test_python_refuses_packed_masks(lib):
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_varlen_fwd(q, q, q, cu, cu, window_left=1, sink_tokens=1)
    for mask in (torch.zeros((2, 1), dtype=torch.int32), torch.zeros((3, 1)),
                 torch.zeros((3, 0), dtype=torch.int32)):
        with pytest.raises((TypeError, ValueError)):
            fa.fa_varlen_fwd(q, q, q, cu, cu, tree_mask=mask)


# ---------------------------------------------------------------- eviction
def weights(lib, **kw):
    a = dict(q=P(0x7000), qr=256, qh=64, lse=P(0x9000), kc=P(0x1000), ks=P(0x3000), cu=P(0x5000),
             sl=P(0x8000), pt=P(0x6000), B=2, T=4, H=4, Hk=2, d=64, pages=8, width=4, scale=0.125,
             causal=1, wl=-1, sinks=0, decay=1.0, w=P(0xa000), cap=256)
    a.update(kw)
    return lib.fa_paged_key_weights(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(lse=None), INV), (dict(kc=None), INV), (dict(ks=None), INV),
    (dict(cu=None), INV), (dict(sl=None), INV), (dict(pt=None), INV), (dict(w=None), INV),
    (dict(B=0), INV), (dict(T=-1), INV), (dict(H=3), INV), (dict(Hk=0), INV), (dict(wl=-2), INV),
    (dict(sinks=-1), INV), (dict(decay=-0.1), INV), (dict(decay=1.5), INV),
    (dict(decay=float("nan")), INV), (dict(cap=0), INV), (dict(scale=0.0), INV),
    (dict(w=P(0xa002)), INV), (dict(lse=P(0x9001)), INV), (dict(q=P(0x7008)), INV),
    (dict(qh=60), INV), (dict(d=72), UNS), (dict(width=2 ** 25), UNS),
])
def test_weights_refusals(lib, kw, expect):
    assert weights(lib, **kw) == expect


def select(lib, **kw):
    a = dict(w=P(0x1000), sl=P(0x2000), B=2, Hk=2, cap=256, budget=64, sinks=4, recent=16,
             keep=P(0x3000), new=P(0x4000))
    a.update(kw)
    return lib.fa_paged_kv_select(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(w=None), INV), (dict(sl=None), INV), (dict(keep=None), INV), (dict(new=None), INV),
    (dict(B=0), INV), (dict(Hk=0), INV), (dict(cap=0), INV), (dict(budget=0), INV),
    (dict(sinks=-1), INV), (dict(recent=-1), INV), (dict(sinks=60), INV),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), INV), (dict(w=P(0x1002)), INV),
    (dict(keep=P(0x3001)), INV), (dict(B=2 ** 30, Hk=4), UNS), (dict(cap=2 ** 31 - 1), UNS),
    (dict(budget=2 ** 31 - 1), UNS),
])
def test_select_refusals(lib, kw, expect):
    assert select(lib, **kw) == expect


def compact(lib, **kw):
    a = dict(kc=P(0x1000), vc=P(0x2000), ks=P(0x3000), vs=P(0x4000), pt=P(0x5000), keep=P(0x6000),
             first=P(0x7000), counts=P(0x8000), B=2, Hk=2, heads=2, row=64, d=64, pages=8, width=4,
             w=P(0x9000), cap=256)
    a.update(kw)
    return lib.fa_paged_kv_compact(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(ks=None), INV), (dict(vs=None), INV),
    (dict(pt=None), INV), (dict(keep=None), INV), (dict(counts=None), INV), (dict(B=0), INV),
    (dict(Hk=0), INV), (dict(heads=3), INV), (dict(heads=0), INV), (dict(row=-1), INV),
    (dict(pages=0), INV), (dict(width=0), INV), (dict(cap=0), INV), (dict(kc=P(0x1008)), INV),
    (dict(keep=P(0x6002)), INV), (dict(first=P(0x7001)), INV), (dict(counts=P(0x8002)), INV),
    (dict(w=P(0x9001)), INV), (dict(d=72), UNS), (dict(width=2 ** 25), UNS),
    (dict(B=2 ** 27), UNS),
])
def test_compact_refusals(lib, kw, expect):
    assert compact(lib, **kw) == expect


def test_valid_eviction_calls_fail_only_for_want_of_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert weights(lib) in none and weights(lib, T=0, q=None, lse=None) in none
    assert select(lib) in none and select(lib, budget=20) in none
    assert compact(lib) in none and compact(lib, first=None, w=None, cap=0, heads=1) in none


def test_python_refuses_eviction_arguments(lib):
    t = tensors()
    kc, vc, ks, vs = t["cache"]
    w = torch.zeros((1, 2, 128))
    lse = torch.zeros((4, 3))
    keep = torch.zeros((1, 2, 3), dtype=torch.int32)
    bad = (TypeError, ValueError)
    for fn in (lambda: fa.fa_paged_key_weights(t["q"], lse[:3], kc, ks, t["cu"], t["lens"], t["pt"], w),
               lambda: fa.fa_paged_key_weights(t["q"], lse, kc, ks, t["cu"], t["lens"], t["pt"], w[0]),
               lambda: fa.fa_paged_key_weights(t["q"], lse, kc, ks, t["cu"], t["lens"], t["pt"],
                                               w.double()),
               lambda: fa.fa_paged_kv_select(w, t["lens"].long(), 5),
               lambda: fa.fa_paged_kv_select(w[0], t["lens"], 5),
               lambda: fa.fa_paged_kv_select(w, t["lens"].expand(2), 5),
               lambda: fa.fa_paged_kv_compact(*t["cache"], t["pt"], keep[0], t["lens"]),
               lambda: fa.fa_paged_kv_compact(*t["cache"], t["pt"], keep.expand(2, 2, 3), t["lens"]),
               lambda: fa.fa_paged_kv_compact(*t["cache"], t["pt"], keep, t["lens"].long()),
               lambda: fa.fa_paged_kv_compact(*t["cache"], t["pt"], keep, t["lens"], weights=w[0]),
               lambda: fa.fa_paged_kv_compact(*t["cache"], t["pt"], keep, t["lens"],
                                              first=t["cu"])):
        with pytest.raises(bad):
            fn()
    for fn in (lambda: fa.fa_paged_key_weights(t["q"], lse, kc, ks, t["cu"], t["lens"], t["pt"], w),
               lambda: fa.fa_paged_kv_select(w, t["lens"], 5),
               lambda: fa.fa_paged_kv_compact(*t["cache"], t["pt"], keep, t["lens"])):
        with pytest.raises(ValueError, match="CUDA"):
            fn()
