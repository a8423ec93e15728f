"""CPU checks of the paged-cache operators: the kernels' index arithmetic on
ordinary and malformed arrays (built for the host from the header the kernels
include), the host refusals of the C entry points, and the Python checks."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

import varlen_flashattention_forward_gb300 as fa
from varlen_flashattention_forward_gb300 import build_ext

HERE = os.path.dirname(os.path.abspath(__file__))
INT_MAX, INT_MIN = 2 ** 31 - 1, -2 ** 31
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return fa.load_library()


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("probe") / "paged_index.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-shared", "-fPIC", "-o", so,
                    os.path.join(HERE, "probes", "paged_index_probe.cpp")], check=True)
    return ctypes.CDLL(so)


def call(fn, n, *args):
    out = (ctypes.c_int * n)()
    fn(*args, out)
    return list(out)


ODD = [0, 1, 2, 63, 64, 65, 100, 1000, -1, -64, INT_MAX, INT_MIN, INT_MAX - 63, INT_MIN + 1]


def test_row_ranges_stay_inside(probe):
    for c0 in ODD:
        for c1 in ODD:
            for total in (0, 1, 64, 1000, INT_MAX):
                lo, n = call(probe.probe_row_range, 2, c0, c1, total)
                assert 0 <= lo <= total and 0 <= n <= total - lo
                if 0 <= c0 <= c1 <= total:
                    assert (lo, n) == (c0, c1 - c0)


def test_append_spans_stay_inside(probe):
    for n in [x for x in ODD if x >= 0]:
        for ln in ODD:
            for limit in (1, 64, 100, 6400, INT_MAX):
                first, got = call(probe.probe_append_span, 2, n, ln, limit)
                assert got >= 0 and first >= 0
                assert got == 0 or (first == ln - n and first + got == min(ln, limit))


def test_pages_of_a_span_cover_it_once(probe):
    rng = random.Random(0)
    for _ in range(500):
        first, n = rng.randrange(0, 300), rng.randrange(0, 300)
        pages = probe.probe_pages_touched(first, n)
        at = first
        for p in range(first // 64, first // 64 + pages):
            slot, count, row = call(probe.probe_page_span, 3, first, n, p)
            assert count > 0 and 0 <= slot and slot + count <= 64
            assert p * 64 + slot == at and row == at - first
            at += count
        assert at == first + n
        # The grid of a call: chunks of its sequences never outnumber this.
        assert pages <= min(n, n // 64 + 2)


def test_pages_outside_the_cache_are_refused(probe):
    for num in (1, 5, INT_MAX):
        for page in ODD + [num - 1, num]:
            if page > INT_MAX:
                continue
            got = probe.probe_checked_page(page, num)
            assert got == (page if 0 <= page < num else -1)


def test_key_ranges(probe):
    rng = random.Random(1)
    for _ in range(3000):
        n = rng.randrange(1, 20)
        ln = rng.choice([rng.randrange(0, 400), -3, INT_MAX, INT_MIN])
        held = 64 * rng.randrange(1, 8)
        i0 = rng.randrange(0, n)
        i1 = rng.randrange(i0, n)
        causal, window = rng.randrange(2), rng.choice([-1, 0, 1, 70, INT_MAX])
        lo, hi = call(probe.probe_key_range, 2, i0, i1, n, ln, held, causal, window)
        keys = min(max(ln, 0), held)
        assert 0 <= lo <= hi <= keys
        if abs(ln) < 1000:
            for j in range(keys):
                seen = any((not causal or j <= ln - n + i) and (window < 0 or j >= ln - n + i - window)
                           for i in (i0, i1))
                assert not seen or lo <= j < hi, (j, lo, hi)


# ----------------------------------------------------------- host refusals
INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


def norm_rope(lib, **kw):
    a = dict(q=P(0x1000), qr=512, qh=128, k=P(0x2000), kr=256, kh=128, pos=P(0x3000),
             tab=P(0x4000), qw=P(0x5000), kw=P(0x6000), T=3, H=4, Hk=2, d=128, rot=128, maxp=10,
             il=0, eps=1e-6, qo=P(0x7000), qor=512, qoh=128, ko=P(0x8000), kor=256, koh=128)
    a.update(kw)
    return lib.fa_qk_norm_rope(*[a[n] for n in (
        "q qr qh k kr kh pos tab qw kw T H Hk d rot maxp il eps qo qor qoh ko kor koh").split()],
        None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(qo=None), INV), (dict(k=None), INV), (dict(ko=None), INV),
    (dict(T=-1), INV), (dict(H=-1), INV), (dict(H=0, Hk=0), INV), (dict(pos=None), INV),
    (dict(tab=None), INV), (dict(rot=-16), INV), (dict(rot=24), INV), (dict(rot=144), INV),
    (dict(maxp=0), INV), (dict(maxp=-1), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(q=P(0x1008)), INV),
    (dict(tab=P(0x4004)), INV), (dict(pos=P(0x3002)), INV), (dict(qw=P(0x5004)), INV),
    (dict(qr=500), INV), (dict(qr=504), INV), (dict(qh=120), INV), (dict(kor=0), INV),
    (dict(koh=-128), INV), (dict(d=4, rot=0), INV), (dict(d=100, rot=0), UNS),
    (dict(d=264, rot=0), UNS), (dict(T=2 ** 29, H=4, Hk=4, kr=512, kor=512), UNS),
])
def test_norm_rope_refusals(lib, kw, expect):
    assert norm_rope(lib, **kw) == expect


CACHE = dict(kc=P(0x1000), vc=P(0x2000), ks=P(0x3000), vs=P(0x4000), cu=P(0x5000), pt=P(0x6000),
             B=2, T=10, Hk=2, d=64, pages=8, width=4)
CACHE_BAD = [
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(ks=None), INV), (dict(vs=None), INV),
    (dict(cu=None), INV), (dict(pt=None), INV), (dict(B=0), INV), (dict(T=-1), INV),
    (dict(Hk=0), INV), (dict(pages=0), INV), (dict(width=0), INV), (dict(kc=P(0x1008)), INV),
    (dict(ks=P(0x3002)), INV), (dict(pt=P(0x6002)), INV), (dict(d=72), UNS), (dict(d=256), UNS),
    (dict(width=2 ** 25), UNS), (dict(pages=2 ** 30), UNS), (dict(T=2 ** 30), UNS),
]


def append(lib, **kw):
    a = dict(CACHE, k=P(0x7000), kr=128, kh=64, v=P(0x8000), vr=128, vh=64, sl=P(0x9000),
             kw=P(0xa000), eps=1e-6, tab=P(0xb000), rot=64, maxp=100, il=0)
    a.update(kw)
    return lib.fa_paged_kv_append(*[a[n] for n in (
        "k kr kh v vr vh cu sl pt B T Hk d pages width kw eps tab rot maxp il kc vc ks vs"
    ).split()], None)


@pytest.mark.parametrize("kw,expect", CACHE_BAD + [
    (dict(k=None), INV), (dict(v=None), INV), (dict(sl=None), INV), (dict(sl=P(0x9001)), INV),
    (dict(kr=120), INV), (dict(kh=60), INV), (dict(vr=127), INV), (dict(k=P(0x7002)), INV),
    (dict(rot=72), INV), (dict(rot=8), INV), (dict(tab=None), INV), (dict(maxp=0), INV),
    (dict(eps=-1e-6), INV), (dict(tab=P(0xb008)), INV),
])
def test_append_refusals(lib, kw, expect):
    assert append(lib, **kw) == expect


def gather(lib, **kw):
    a = dict(CACHE, ko=P(0x7000), vo=P(0x8000))
    a.update(kw)
    return lib.fa_paged_kv_gather(*[a[n] for n in (
        "kc vc ks vs cu pt B T Hk d pages width ko vo").split()], None)


@pytest.mark.parametrize("kw,expect", CACHE_BAD + [
    (dict(ko=None), INV), (dict(vo=None), INV), (dict(vo=P(0x8008)), INV)])
def test_gather_refusals(lib, kw, expect):
    assert gather(lib, **kw) == expect


def attn(lib, **kw):
    a = dict(CACHE, q=P(0x7000), qr=256, qh=64, sl=P(0x8000), H=4, mq=1, mk=64, scale=0.125,
             causal=1, wl=-1, out=P(0x9000), lse=None, ws=P(0x10000), wsb=1 << 40)
    a.update(kw)
    return lib.fa_paged_attn(*[a[n] for n in (
        "q qr qh kc vc ks vs cu sl pt B T H Hk d pages width mq mk scale causal wl out lse ws wsb"
    ).split()], None)


@pytest.mark.parametrize("kw,expect", CACHE_BAD + [
    (dict(q=None), INV), (dict(out=None), INV), (dict(sl=None), INV), (dict(H=3), INV),
    (dict(H=0), INV), (dict(mq=-1), INV), (dict(mk=-1), INV), (dict(scale=0.0), INV),
    (dict(scale=float("inf")), INV), (dict(wl=-2), INV), (dict(q=P(0x7008)), INV),
    (dict(out=P(0x9004)), INV), (dict(lse=P(0x9001)), INV), (dict(ws=P(0x10004)), INV),
    (dict(qr=200), INV), (dict(qh=63), INV),
])
def test_attn_refusals(lib, kw, expect):
    assert attn(lib, **kw) == expect


def plan(lib, B=2, T=4, H=4, Hk=2, d=64, mq=1, outs=(True, True, True)):
    g, r, w = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    return lib.fa_paged_attn_plan(B, T, H, Hk, d, mq, *[
        ctypes.byref(x) if on else None for x, on in zip((g, r, w), outs)])


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), INV), (dict(T=-1), INV), (dict(H=3), INV), (dict(Hk=0), INV), (dict(mq=-1), INV),
    (dict(d=72), UNS), (dict(outs=(False, True, True)), INV), (dict(outs=(True, False, True)), INV),
    (dict(outs=(True, True, False)), INV)])
def test_attn_plan_refusals(lib, kw, expect):
    assert plan(lib, **kw) == expect


def test_valid_calls_fail_only_for_want_of_a_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert norm_rope(lib) in none and norm_rope(lib, k=None, ko=None, Hk=0) in none
    assert norm_rope(lib, rot=0, pos=None, tab=None, maxp=0, qw=None, kw=None) in none
    assert append(lib) in none and append(lib, kw=None, rot=0, tab=None, maxp=0) in none
    assert append(lib, T=0, k=None, v=None) in none
    assert gather(lib) in none and gather(lib, T=0, ko=None, vo=None) in none
    assert attn(lib) in none and plan(lib) in none
    assert attn(lib, T=0, q=None, out=None, ws=None, wsb=0) in none


# ----------------------------------------------------------- Python checks
def tensors():
    kc = torch.zeros((4, 2, 64, 64), dtype=torch.float8_e4m3fn)
    ks = torch.zeros((4, 2))
    cu = torch.tensor([0, 3], dtype=torch.int32)
    pt = torch.zeros((1, 2), dtype=torch.int32)
    return dict(k_cache=kc, v_cache=kc.clone(), k_scale=ks, v_scale=ks.clone(), cu=cu, pt=pt,
                lens=torch.tensor([3], dtype=torch.int32),
                q=torch.zeros((3, 4, 64), dtype=torch.bfloat16),
                kv=torch.zeros((3, 2, 64), dtype=torch.bfloat16))


def cache_args(t):
    return t["k_cache"], t["v_cache"], t["k_scale"], t["v_scale"]


@pytest.mark.parametrize("name,bad", [
    ("k_cache", lambda t: t.view(torch.uint8)), ("k_cache", lambda t: t[:, :, :32]),
    ("v_cache", lambda t: t[:3]), ("k_scale", lambda t: t.double()), ("v_scale", lambda t: t[:, :1]),
    ("cu", lambda t: t.long()), ("pt", lambda t: t.expand(2, 2)), ("lens", lambda t: t.expand(2)),
    ("kv", lambda t: t.float()), ("kv", lambda t: t[..., ::2]), ("q", lambda t: t[..., :32]),
])
def test_python_refuses_shapes_and_types(lib, name, bad):
    t = tensors()
    t[name] = bad(t[name])
    calls = [lambda: fa.fa_paged_kv_append(t["kv"], t["kv"], t["cu"], t["lens"], t["pt"],
                                           *cache_args(t)),
             lambda: fa.fa_paged_attn(t["q"], *cache_args(t), t["cu"], t["lens"], t["pt"])]
    for fn in calls if name not in ("kv", "q") else calls[:1] if name == "kv" else calls[1:]:
        with pytest.raises((TypeError, ValueError)):
            fn()


def test_python_refuses_tensors_that_are_not_on_the_gpu(lib):
    t = tensors()
    for fn in (lambda: fa.fa_paged_kv_append(t["kv"], t["kv"], t["cu"], t["lens"], t["pt"],
                                             *cache_args(t)),
               lambda: fa.fa_paged_attn(t["q"], *cache_args(t), t["cu"], t["lens"], t["pt"]),
               lambda: fa.fa_paged_kv_gather(*cache_args(t), t["cu"], t["pt"], 3),
               lambda: fa.fa_qk_norm_rope(t["q"], t["kv"], None, None)):
        with pytest.raises(ValueError, match="CUDA"):
            fn()


def test_python_refuses_inconsistent_norm_rope_calls(lib):
    t = tensors()
    q, k, tab = t["q"], t["kv"], torch.zeros((5, 64))
    pos = torch.zeros(3, dtype=torch.int32)
    for fn in (lambda: fa.fa_qk_norm_rope(None, None, pos, tab),
               lambda: fa.fa_qk_norm_rope(q, k[:2], pos, tab),
               lambda: fa.fa_qk_norm_rope(q, k, None, tab),
               lambda: fa.fa_qk_norm_rope(q, k, pos[:2], tab),
               lambda: fa.fa_qk_norm_rope(q, k, pos, tab, q_weight=torch.zeros(32))):
        with pytest.raises(ValueError):
            fn()


# ------------------------------------------------------------ work split
def walk(probe, q_lens, lens, hk, group, rows, causal, window, held, ctas):
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    arr = lambda x: (ctypes.c_int * len(x))(*x)  # noqa: E731
    most = 200000
    out = (ctypes.c_int * (8 * most))()
    n = probe.probe_walk(arr(cu), arr(lens), len(lens), cu[-1], hk, group, rows, causal, window,
                         held, ctas, most, out)
    assert n >= 0
    return [tuple(out[8 * i:8 * i + 8]) for i in range(n)]


def test_segments_cover_every_tile_once(probe):
    rng = random.Random(2)
    for trial in range(400):
        batch = rng.choice([1, 2, 5, 30])
        q_lens = [rng.choice([0, 1, 1, 2, 7, 40]) for _ in range(batch)]
        held = 64 * rng.randrange(1, 60)
        lens = [rng.choice([0, 1, 64, 127, 128, 129, rng.randrange(0, 4000), -3])
                for _ in range(batch)]
        hk, group, rows = rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 16, 40]), rng.choice([16, 64])
        causal, window = rng.randrange(2), rng.choice([-1, 0, 100, 1000])
        ctas = rng.choice([1, 2, 7, 152])
        segs = walk(probe, q_lens, lens, hk, group, rows, causal, window, held, ctas)
        want = {}
        for b, (n, ln) in enumerate(zip(q_lens, lens)):
            for h in range(hk):
                for t in range(-(-n * group // rows)):
                    i0, i1 = t * rows // group, (min((t + 1) * rows, n * group) - 1) // group
                    keys = min(max(ln, 0), held)
                    hi = min(keys, ln - n + i1 + 1) if causal else keys
                    lo = max(0, ln - n + i0 - window) if window >= 0 else 0
                    want[b, h, t] = (lo // 128, -(-hi // 128)) if hi > lo else None
        got = {}
        where = {}
        expect = {}
        for c, b, h, t, tile0, count, part_lo, unit_count in segs:
            if part_lo == 0:
                expect[b, h, t] = unit_count >> 16
                unit_count &= 65535
            assert count > 0 and 0 <= part_lo and part_lo + count <= unit_count
            where.setdefault((b, h, t), []).append(c)
            got.setdefault((b, h, t), []).append((tile0, count, part_lo, unit_count))
        assert set(got) == set(want)
        # A split unit's parts are in neighbouring CTAs, as many as announced.
        for key, cs in where.items():
            assert cs == list(range(cs[0], cs[0] + len(cs))) and len(cs) == expect[key]
        for key, parts in got.items():
            at = parts[0][0]
            assert parts[0][2] == 0
            for tile0, count, part_lo, unit_count in parts:
                assert tile0 == at and tile0 - parts[0][0] == part_lo
                at += count
            assert at - parts[0][0] == parts[0][3]
            if want[key] is None:
                assert parts[0][3] == 1
            else:
                assert (parts[0][0], at) == want[key]
        # At most a CTA's first and last segment hold part of a unit.
        for c in range(ctas):
            mine = [s for s in segs if s[0] == c]
            assert all(s[5] == s[7] & 65535 for s in mine[1:-1])


# ------------------------------------------------- strides that step nowhere
def varlen_strided(lib, q=(256, 64), k=(128, 64), v=(128, 64), Tq=5, Tk=5, H=4, Hk=2, d=64):
    return lib.fa_varlen_fwd_strided(P(0x1000), *q, P(0x2000), *k, P(0x3000), *v, P(0x4000),
                                     P(0x5000), 1, Tq, Tk, H, Hk, d, d, Tq, Tk, 0.125, 0, -1, -1,
                                     P(0x6000), None, None)


@pytest.mark.parametrize("row,head", [(64, 64), (8, 64), (0, 64), (-3, 64), (77, 72)])
def test_the_row_stride_of_one_row_is_not_read(lib, row, head):
    # A contiguous [heads, 1, dim] tensor turned round has the strides (dim,
    # dim), and they are as good as any.
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert norm_rope(lib, d=64, rot=64, T=1, qr=row, qh=head, kr=row, kh=head, qor=row, qoh=head,
                     kor=row, koh=head) in none
    assert append(lib, T=1, kr=row, kh=head, vr=row, vh=head) in none
    assert attn(lib, T=1, qr=row, qh=head) in none
    assert varlen_strided(lib, (row, head), (row, head), (row, head), 1, 1) in none
    # What is wrong with two rows stays wrong.
    assert norm_rope(lib, d=64, rot=64, T=2, qr=row, qh=head, kr=256) == INV
    assert append(lib, T=2, kr=row, kh=head) == INV and attn(lib, T=2, qr=row, qh=head) == INV
    assert varlen_strided(lib, (row, head)) == INV


@pytest.mark.parametrize("head", [1, 0, -64, 63, 2 ** 40])
def test_the_head_stride_of_one_head_is_not_read(lib, head):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert norm_rope(lib, d=64, rot=64, H=1, Hk=1, qr=64, qh=head, kr=72, kh=head, qor=64, qoh=head,
                     kor=64, koh=head) in none
    assert append(lib, Hk=1, kr=64, kh=head, vr=64, vh=head) in none
    assert attn(lib, H=1, Hk=1, qr=64, qh=head) in none
    assert varlen_strided(lib, (64, head), (64, head), (64, head), H=1, Hk=1) in none
    assert append(lib, Hk=1, T=1, kr=-1, kh=head, vr=3, vh=head) in none
    # With two heads it is.
    assert append(lib, kr=2 ** 37 - 8, kh=head) == INV
    assert append(lib, Hk=1, kr=56, kh=head) == INV      # rows that overlap


# -------------------------------------------------------------------- build
def test_the_build_sees_every_file_that_the_sources_include():
    deps = {os.path.realpath(p) for p in build_ext._deps()}
    todo, seen = list(build_ext._sources()), set()
    while todo:
        path = os.path.realpath(todo.pop())
        if path in seen:
            continue
        seen.add(path)
        with open(path) as f:
            for line in f:
                if line.startswith('#include "'):
                    todo.append(os.path.join(os.path.dirname(path), line.split('"')[1]))
    assert any(p.endswith("paged_index.h") for p in seen)
    assert seen <= deps, sorted(seen - deps)


def test_window_sizes_do_not_wrap():
    got = [fa._window(n) for n in (-2 ** 40, -2 ** 32 + 5, -2, -1, 0, 7, 2 ** 31 - 1, 2 ** 31,
                                   2 ** 32, 2 ** 32 + 5, 2 ** 64)]
    assert got == [-2, -2, -2, -1, 0, 7] + [2 ** 31 - 1] * 5


# ------------------------------------------- ranges and splits, row for row
def test_key_ranges_are_no_wider_than_what_the_rows_see(probe):
    rng = random.Random(3)
    for _ in range(4000):
        n = rng.randrange(1, 20)
        ln = rng.randrange(-5, 400)
        held = 64 * rng.randrange(1, 8)
        i0 = rng.randrange(0, n)
        i1 = rng.randrange(i0, n)
        causal, window = rng.randrange(2), rng.choice([-1, 0, 1, 70, 300])
        lo, hi = call(probe.probe_key_range, 2, i0, i1, n, ln, held, causal, window)
        seen = [j for j in range(min(max(ln, 0), held))
                if any((not causal or j <= ln - n + i) and (window < 0 or j >= ln - n + i - window)
                       for i in range(i0, i1 + 1))]
        assert (lo, hi) == (seen[0], seen[-1] + 1) if seen else lo == hi


@pytest.mark.parametrize("rows", [16, 32])
def test_splits_of_the_kernels_row_tiles(probe, rows):
    # Every key tile that a row tile needs is in one CTA's range, and no other
    # is; the ranges' costs differ by one at most.
    rng = random.Random(rows)
    for trial in range(150):
        batch = rng.choice([1, 3, 20])
        q_lens = [rng.choice([0, 1, 1, 5, 33, 200]) for _ in range(batch)]
        held = 64 * rng.randrange(1, 60)
        lens = [rng.choice([0, 1, 128, 129, rng.randrange(0, 4000), -3]) for _ in range(batch)]
        hk, group = rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 16, 40, 128])
        causal, window = rng.randrange(2), rng.choice([-1, 0, 100, 1000])
        ctas = rng.choice([1, 5, 152])
        segs = walk(probe, q_lens, lens, hk, group, rows, causal, window, held, ctas)
        want = set()
        cost = 0
        for b, (n, ln) in enumerate(zip(q_lens, lens)):
            for t in range(-(-n * group // rows)):
                i0, i1 = t * rows // group, min((t + 1) * rows, n * group) - 1
                lo, hi = call(probe.probe_key_range, 2, i0, i1 // group, n, ln, held, causal,
                              window)
                tiles = range(lo // 128, -(-hi // 128)) if hi > lo else [lo // 128]
                want |= {(b, h, t, j) for h in range(hk) for j in tiles}
                cost += hk * (7 + len(tiles))
        got = [(b, h, t, tile0 + i) for _, b, h, t, tile0, count, _, _ in segs for i in range(count)]
        assert len(got) == len(set(got)) and set(got) == want
        per_cta = [0] * ctas
        for s in segs:
            per_cta[s[0]] += s[5]
        assert max(per_cta) <= -(-cost // ctas)
