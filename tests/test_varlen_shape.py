"""The packed forward's split over a cluster under sinks and trees: the key tiles that it
counts an item to have (CPU), and outputs where long sinks stand before a short window
(GPU, against the plain fp64 form)."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("probe") / "varlen_shape.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-o", so,
                    os.path.join(HERE, "probes", "varlen_shape_probe.cpp")], check=True)
    f = ctypes.CDLL(so).probe_item_key_tiles
    f.restype = ctypes.c_longlong
    f.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 5 + [ctypes.c_longlong]
    return f


def walked(lq, lk, causal, wl, wr, sinks, tree):
    """Tiles of 128 keys of which some key is seen by one of the lq rows."""
    seen = set()
    for i in (0, lq - 1):  # (the outermost rows' windows; those between lie between)
        at = lk - lq + i
        lo = at - wl if wl >= 0 else 0
        hi = lk if tree or (wr < 0 and not causal) else at + 1 + (0 if causal else wr)
        seen |= {(max(lo, 0), min(hi, lk))}
    lo, hi = min(a for a, _ in seen), max(b for _, b in seen)
    keys = set(range(lo // 128, -(-hi // 128)))
    return len(keys | set(range(-(-min(sinks, lo) // 128))))


def test_an_item_has_about_the_tiles_that_are_counted(tiles):
    rng = random.Random(5)
    for _ in range(3000):
        lk = rng.choice([300, 5000, 16384, 100000])
        lq = min(lk, rng.choice([1, 2, 64, 200, 256]))
        causal, wr = rng.choice([(1, -1), (0, -1), (0, 0), (0, 300)])
        wl = rng.choice([-1, 0, 100, 128, 4000, 2 ** 31 - 1])
        sinks = rng.choice([0, 1, 4, 128, 129, 8192, 12000, 2 ** 31 - 1])
        tree = rng.random() < 0.3
        got = tiles(lk, lk, causal, wl, wr, sinks, lq if tree else 0)
        want = walked(lq, lk, causal, wl, -1 if tree else wr, sinks, tree)
        if wl >= 0 and not (tree or causal or wr >= 0):
            # (A window that is open to the right counts as all keys: the first rows of a
            # sequence see that many.)
            assert got == -(-lk // 128) >= want
            continue
        # (256 rows are counted, whatever the sequence has, and ends inside tiles.)
        assert want - 2 <= got <= want + 5, (lq, lk, causal, wl, wr, sinks, tree, got, want)


def test_without_sinks_or_a_tree_it_is_keys_or_window(tiles):
    for lk in (1, 127, 128, 129, 5000, 2 ** 31 - 1):
        for causal, wl, wr in ((0, -1, -1), (1, -1, -1), (0, -1, 5), (1, 0, -1), (1, 100, -1),
                               (0, 100, -1), (0, 100, 300), (0, 2 ** 31 - 1, 2 ** 31 - 1)):
            keys = lk
            if wl >= 0 and (causal or wr >= 0):
                keys = min(lk, wl + (0 if causal else wr) + 256)
            assert tiles(lk, 0, causal, wl, wr, 0, 0) == -(-keys // 128)


def test_long_sinks_before_a_short_window_are_counted(tiles):
    assert tiles(16384, 16384, 1, 128, -1, 8192, 0) >= 64    # 3 without the sinks
    # A tree does not look at causal.
    for causal in (0, 1):
        assert tiles(16384, 16384, causal, 256, -1, 0, 64) == 3
        assert tiles(16384, 16384, causal, 256, -1, 8192, 64) == 67
        assert tiles(16384, 16384, causal, -1, -1, 0, 64) == 128


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("n,wl,sinks", [(1, 128, 8192), (64, 100, 12000), (200, 0, 16000)])
def test_long_sinks_before_a_short_window(cuda_device, d, dv, n, wl, sinks):
    from test_gpu_masked import check_packed
    check_packed([n], [16384], 2, 2, d, dv, wl=wl, sinks=sinks, seed=n + d)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("wl,sinks", [(256, 0), (256, 8192), (30, 130)])
def test_trees_whether_causal_is_given_or_not(cuda_device, causal, wl, sinks):
    from test_gpu_masked import check_packed, trees_of
    check_packed([64, 9], [16384, 700], 4, 2, 128, causal=causal, wl=wl, sinks=sinks,
                 trees=trees_of([64, 9], 11), seed=wl)
