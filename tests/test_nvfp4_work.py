"""How work over caches held in 4 bits is counted and which way it goes, compiled
for the host."""
import ctypes
import os
import random
import subprocess

import pytest

from sparse_attention_indexer_logits_gb300 import _build


@pytest.fixture(scope="module")
def W(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("work") / "nvfp4_work.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "nvfp4_work.cu")
    subprocess.run([_build._nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-shared", "-Xcompiler", "-fPIC", "-gencode",
                    "arch=compute_103a,code=sm_103a", "-I", _build.CSRC, "-I", _build.INCLUDE, src, "-o", so],
                   check=True, capture_output=True, text=True)
    lib, i64 = ctypes.CDLL(so), ctypes.c_longlong
    lib.items.restype = i64
    lib.items.argtypes = [i64, i64, ctypes.c_int, ctypes.c_int]
    lib.large_items.argtypes = [i64, i64, ctypes.c_int]
    lib.by_tiles.argtypes = [i64, i64, ctypes.c_int, ctypes.c_int]
    lib.lists_by_tiles.argtypes = [i64] + [ctypes.c_int] * 4
    return lib


@pytest.mark.parametrize("n", [-2 ** 31, -1, 0, 1, 63, 64, 65, 5000, 2 ** 31 - 129, 2 ** 31 - 65, 2 ** 31 - 64, 2 ** 31 - 63,
                               2 ** 31 - 1])
def test_blocks_of_any_length(W, n):
    assert W.blocks(n) == max(0, (n + 63) // 64)


def items(tokens, batch, group, rows):
    """By the definition: every request's tokens `rows // group` at a time, or a
    token's heads in `ceil(group / rows)` parts."""
    count = 0
    for b in range(batch):
        n = tokens // batch + (b < tokens % batch)
        for t0 in range(0, n, max(1, rows // group)):
            count += len(range(0, group, rows)) if group > rows else 1
    return count


def test_items(W):
    r = random.Random(1)
    for _ in range(2000):
        tokens, batch, group = r.randint(1, 300), r.randint(1, 70), r.choice([1, 2, 3, 5, 7, 8, 9, 12, 16, 17, 20, 33, 64, 300])
        for rows in (8, 16):
            assert W.items(tokens, batch, group, rows) == items(tokens, batch, group, rows)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 20, 32])
@pytest.mark.parametrize("batch", [16, 64, 1000])
@pytest.mark.parametrize("more", [1, 2])
def test_a_few_more_tokens_keep_the_way(W, group, batch, more):
    """A decode step of single tokens, and with a second token for one or two of its requests."""
    heads = 8 * group
    assert not W.by_tiles(batch, batch, heads, group) and not W.by_tiles(batch + more, batch, heads, group)
    assert W.large_items(batch, batch, group) == W.large_items(batch + more, batch, group) == (group > 8)


def test_equal_batches(W):
    """Items of 16 for more than 8 rows, tiles for more than 32."""
    for group in range(1, 200):
        for q in (1, 2, 3, 4, 5, 8, 30):
            tiles = q * group > 32 and group <= 128
            assert W.by_tiles(64 * q, 64, 8 * group, group) == tiles
            if not tiles:
                assert W.large_items(64 * q, 64, group) == (q * group > 8)


def test_unequal_batches(W):
    """Where a part of the requests has one more token: items of 16 once they are less
    than three quarters of those of 8, tiles past 19/8 items a request and where the
    longer ones have more than 32 rows."""
    assert [W.large_items(n, 64, 8) for n in (64, 85, 86, 100)] == [0, 0, 1, 1]
    assert [W.by_tiles(n, 64, 160, 20) for n in (64, 65, 76, 77, 100)] == [0, 0, 0, 1, 1]
    assert [W.by_tiles(n, 64, 96, 12) for n in (64, 100, 128, 152, 153)] == [0, 0, 0, 0, 1]
    assert [W.by_tiles(n, 64, 48, 6) for n in (280, 320, 321)] == [0, 0, 1]


def test_calls_of_few_rows(W):
    """Fewer than 128 in all go by warps."""
    assert [W.by_tiles(n, 1, 64, 64) for n in (1, 2)] == [0, 1]
    assert [W.by_tiles(n, 3, 40, 40) for n in (3, 4)] == [0, 1]
    assert [W.by_tiles(n, 1, 1, 1) for n in (127, 128)] == [0, 1]


def test_lists(W):
    lists = lambda n, heads, group, k: W.lists_by_tiles(n, heads, group, k, 152)  # noqa: E731
    assert [lists(64, 64, 64, k) for k in (500, 1500, 2048)] == [0, 0, 1]
    assert [lists(n, 64, 64, 2048) for n in (57, 58)] == [0, 1]
    assert [lists(1000, g, g, 2048) for g in (1, 8, 32, 33, 128, 129, 300)] == [0, 0, 0, 1, 1, 0, 0]
    assert lists(10 ** 6, 128, 64, 2 ** 31 - 256) == 1
