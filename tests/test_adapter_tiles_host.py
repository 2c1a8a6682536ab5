"""The adapter kernels' search for tiles, run on the CPU as the device runs it (adapter_tiles_host.cpp): every token
stands in exactly one tile, with its own adapter, and no tile names a token that there is not."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("tiles") / "adapter_tiles.so")
    r = subprocess.run(["g++", "-O2", "-U_FORTIFY_SOURCE", "-std=c++17", "-fPIC", "-shared", "-w", "-o", lib,
                        os.path.join(HERE, "adapter_tiles_host.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return C.CDLL(lib).tiles


def tiles(search, lens, slot, n, r=16, rank=None, scale=None, bm=0, starts=None):
    """[(slot, first token, rows, rank, scale, tokens)] of the blocks that have rows."""
    T, R = sum(lens), len(lens)
    i32 = lambda v: np.ascontiguousarray(v, np.int32)  # noqa: E731
    st, sl = i32(np.concatenate([[0], np.cumsum(lens)]) if starts is None else starts), i32(slot)
    rk = None if rank is None else i32(rank)
    sc = None if scale is None else np.ascontiguousarray(scale, np.float32)
    most = T + R + n + 2
    found, scales, tok = np.zeros((most, 4), np.int32), np.zeros(most, np.float32), np.zeros((most, 16), np.int32)
    at = lambda v: None if v is None else C.c_void_p(v.ctypes.data)  # noqa: E731
    blocks = search(T, R, n, r, at(st), at(sl), at(rk), at(sc), bm, most, at(found), at(scales), at(tok))
    assert blocks >= 0
    return [(*found[b].tolist(), float(scales[b]), tok[b, :found[b, 2]].tolist()) for b in range(blocks) if found[b, 2]]


def check(search, lens, slot, n, r=16, rank=None, scale=None, bm=0):
    T, owner = sum(lens), np.repeat(slot, lens)
    seen = np.zeros(T, int)
    for s, t0, count, rk, sc, tok in tiles(search, lens, slot, n, r, rank, scale, bm):
        tok = list(range(t0, t0 + count)) if bm else tok
        assert 1 <= count <= (bm or 16)
        assert all(0 <= t < T for t in tok), f"{len(lens)} requests: a tile of adapter {s} names {tok} of {T} tokens"
        seen[tok] += 1
        assert all((owner[t] if 0 <= owner[t] < n else -1) == s for t in tok)
        assert rk == (0 if s < 0 else min(max(rank[s], 0), r) if rank is not None else r)
        assert sc == (1.0 if s < 0 or scale is None else np.float32(scale[s]))
    assert (seen == 1).all(), f"{len(lens)} requests: tokens in no tile or in several"


RESIDUES = sorted({*range(32, 100), *range(100, 500, 23), 257, 479, 480, 481, 510, 511, 512})


@pytest.mark.parametrize("kind", ["ones", "ragged", "no adapter", "all adapters"])
def test_tiles_of_an_adapters_tokens(search, kind):
    for R in RESIDUES:
        lens, n = [1] * R, 2
        if kind == "ragged":
            lens = [(i * 7 + R) % 12 for i in range(R)]
        slot = [{"no adapter": -1, "all adapters": i % n}.get(kind, (i * i + i // 5) % 7 % 4 - 1) for i in range(R)]
        check(search, lens, slot, n)


def test_tiles_of_an_adapters_tokens_after_other_batches(search):
    """Shared memory still holds a longer batch's requests."""
    for R in (33, 40, 50, 90, 100, 257):
        check(search, [3] * 512, [i % 5 - 1 for i in range(512)], 5, rank=[0, 3, 8, 16, 40], scale=[0.5, 1, 2, 3, 4])
        check(search, [1] * R, [-1 if i % 7 == 6 else i % 2 for i in range(R)], 2, rank=[16, -3], scale=[2.0, 0.25])
        check(search, [i % 3 for i in range(R)], [-1 if i % 7 == 6 else 9 if i % 5 == 0 else i % 2 for i in range(R)], 2)


def test_tiles_of_an_adapters_tokens_with_wrong_starts(search):
    """Starts that do not ascend or leave the batch are cut to it: whatever is found lies in the batch."""
    for starts in ([0, 50, 20, 40], [-9, 10, 99, 40], [40, 30, 20, 10], [5, 2 ** 31 - 1, -2 ** 31, 40]):
        starts = (starts + [40] * 40)[:41]
        for *_, count, _, _, tok in tiles(search, [1] * 40, [i % 3 - 1 for i in range(40)], 2, starts=starts):
            assert all(0 <= t < 40 for t in tok)


@pytest.mark.parametrize("bm", [16, 32, 128])
def test_tiles_of_a_request(search, bm):
    for R in (1, 5, 63, 64, 65, 130):
        lens = [(i * 37 + R) % 150 for i in range(R)]
        check(search, lens, [i % 5 - 1 for i in range(R)], 3, r=24, rank=[24, 7, 90], scale=[1.0, 2.0, 0.5], bm=bm)
