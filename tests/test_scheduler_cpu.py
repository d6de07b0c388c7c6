"""The scheduler of the persistent kernels (csrc/stream_common.cuh), compiled for the host: who owns
which unit when only some of a grid's CTA pairs run.  No GPU."""
import ctypes
import os
import subprocess

import pytest

from sparse_moe_layer_warp_b200 import build as b

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "scheduler_host.cu")


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("scheduler") / "libscheduler_host.so")
    flags = [f for f in b.NVCC_FLAGS if f != "-lineinfo"]
    subprocess.run([b._nvcc(), *flags, SRC, "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def call(counts, n_shared, T, k, bt, up_tiles, down_tiles, n, n_first, by_position=False):
        most = 1 << 16
        out, first = (ctypes.c_int * (8 * most))(), ctypes.c_int()
        got = lib.run_schedulers((ctypes.c_int * len(counts))(*counts), len(counts), n_shared, T,
                                 k, bt, up_tiles, down_tiles, n, n_first, int(by_position), out,
                                 most, ctypes.byref(first))
        assert got < most
        return [tuple(out[8 * i:8 * i + 8]) for i in range(got)], first.value

    return call


def _units(counts, n_shared, T, k, bt, up_tiles, down_tiles):
    """Every unit: (kind, group, weight tile, first token, rows, first row)."""
    groups, off = [], 0
    for g, n in enumerate(counts):
        groups.append((g, n, off))
        off += n
    if n_shared:
        groups.append((len(counts), T, T * k))
    return {(kind, g, mt, t, min(bt, n - t), off + t)
            for kind, tiles in ((0, up_tiles), (1, down_tiles)) for g, n, off in groups
            for mt in range(tiles) for t in range(0, n, bt)}


CASES = [
    dict(counts=[8, 8, 8, 8], n_shared=1, T=16, k=2, bt=8, up_tiles=3, down_tiles=2),
    dict(counts=[0, 130, 0, 0, 70, 0], n_shared=0, T=100, k=2, bt=32, up_tiles=5, down_tiles=8),
    dict(counts=[5] * 40 + [0] * 24, n_shared=1, T=100, k=2, bt=112, up_tiles=5, down_tiles=8),
    dict(counts=[300], n_shared=1, T=300, k=1, bt=112, up_tiles=44, down_tiles=8),
    dict(counts=[1, 0], n_shared=0, T=1, k=1, bt=32, up_tiles=1, down_tiles=1),
]
IDS = ["even", "empty groups", "one tile each", "dense", "one unit"]


@pytest.mark.parametrize("n,n_first", [(74, 74), (74, 73), (74, 20), (74, 1), (4, 2)])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_pairs_that_run_own_every_unit(run, case, n, n_first):
    """A pair leaves its down units only when the h that they read is there, so the pairs that run
    must own every up unit between them: the others may not start before they leave."""
    units, from_first = run(**case, n=n, n_first=n_first)
    assert len(units) == from_first  # those that start late find nothing
    assert {u[1:7] for u in units} == _units(**case) and len(units) == len(_units(**case))
    for me in range(n_first):  # each takes its up units first
        kinds = [u[1] for u in units if u[0] == me]
        assert kinds == sorted(kinds)
    # token tiles have numbers of their own, below the number that the scale blocks have room for
    tiles = {(u[2], u[4]): u[7] for u in units}
    assert len(set(tiles.values())) == len(tiles)
    rows = case["T"] * (case["k"] + case["n_shared"])
    assert max(tiles.values()) < rows // case["bt"] + len(case["counts"]) + case["n_shared"]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_positions_need_the_whole_grid(run, case):
    """Tickets by position (the cooperative launches): complete when all schedulers run, and not when
    one starts late and had units of its own -- which is why the CTA pairs draw theirs."""
    units, from_first = run(**case, n=74, n_first=74, by_position=True)
    assert {u[1:7] for u in units} == _units(**case) and len(units) == len(_units(**case))
    units, from_first = run(**case, n=74, n_first=1, by_position=True)
    assert {u[1:7] for u in units} == _units(**case)
    assert (from_first < len(units)) == (len(units) > 1)
