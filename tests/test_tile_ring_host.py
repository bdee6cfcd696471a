"""The stages of the training attention's key and value tiles (csrc/tile_ring.h), compiled for the host with
g++.  A wait for a fill of a stage is by parity, which the fill two before meets too: whoever waits must have taken the
fill before, and the copies must fill a stage in order."""
import collections
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "bitwise_deterministic_shard_gb300", "csrc")


@pytest.fixture(scope="module")
def slots(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("ring") / "drv")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, os.path.join(HERE, "tile_ring_driver.cpp"), "-o", exe], check=True)
    calls = collections.defaultdict(dict)
    for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines():
        split, nst, tiles, value, n, stage, fill, last = map(int, line.split())
        calls[bool(split), nst, tiles][value, n] = stage, fill, bool(last)
    return calls


def _copies(tiles):
    """The order in which the tiles are copied: (value, tile)."""
    order = [(0, 0)] + ([(0, 1)] if tiles > 1 else [])
    for n in range(tiles):
        order += [(1, n)] + ([(0, n + 2)] if n + 2 < tiles else [])
    return order


def _taken(split, before, wait):
    """Whether a group that waits for a tile has taken another before it: its key tiles and its value tiles come in
    order, a value tile after its key tile, and key tile n only when the value tile three of the group's steps before
    is done (scores n after the softmax read n - 1, which it does after it wrote n - 2, once n - 3 was multiplied)."""
    step = 2 if split else 1
    if split and (before[1] - wait[1]) % 2:
        return False
    if before[0] == wait[0]:
        return before[1] < wait[1]
    return before[1] <= wait[1] if wait[0] else before[1] <= wait[1] - 3 * step


def _faults(split, nst, tiles, table):
    held, bad = {}, []
    for tile in _copies(tiles):
        stage, fill, last = table[tile]
        if not 0 <= stage < nst or fill != (held[stage][1] + 1 if stage in held else 0):
            bad.append(("order", tile))
        if stage in held:
            if held[stage][2]:
                bad.append(("last", tile))
            if not _taken(split, held[stage][0], tile):
                bad.append(("parity", tile))
        held[stage] = tile, fill, last
    return bad + [("last", h[0]) for h in held.values() if not h[2]]


def test_waits_by_parity_are_sound(slots):
    assert {k[:2] for k in slots} == {(False, 3), (False, 7), (True, 4), (True, 8)}
    for (split, nst, tiles), table in slots.items():
        assert len(table) == 2 * tiles
        assert not _faults(split, nst, tiles, table), (split, nst, tiles)


@pytest.mark.parametrize("nst, tiles", [(4, 4), (4, 9), (8, 12), (6, 9)])
def test_one_ring_for_two_groups_is_found_unsound(nst, tiles):
    """One ring in the order of the copies, where each group takes every other tile: the second group's first value
    tile follows the first group's key tile."""
    order = _copies(tiles)
    table = {t: (k % nst, k // nst, k + nst >= len(order)) for k, t in enumerate(order)}
    assert any(kind == "parity" for kind, _ in _faults(True, nst, tiles, table))
