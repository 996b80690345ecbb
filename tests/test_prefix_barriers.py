"""The shared-prefix kernel's roles and barriers, walked through in every order.

The model has the kernel's roles (the keys' and values' warps, two streams of
softmax warps, the MMA thread and the tensor cores behind it) with the
kernel's barriers, whose numbers and parities come from prefix_barriers.h
itself, compiled here.  All interleavings are visited: no role may be left
waiting, and what a role reads must be of its own tile.  CPU only."""
import ctypes
import os
import subprocess

import pytest

from fp16_tensor_core_gb300 import build as dg_build

EVENTS = ("keys", "values", "scores", "weights", "output", "factors")


@pytest.fixture(scope="module")
def phase(tmp_path_factory):
    """phase[event](j) -> (barrier, parity) of the header's functions; slots."""
    where = tmp_path_factory.mktemp("barriers")
    source = where / "probe.cpp"
    source.write_text('#include "prefix_barriers.h"\nextern "C" {\n' + "".join(
        f"int bar_{e}(int j) {{ return dg::prefix::{e}(j).barrier; }}\n"
        f"int parity_{e}(int j) {{ return (int)dg::prefix::{e}(j).parity; }}\n" for e in EVENTS) +
        "int slot(int j) { return dg::prefix::factor_slot(j); }\n"
        "int slots() { return dg::prefix::kFactorSlots; }\nint barriers() { return dg::prefix::kBarriers; }\n}\n")
    lib = where / "probe.so"
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", dg_build.CSRC, str(source), "-o", str(lib)], check=True)
    L = ctypes.CDLL(os.fspath(lib))
    table = {e: (lambda j, b=getattr(L, "bar_" + e), p=getattr(L, "parity_" + e): (b(j), p(j))) for e in EVENTS}
    table["slot"], table["slots"], table["barriers"] = L.slot, L.slots(), L.barriers()
    return table


def programs(phase, tiles, softmax_warps, softmax_waits_for="factors"):
    """Each role as a list of steps:
    ("wait", event, j), ("arrive", event, j), ("write", memory, slot, j),
    ("read", memory, slot, j), ("issue", product, j)."""
    slot = phase["slot"]
    key, value, mma = [], [], []
    for j in range(tiles):
        if j >= 2:
            key.append(("wait", "scores", j - 2))
            value.append(("wait", "output", j - 2))
        key += [("write", "K", j & 1, j), ("write", "F", slot(j), j), ("arrive", "keys", j), ("arrive", "factors", j)]
        value += [("write", "V", j & 1, j), ("arrive", "values", j)]
    for j in range(min(2, tiles)):
        mma += [("wait", "keys", j), ("issue", "scores", j)]
    for j in range(tiles):
        mma += [("wait", "values", j), ("wait", "weights", j), ("issue", "output", j)]
        if j + 2 < tiles:
            mma += [("wait", "keys", j + 2), ("wait", "output", j), ("issue", "scores", j + 2)]
    roles = [key, value, mma]
    for b, warps in enumerate(softmax_warps):
        one = []
        for j in range(b, tiles, 2):
            one += [("wait", softmax_waits_for, j), ("wait", "scores", j), ("read", "S", b, j), ("read", "F", slot(j), j)]
            if j >= 2:
                one.append(("wait", "output", j - 2))   # a reference that moved
            one.append(("arrive", "weights", j))
        if tiles > b:
            one.append(("wait", "output", tiles - 1 - ((tiles - 1 - b) & 1)))
        roles += [one] * warps
    return roles


def explore(phase, tiles, softmax_warps=(2, 1), **kw):
    """Every state that can be reached; returns those where nothing moves
    though a role is not done.  Raises when a role reads another tile."""
    roles = programs(phase, tiles, softmax_warps, **kw)
    need = [1] * phase["barriers"]
    for b, warps in enumerate(softmax_warps):
        need[phase["weights"](b)[0]] = warps

    def arrive(bars, event, j):
        at = phase[event](j)[0]
        n, pending = bars[at]
        pending += 1
        bars[at] = (n + 1, 0) if pending == need[at] else (n, pending)

    # memories: K[2], V[2], factors, S[2] (scores or weights), by the tile they hold
    cells = [("K", 0), ("K", 1), ("V", 0), ("V", 1), ("S", 0), ("S", 1)] + [("F", i) for i in range(phase["slots"])]
    index = {c: i for i, c in enumerate(cells)}
    start = ((0,) * len(roles), (), ((0, 0),) * phase["barriers"], (-1,) * len(cells))
    seen, todo, stuck = {start}, [start], []
    while todo:
        state = todo.pop()
        pcs, queue, bars, held = state
        after = []
        for r, role in enumerate(roles):
            if pcs[r] == len(role):
                continue
            what, name, *rest = role[pcs[r]]
            new_queue, new_bars, new_held = queue, bars, held
            if what == "wait":
                at, parity = phase[name](rest[0])
                if bars[at][0] & 1 == parity:           # the phase of that parity is the current one
                    continue
            elif what == "arrive":
                new_bars = list(bars)
                arrive(new_bars, name, rest[0])
            elif what == "write":
                new_held = list(held)
                new_held[index[name, rest[0]]] = rest[1]
            elif what == "read":
                assert held[index[name, rest[0]]] == rest[1], (role[pcs[r]], held)
            else:
                new_queue = queue + ((name, rest[0]),)
            after.append((pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], new_queue, tuple(new_bars), tuple(new_held)))
        if queue:   # the tensor cores finish the oldest product
            (name, j), b = queue[0], queue[0][1] & 1
            new_bars, new_held = list(bars), list(held)
            if name == "scores":
                assert held[index["K", b]] == j, (queue[0], held)
                new_held[index["S", b]] = j
            else:
                assert held[index["V", b]] == j and held[index["S", b]] == j, (queue[0], held)
            arrive(new_bars, name, j)
            after.append((pcs, queue[1:], tuple(new_bars), tuple(new_held)))
        if not after and any(pc < len(role) for pc, role in zip(pcs, roles)):
            stuck.append(pcs)
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return stuck


@pytest.mark.parametrize("tiles,softmax_warps", [(1, (2, 2)), (2, (2, 2)), (3, (2, 2)), (4, (2, 1)), (5, (2, 1)), (9, (1, 1))])
def test_no_order_leaves_a_role_waiting(phase, tiles, softmax_warps):
    assert explore(phase, tiles, softmax_warps) == []


def test_the_walk_finds_a_phase_that_passes_unseen(phase):
    """A softmax that waits for the keys' barrier, as the MMA thread does,
    can be late by a phase: the keys of tile j + 2 need only the product of
    tile j."""
    assert explore(phase, 3, softmax_waits_for="keys")


def test_barriers_do_not_overlap(phase):
    used = [phase[e](j)[0] for e in EVENTS[:5] for j in (0, 1)] + [phase["factors"](j)[0] for j in range(phase["slots"])]
    assert len(set(used)) == len(used) and max(used) < phase["barriers"]
