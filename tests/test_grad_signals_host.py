"""The signals between the warps of the distillation gradient's pipeline,
explored state by state on the CPU for one CTA: whatever the order of the warps'
steps and of the copies' arrivals, no warp uses a slice before its row's copy is
there or after another row's has begun, no barrier is signalled again before all
have passed it, and every row is finished.

The slices and the copies' mbarriers are the library's (grad_signals.cuh,
compiled for the host).  A wait for an mbarrier follows the hardware's rule: it
returns when the phase in progress has another parity than the one asked for.
The exchange of a cluster only delays warps B, which the exploration does too."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("shim") / "libgrad_signals.so")
    cmd = [nvcc, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-gencode", "arch=compute_103a,code=sm_103a",
           f"-I{os.path.join(ROOT, 'verify_dspark_markov_gb300', 'csrc')}",
           os.path.join(ROOT, "tests", "grad_signals_shim.cu"), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    return lib.grad_slice_of, lib.grad_full_of, lib.grad_full_parity


class Fault(Exception):
    pass


def programs(rows):
    """The warps' steps, in the kernel's order; a group of workers and a pair of
    warps of one role take the rows of one parity."""
    def sync(bar, n):
        return [("arrive", bar, n), ("wait", bar, n)]
    every = []
    for own in (0, 1):
        a, w, b, c = [], [], [], []
        for n in range(own, rows, 2):
            a += [("passed", n - 2)] if n > 1 else []
            a += [("full", n), ("use", n), ("arrive", "ready", n), ("arrive", "entries", n)]
            w += [*sync("ready", n), ("use", n), ("arrive", "sums", n), *sync("scalars", n), ("use", n),
                  ("arrive", "stored", n)]
            b += [*sync("entries", n), *sync("sums", n), ("arrive", "scalars", n)]
            c += [*sync("scalars", n), ("pass", n), *sync("stored", n)]
        every += [a, w, b, c]
    d = [("copy", n) for n in range(min(3, rows))]
    for n in range(rows):
        d += sync("stored", n) + ([("copy", n + 3)] if n + 3 < rows else [])
    return every + [d]


def model(rows, masked, slice_of, full_of, full_parity):
    """The first state, and the successors of a state (none once every row is finished)."""
    progs = programs(rows)
    parties = {}  # (barrier, row) -> the (program, step) of everyone who takes part
    at_step = {}
    for i, prog in enumerate(progs):
        for k, step in enumerate(prog):
            if step[0] == "arrive":
                parties.setdefault(step[1:], []).append((i, k))
            at_step[step] = (i, k)
    copies = [at_step["copy", n] for n in range(rows)]
    passes = [[at_step["pass", n] for n in range(own, rows, 2)] for own in (0, 1)]
    same_full = [[m for m in range(rows) if full_of(m) == full_of(n)] for n in range(rows)]
    same_slice = [[m for m in range(rows) if slice_of(m) == slice_of(n)] for n in range(rows)]
    parity = [full_parity(n) for n in range(rows)]

    def issued(pc, among):
        return [m for m in among if pc[copies[m][0]] > copies[m][1]]

    def phases(landed, begun):
        """The completed phases of an mbarrier of which these rows' copies have begun."""
        return sum(landed >> m & 1 for m in begun)

    def passed(pc, own):
        return sum(pc[i] > k for i, k in passes[own])

    def steps(pc, landed):
        for n in range(rows):
            i, k = copies[n]
            if pc[i] > k and not landed >> n & 1:
                yield pc, landed | 1 << n  # the copy arrives
        for i, prog in enumerate(progs):
            if pc[i] == len(prog):
                continue
            step, now = prog[pc[i]], landed
            kind, n = step[0], step[-1]
            if kind == "arrive":
                if any(pc[j] <= k for j, k in parties.get((step[1], n - 2), ())):
                    raise Fault(f"{step[1]}({n}) signalled before all have signalled {step[1]}({n - 2})")
            elif kind == "wait":
                continue
            elif kind == "passed":
                if passed(pc, n & 1) & 1 == n // 2 & 1:
                    continue
            elif kind == "full":
                if phases(landed, issued(pc, same_full[n])) & 1 == parity[n]:
                    continue
            elif kind == "use":
                begun = issued(pc, same_slice[n])
                if begun[-1:] != [n]:
                    raise Fault(f"row {n} takes its slice before its copy is issued")
                if any(not landed >> m & 1 for m in begun):
                    raise Fault(f"row {n} takes a slice that a copy is landing in")
            elif kind == "copy":
                begun = issued(pc, same_full[n])
                if phases(landed, begun) < len(begun):
                    raise Fault(f"row {n} arrives on a barrier whose phase is in progress")
                if masked[n]:
                    now = landed | 1 << n  # an arrival alone
            yield pc[:i] + (pc[i] + 1,) + pc[i + 1:], now

    def settle(state):
        """What a passed wait adds to a state changes nothing for the others: waits are passed at once."""
        pc, landed = state
        moved = True
        while moved:
            moved = False
            for i, prog in enumerate(progs):
                if pc[i] < len(prog) and prog[pc[i]][0] == "wait" and \
                        all(pc[j] > k for j, k in parties[prog[pc[i]][1:]]):
                    pc = pc[:i] + (pc[i] + 1,) + pc[i + 1:]
                    moved = True
        return pc, landed

    def successors(state):
        nexts = [settle(s) for s in steps(*state)]
        if not nexts and any(k < len(p) for k, p in zip(state[0], progs)):
            raise Fault("no warp can go on")
        return nexts

    return settle(((0,) * len(progs), 0)), successors


def explore(*args):
    """Every state; their number, or a Fault."""
    start, successors = model(*args)
    seen, todo = {start}, [start]
    while todo:
        for s in successors(todo.pop()):
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


def walk(rng, *args):
    """One schedule."""
    state, successors = model(*args)
    while nexts := successors(state):
        state = rng.choice(nexts[:rng.randint(1, len(nexts))])


NONE, ONE, SOME, MOST = [0] * 7, [0, 1, 0, 0, 0, 0, 0], [0, 1, 1, 0, 1, 0, 0], [1, 1, 1, 0, 1, 0, 0]


@pytest.mark.parametrize("masked", [NONE, ONE, SOME, MOST])
def test_every_order_of_seven_rows(library, masked):
    assert explore(7, masked, *library) > 10_000


def test_random_orders_of_many_rows(library):
    for seed in range(200):
        rng = random.Random(seed)
        rows = rng.randint(8, 24)
        walk(rng, rows, [rng.random() < 0.5 for _ in range(rows)], *library)


@pytest.mark.parametrize("masked", [NONE, ONE, MOST])
def test_a_barrier_to_a_slice_would_be_found(masked):
    """The exploration sees the fault of one mbarrier to a slice, whose phases
    two warps wait for in turn."""
    with pytest.raises(Fault):
        explore(7, masked, lambda n: n % 3, lambda n: n % 3, lambda n: n // 3 & 1)
