"""The 256 x 256 matrix-product core (csrc/mma256.hpp) without a GPU.

Its loads go straight to LDS and its waits are counts, so what they rely on is
checked here: on a simulation of the issue order (what a phase reads has
landed; a region is refilled only after every wave has read it; across tiles
of any stage counts), and in the generated code of every kernel built on it
(four loads per read part, one vmcnt(8) and an lgkmcnt(0) before the barrier
that ends it, nothing but matrix instructions in the other parts, no spills).
"""
import re
import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
sys.path.insert(0, str(ROOT / "tests"))
from asm_check import kernel_bodies  # noqa: E402
from test_codegen import _hipcc  # noqa: E402


def wave_program(tiles):
    """One wave's events. tiles: stage counts. Events: ("load", region, tag),
    ("read", region, tag), ("wait", n), ("barrier",), with tag (tile, stage,
    half) or None for a load of nothing; region (operand and half, LDS stage)."""
    seq = []  # the loaded stages in order: every tile's, padded to pairs
    for t, n in enumerate(tiles):
        seq += [(t, s) if s < n else None for s in range(n + n % 2)]
    total = len(seq)
    at = lambda i: seq[i] if i < total else None
    ev = []

    def load(half, i):
        ev.append(("load", (half, i % 2), None if at(i) is None else (*at(i), half)))

    def read(half, i):
        ev.append(("read", (half, i % 2), None if at(i) is None else (*at(i), half)))

    for h in ("B0", "A0", "B1", "A1"):
        load(h, 0)
    for h in ("B0", "A0", "B1"):
        load(h, 1)
    ev += [("wait", 8), ("barrier",)]
    read("B0", 0)
    ev.append(("barrier",))
    for i in range(total):
        # phase X
        read("A0", i), read("B1", i), load("A1", i + 1), load("B0", i + 2)
        ev += [("wait", 8), ("barrier",), ("barrier",)]
        # phase Y
        read("A1", i), read("B0", i + 1), load("A0", i + 2), load("B1", i + 2)
        ev += [("wait", 8), ("barrier",), ("barrier",)]
    return ev


def check(tiles):
    """Runs two waves, one of each group (the second a barrier behind), through
    the program. A load may write its region from its issue on and has landed
    for certain only once its wave's wait allows at most the loads issued
    after it; a barrier makes that known to the other wave. Reads return before
    the barrier that ends their part."""
    prog = wave_program(tiles)
    first = [k for k, e in enumerate(prog) if e[0] == "barrier"][1]
    progs = [prog, prog[:first + 1] + [("barrier",)] + prog[first + 1:]]
    pc, pending = [0, 0], [[], []]   # pending: (region, tag), oldest first, two loads each
    landed = [{}, {}]                # this wave's share of a region that it knows to have landed
    known = {}                       # ... that both waves know
    reads_open = [set(), set()]      # regions whose reads may not have returned

    def run(w):
        while pc[w] < len(progs[w]):
            e = progs[w][pc[w]]
            pc[w] += 1
            if e[0] == "barrier":
                reads_open[w].clear()  # lgkmcnt(0) before it
                return True
            if e[0] == "wait":
                while 2 * len(pending[w]) > e[1]:
                    r, tag = pending[w].pop(0)
                    landed[w][r] = tag
            elif e[0] == "load":
                _, r, tag = e
                assert r not in reads_open[0] and r not in reads_open[1], (tiles, "refilled while read", e)
                pending[w].append((r, tag))
                landed[w].pop(r, None)
            else:
                _, r, tag = e
                for x in (0, 1):
                    assert all(p[0] != r for p in pending[x]), (tiles, "read while loading", e)
                    assert known.get((x, r), "?") == tag, (tiles, "read before known", e, known.get((x, r)))
                reads_open[w].add(r)
        return False

    while True:
        more = [run(0), run(1)]
        for x in (0, 1):
            for r in list(k for k in known if k[0] == x):
                if r[1] not in landed[x]:
                    known.pop(r)
            for r, tag in landed[x].items():
                known[(x, r)] = tag
        if not any(more):
            break
    assert pc[0] == len(progs[0])


@pytest.mark.parametrize("tiles", [[1], [2], [3], [4], [5], [16], [1, 1], [1, 2, 3], [2, 2, 2], [5, 1, 4, 1, 1, 7]])
def test_waits_and_refills(tiles):
    check(tiles)


def test_the_simulation_sees_a_short_wait(monkeypatch):
    """With one half-tile more left in flight the check fails."""
    real = wave_program

    def loose(tiles):
        return [("wait", 10) if e == ("wait", 8) else e for e in real(tiles)]
    monkeypatch.setattr(sys.modules[__name__], "wave_program", loose)
    with pytest.raises(AssertionError):
        check([4, 4])


@pytest.fixture(scope="module", params=["xent.hip", "int8.hip"])
def asm(request, tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    import importlib.util
    spec = importlib.util.spec_from_file_location("lmhead_build", ROOT / "lm_head_logits_amd" / "_build.py")
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    out = tmp_path_factory.mktemp("asm") / (request.param + ".s")
    cmd = [hipcc, *b.HIPCC_FLAGS, "-S", "--cuda-device-only", "-I", str(ROOT / "include"), "-o", str(out),
           str(ROOT / "lm_head_logits_amd" / "csrc" / request.param)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return request.param, out.read_text()


MM_KERNELS = {"xent.hip": ("xent_stats_kernel", "xent_grad_kernel", "xent_dhidden_kernel", "xent_dweight_kernel",
                           "xent_products_kernel"), "int8.hip": ("int8_tiled_kernel",)}


def test_generated_code(asm):
    src, text = asm
    seen = set()
    for name, (lines, labels) in kernel_bodies(text).items():
        which = [k for k in MM_KERNELS[src] if k in name]
        if not which:
            continue
        seen.add(which[0])
        assert not any(t.startswith("scratch_") for t in lines), f"{name}: spills"
        parts, cur = [], []  # the code between barriers, in its order in memory
        for t in lines:
            if t == "s_barrier":
                parts.append(cur)
                cur = []
            else:
                cur.append(t)
        parts.append(cur)
        products = 0
        for k, p in enumerate(parts):
            n_mfma = sum("v_mfma" in t for t in p)
            if not n_mfma:
                continue
            products += n_mfma
            # a part of matrix instructions reads and loads nothing
            assert not any(re.match(r"(ds_|buffer_|global_)", t) for t in p), (name, k)
        assert products % 128 == 0 and products > 0, name
        # every part that ends a phase's loads: vmcnt(8), then lgkmcnt(0), last before the barrier
        ends = [p for p in parts if p and any("vmcnt(8)" in t for t in p)]
        assert len(ends) >= 4, name
        for p in ends:
            waits = [t for t in p if t.startswith("s_waitcnt")]
            assert "vmcnt(8)" in waits[-2] or "vmcnt(8)" in waits[-1], name
            tail = p[max(i for i, t in enumerate(p) if "vmcnt(8)" in t):]
            assert not any(t.startswith("buffer_load") for t in tail), name
    assert seen == set(MM_KERNELS[src])
