"""Counted waits of the kernels outside the 256 x 256 core and the projection
(CPU: generated code): xent_outer_kernel, whose wait for the next columns of G
counts on sixteen stores behind their loads, and int8_stream_kernel, a ring
with the waits of csrc/ring.hpp's Schedule."""
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from asm_check import _VMCNT, kernel_bodies, lds_loads_with_pending_lds_ops
from test_ring_schedule import (_HEADER_RE, CSRC, ROOT, _flags, _hipcc, _loop_follows_schedule, _main_loop, _tokens,
                                schedules)  # noqa: F401  (schedules: a fixture)


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("waits")

    def build(name):
        out = d / f"{name}.s"
        r = subprocess.run([hipcc, *_flags(), "-S", "--cuda-device-only", "-I", str(ROOT / "include"), "-o", str(out),
                            str(CSRC / f"{name}.hip")], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return name, out.read_text()

    with ThreadPoolExecutor(2) as ex:
        return dict(ex.map(build, ("xent", "int8")))


def barriers_with_pending_lds_loads(lines, labels):
    """As in asm_check, with every state of every instruction followed: 0, or
    how many vector memory operations there are from the youngest direct-to-LDS
    load on (on a path where a store is skipped there are fewer, and vmcnt(k)
    retires less)."""
    bad, seen, work = set(), set(), [(0, 0)]
    while work:
        p, st = work.pop()
        while p < len(lines) and (p, st) not in seen:
            seen.add((p, st))
            t = lines[p]
            op = t.split()[0]
            if op.startswith("buffer_load") and t.endswith(" lds"):
                st = 1
            elif op.startswith(("buffer_", "global_", "scratch_", "flat_")) and st:
                st = min(st + 1, 64)
            if op == "s_waitcnt":
                w = _VMCNT.search(t)
                if w and st and int(w.group(1)) < st:
                    st = 0
            if op == "s_barrier" and st:
                bad.add(p)
            if op == "s_branch" or op.startswith("s_cbranch"):
                work.append((labels[t.split()[1]], st))
                if op == "s_branch":
                    break
            if op == "s_endpgm":
                break
            p += 1
    return sorted(bad)


def test_outer_kernel(asm):
    """No barrier is reached with a direct-to-LDS load possibly in flight, none
    is issued over an LDS operation in flight, and nothing spills (a spill's
    loads and stores would be counted by the waits)."""
    kernels = {k: v for k, v in kernel_bodies(asm["xent"]).items() if "xent_outer_kernel" in k}
    assert len(kernels) == 2
    for name, (lines, labels) in kernels.items():
        assert any(t.startswith("buffer_load") and t.endswith(" lds") for t in lines)
        assert any("vmcnt(16)" in t for t in lines), name
        assert not any(t.startswith("scratch_") for t in lines), name
        assert barriers_with_pending_lds_loads(lines, labels) == [], name
        assert lds_loads_with_pending_lds_ops(lines, labels) == [], name


def test_a_store_too_few_is_seen(asm):
    """With one of the stores taken out of the listing, or skipped by a branch,
    the check above finds the barrier behind the wait."""
    name, (lines, labels) = next((k, v) for k, v in kernel_bodies(asm["xent"]).items() if "xent_outer_kernel" in k)
    stores = [i for i, t in enumerate(lines) if t.startswith("buffer_store_dwordx4")]
    assert len(stores) % 16 == 0 and stores
    for i in (stores[0], stores[7], stores[15]):
        gone = lines[:i] + ["s_nop 0"] + lines[i + 1:]
        assert barriers_with_pending_lds_loads(gone, labels), i
        jump = lines[:i] + ["s_cbranch_execz .LBBx", lines[i]] + lines[i + 1:]
        moved = {k: v + (v > i) for k, v in labels.items()} | {".LBBx": i + 2}
        assert barriers_with_pending_lds_loads(jump, moved), i


_I8_RE = re.compile(r"int8_stream_kernelILi(\d+)ELi(\d+)E\w+?Li(\d+)ELi(\d+)EE")


def test_int8_ring(asm, schedules):  # noqa: F811
    text, checked, bad = asm["int8"], 0, []
    for name, (lines, labels) in kernel_bodies(text).items():
        m = _I8_RE.search(name)
        if not m:
            continue
        R, NB, NW, NSL = (int(x) for x in m.groups())
        HL = -(-16 * R * 8 // (64 * NW))
        assert ("bf16", NB, NSL, HL) in schedules, name
        period, table = schedules[("bf16", NB, NSL, HL)]
        assert not any(t.startswith("scratch_") for t in lines), name
        assert lds_loads_with_pending_lds_ops(lines, labels) == [], name
        start = text.index("\n" + name + ":")
        headers = set(_HEADER_RE.findall(text[start:text.index(".Lfunc_end", start)]))
        if not _loop_follows_schedule("bf16", NB, NSL, HL, period, table, lines, labels, headers):
            j, i = _main_loop(lines, labels, headers)
            bad.append(f"{name}: {_tokens(lines[j:i + 1])[:80]}")
        checked += 1
    assert not bad, "\n".join(bad)
    assert checked == 3 * (3 * 6 + 5)  # outputs; rows of blocks 1-3 with 1-4 column blocks, 4 with 1-3, two small shapes
