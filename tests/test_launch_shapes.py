"""Launch shapes at the shape contract's maxima, without a GPU.

A child process puts a recorder in the place of HIP's launch function (a
library of one C file, loaded before the HIP runtime, whose symbol it takes)
and calls the entry points with addresses that nothing reads. Every launch has
to be one that HIP takes: fewer than 2^32 threads per dimension, at most 1024
per work-group, no empty dimension.
"""
import json
import shutil
import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]

RECORDER = r"""
#include <stdint.h>
typedef struct { uint32_t x, y, z; } Dim3;
static uint64_t seen[4096][6];
static int n;
int hipLaunchKernel(const void *f, Dim3 g, Dim3 b, void **args, unsigned long lds, void *s) {
  uint64_t v[6] = {g.x, g.y, g.z, b.x, b.y, b.z};
  for (int i = 0; i < 6; ++i) if (n < 4096) seen[n][i] = v[i];
  ++n;
  for (int i = 0; i < 3; ++i) if (v[i] == 0 || v[3 + i] == 0 || v[i] * v[3 + i] >> 32) return 9;
  return v[3] * v[4] * v[5] > 1024 ? 9 : 0;
}
int hipGetDevice(int *d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int *v, int attr, int dev) { *v = 256; return 0; }
int recorded(uint64_t *out, int most) {
  int k = n < most ? n : most;
  for (int i = 0; i < 6 * k; ++i) out[i] = seen[i / 6][i % 6];
  k = n; n = 0;
  return k;
}
"""

CHILD = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from lm_head_logits_amd import _lib
lib = _lib.load()
P, MAX = 1 << 20, (1 << 63) - 1
buf = (ctypes.c_uint64 * (6 * 4096))()
for line in sys.stdin:
    name, args = json.loads(line)
    st = getattr(lib, name)(*[P if a == "p" else MAX if a == "max" else a for a in args])
    n = rec.recorded(buf, 4096)
    print(json.dumps([st, [list(buf[6 * i:6 * i + 6]) for i in range(min(n, 4096))]]), flush=True)
"""


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    d = tmp_path_factory.mktemp("recorder")
    (d / "rec.c").write_text(RECORDER)
    subprocess.run([cc, "-O1", "-shared", "-fPIC", "-o", str(d / "librec.so"), str(d / "rec.c")], check=True)
    p = subprocess.Popen([sys.executable, "-c", CHILD, str(d / "librec.so"), str(ROOT)], text=True,
                         stdin=subprocess.PIPE, stdout=subprocess.PIPE)

    def call(name, *args):
        p.stdin.write(json.dumps([name, args]) + "\n")
        p.stdin.flush()
        st, launches = json.loads(p.stdout.readline())
        return st, launches

    yield call
    p.stdin.close()
    p.wait(timeout=60)


def groups(launch):
    return launch[0] * launch[1] * launch[2]


def taken(st, launches):
    for x, y, z, bx, by, bz in launches:
        assert 0 < x * bx < 1 << 32 and 0 < y * by < 1 << 32 and 0 < z * bz < 1 << 32, (x, y, z, bx, by, bz)
        assert bx * by * bz <= 1024
    assert st == 0 and launches


def test_the_recorder_sees_launches(calls):
    st, launches = calls("lmhead_quantize_int8", "p", 5, 64, 1, "p", "p", None)
    taken(st, launches)
    assert launches == [[5, 1, 1, 256, 1, 1]]


@pytest.mark.parametrize("rows", [(1 << 21) - 1, (1 << 21) + 1, (1 << 24) - 1, 1 << 24])
@pytest.mark.parametrize("H", [32, 1 << 16])
def test_quantiser(calls, rows, H):
    st, launches = calls("lmhead_quantize_int8", "p", rows, H, 1, "p", "p", None)
    taken(st, launches)
    assert groups(launches[0]) >= rows


def test_group_numbering(tmp_path):
    """Every group 0 .. n - 1 has one place in the grid, in rows of 2^21, the last row begun."""
    src = tmp_path / "g.cpp"
    src.write_text(f'''#include "{ROOT}/lm_head_logits_amd/csrc/groups.hpp"
#include <cstdio>
#include <cstdlib>
int main(int, char **v) {{ auto g = lmhead::group_grid(atoll(v[1])); printf("%u %u", g.x, g.y); }}''')
    exe = tmp_path / "g"
    subprocess.run(["g++", "-std=c++17", "-o", str(exe), str(src)], check=True)
    for n in (1, 2, 1000, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, 5 << 21, (5 << 21) + 7, 1 << 24, 1 << 33):
        x, y = map(int, subprocess.run([str(exe), str(n)], capture_output=True, text=True, check=True).stdout.split())
        assert x * 1024 < 1 << 32 and y < 1 << 16 and x * y >= n > x * (y - 1)
        assert y == 1 or x == 1 << 21


# the contract's maxima (M 2^24, H 2^16, V 2^20, M V 2^42), and either side of
# what 2^32 threads in one dimension would cover
SHAPES = [(1, 1 << 16, 1 << 20), (8192, 1 << 16, 1 << 20), (8192, 1 << 15, 1 << 20), (8192, (1 << 15) - 32, 1 << 20),
          (1 << 24, 8192, 1), (1 << 24, 2048, 5), (1 << 24, 1 << 16, 1 << 18), (1 << 22, 1 << 16, 1 << 20)]


@pytest.mark.parametrize("M,H,V", SHAPES)
def test_embedding(calls, M, H, V):
    st, launches = calls("lmhead_embed", "p", 1, M, "p", V, H, 1, 1.0, "p", None)
    taken(st, launches)
    assert groups(launches[0]) * 256 * 4 >= M * H // 8


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("M,H,V", [(0, 1 << 16, 1 << 20), *SHAPES])
def test_embedding_gradient(calls, M, H, V, accumulate):
    st, launches = calls("lmhead_embed_backward", "p", 1, M, "p", V, H, 1, 1.0, -1, accumulate, "p", "p", "max", None)
    if M or not accumulate:
        taken(st, launches)


@pytest.mark.parametrize("M,H,V", SHAPES)
def test_cross_entropy(calls, M, H, V):
    taken(*calls("lmhead_xent_forward", "p", M, H, "p", V, 1.0, "p", 1, "p", 1, -100, "p", "p", "p", "max", None))
    taken(*calls("lmhead_xent_backward", "p", M, H, "p", V, 1.0, "p", 1, "p", 1, -100, "p", "p", "p", "p", "p", "p",
                 "p", "max", None))


# the other heads at sizes whose outputs (the row reduction's scratch) the
# card's memory holds: M V up to 2^37
@pytest.mark.parametrize("M,H,V", [(1, 1 << 16, 1 << 20), (1 << 17, 1 << 16, 1 << 20), (1 << 24, 8192, 1),
                                   ((1 << 22) + 1, 2048, 5), (1 << 24, 32, 1 << 13)])
def test_heads(calls, M, H, V):
    for name, *args in (("lmhead_logits_int8", "p", "p", M, H, "p", "p", V, 1.0, "p", 1, "p", None),
                        ("lmhead_logits", "p", M, H, "p", V, 1.0, "p", 1, "p", None),
                        ("lmhead_logits_nvfp4", "p", M, H, "p", "p", 1.0, V, 1.0, "p", "p", None),
                        ("lmhead_quantize_nvfp4", "p", V, H, "p", "p", "p", "p", "max", None),
                        ("lmhead_logits_rowreduce", "p", M, H, "p", V, 1.0, "p", 1, 1, None, "p", "p", "p", "p", "max",
                         None, -2)):
        taken(*calls(name, *args))
