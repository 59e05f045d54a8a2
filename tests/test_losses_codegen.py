"""The losses' matrix-product kernels in the generated code (CPU): as the
cross entropy's (tests/test_mma256_schedule.py, tests/test_stream_waits.py), and
launch shapes of the losses and the top logits at the contract's maxima."""
import re
import subprocess

import pytest

from asm_check import kernel_bodies, lds_loads_with_pending_lds_ops
from test_codegen import ROOT, _hipcc
from test_launch_shapes import SHAPES, calls, groups, taken  # noqa: F401  (calls: a fixture)
from test_stream_waits import barriers_with_pending_lds_loads

MM_KERNELS = ("loss_stats_kernel", "loss_grad_kernel", "loss_dhidden_kernel", "loss_dweight_kernel", "loss_products_kernel")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    import importlib.util
    spec = importlib.util.spec_from_file_location("lmhead_build", ROOT / "lm_head_logits_amd" / "_build.py")
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    d = tmp_path_factory.mktemp("asm")
    out = {}
    for name in ("losses", "topk"):
        cmd = [hipcc, *b.HIPCC_FLAGS, "-S", "--cuda-device-only", "-I", str(ROOT / "include"), "-o", str(d / f"{name}.s"),
               str(ROOT / "lm_head_logits_amd" / "csrc" / f"{name}.hip")]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        out[name] = (d / f"{name}.s").read_text()
    return out


def test_products(asm):
    """Nothing spills; the matrix parts read and load nothing; each read part
    ends with its counted wait."""
    seen = {}
    for name, (lines, labels) in kernel_bodies(asm["losses"]).items():
        which = [k for k in MM_KERNELS if k in name]
        if not which:
            continue
        seen[which[0]] = seen.get(which[0], 0) + 1
        assert not any(t.startswith("scratch_") for t in lines), f"{name}: spills"
        parts, cur = [], []
        for t in lines:
            if t == "s_barrier":
                parts.append(cur)
                cur = []
            else:
                cur.append(t)
        parts.append(cur)
        products = 0
        for k, p in enumerate(parts):
            n = sum("v_mfma" in t for t in p)
            products += n
            assert not n or not any(re.match(r"(ds_|buffer_|global_)", t) for t in p), (name, k)
        assert products % 128 == 0 and products > 0, name
        ends = [p for p in parts if any("vmcnt(8)" in t for t in p)]
        assert len(ends) >= 4, name
        for p in ends:
            waits = [t for t in p if t.startswith("s_waitcnt")]
            assert "vmcnt(8)" in waits[-2] or "vmcnt(8)" in waits[-1], name
            tail = p[max(i for i, t in enumerate(p) if "vmcnt(8)" in t):]
            assert not any(t.startswith("buffer_load") for t in tail), name
    # types times: teacher, target or kept; column sums or not; ...
    assert seen == dict(zip(MM_KERNELS, (6, 4, 2, 2, 2)))


def test_outer_kernel(asm):
    kernels = {k: v for k, v in kernel_bodies(asm["losses"]).items() if "loss_outer_kernel" in k}
    assert len(kernels) == 2
    for name, (lines, labels) in kernels.items():
        assert any("vmcnt(16)" in t for t in lines), name
        assert not any(t.startswith("scratch_") for t in lines), name
        assert barriers_with_pending_lds_loads(lines, labels) == [], name
        assert lds_loads_with_pending_lds_ops(lines, labels) == [], name


def test_no_kernel_spills(asm):
    for text in asm.values():
        for name, (lines, _) in kernel_bodies(text).items():
            assert not any(t.startswith("scratch_") for t in lines), name



@pytest.mark.parametrize("keep", [0, 1])
@pytest.mark.parametrize("M,H,V", SHAPES)
def test_losses_launch(calls, M, H, V, keep):  # noqa: F811
    head = ("p", M, H, "p", V, 1.0, "p", 1, 2.0)
    mem = ("p", "max", keep, "p", "max", None)
    taken(*calls("lmhead_policy_forward", *head, "p", 1, -100, "p", "p", "p", 0.2, 0.2, 0.1, "p", "p", *mem))
    taken(*calls("lmhead_preference_forward", *head, "p", 1, -100, "p", 1, max(1, M // 2), "p", 0.1, 0.0, 0.0, 0, "p", "p",
                 *mem))
    for K in (1, 1024):
        taken(*calls("lmhead_distill_forward", *head, "p", 1, "p", 0, K, "p", "p", *mem))
    for K in (0, 1, 1024):
        taken(*calls("lmhead_loss_backward", *head, K, "p", "p", "max", keep, "p", "p", "p", "p", "max", None))


@pytest.mark.parametrize("M,V", [(1, 1), (1, 1 << 20), (1023, 1 << 20), (1 << 22, 1 << 20), (1 << 24, 1 << 18)])
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_topk_launches(calls, M, V, dt):  # noqa: F811
    for K in (1, 64, 1024):
        if K <= V:
            st, launches = calls("lmhead_logits_topk", "p", M, V, V, dt, K, 1.0, "p", "p", "p", "p", "max", None)
            taken(st, launches)
            assert groups(launches[0]) >= M
