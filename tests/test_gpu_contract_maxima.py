"""The training and int8 operators at the shape contract's maxima, where a
launch passes 2^32 threads in one dimension."""
import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def test_quantiser_of_all_rows():
    """2^24 rows: every row's scale and codes, from the definition (elementary
    operations of torch on the device; the rows' maxima and quotients are exact
    or correctly rounded)."""
    R, H = 1 << 24, 32
    say(f"quantize_int8 R={R} H={H}")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(R, H, generator=g, device=DEV, dtype=torch.bfloat16)
    x[-1] = torch.arange(H, device=DEV) - 15
    q, s = L.quantize_int8(x)
    for r in range(0, R, 1 << 20):
        f = x[r:r + (1 << 20)].float()
        scale = f.abs().amax(1) / torch.full((1,), 127.0, device=DEV)
        assert torch.equal(s[r:r + (1 << 20)], scale)
        assert torch.equal(q[r:r + (1 << 20)].float(), torch.round(f / scale[:, None]))


@pytest.mark.parametrize("M,H", [((1 << 20) + 5, (1 << 14) + 32), ((1 << 20) + 3, 1 << 15)])
def test_lookup_of_many_rows(M, H):
    """More than 2^21 work-groups, with 32-bit and with 64-bit piece numbers."""
    V = 40
    say(f"embed M={M} H={H}")
    g = torch.Generator(device=DEV).manual_seed(2)
    W = torch.randn(V, H, generator=g, device=DEV).half()
    ids = torch.randint(-1, V + 1, (M,), generator=g, device=DEV, dtype=torch.int32)
    out = L.embed(ids, W, 0.5)
    Wz = torch.cat([W * 0.5, torch.zeros(1, H, dtype=W.dtype, device=DEV)])  # halves are exact
    at = torch.where((ids >= 0) & (ids < V), ids, torch.full_like(ids, V)).long()
    for r in range(0, M, 1 << 16):
        assert torch.equal(out[r:r + (1 << 16)], Wz[at[r:r + (1 << 16)]]), r
    del out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [0, 3, 9000])
def test_dense_gradient_of_2_35_elements(M):
    """A gradient of 64 GiB, filled behind either sort and alone."""
    V, H = 1 << 20, 1 << 15
    say(f"embed grad M={M} V={V} H={H}")
    ids = torch.tensor([V - 1, 0, V - 1, (1 << 19) + 1], device=DEV).repeat(M // 4 + 1)[:M]
    go = torch.ones(M, H, dtype=torch.bfloat16, device=DEV)
    gw = torch.empty(V, H, dtype=torch.bfloat16, device=DEV).fill_(7.0)  # what the call's own may reuse
    del gw
    gw = L.embed_backward(go, ids, V)
    want = torch.zeros(V, device=DEV).index_add_(0, ids, torch.ones(M, device=DEV)).to(torch.bfloat16)  # whole numbers
    for r in range(0, V, 1 << 15):
        part = gw[r:r + (1 << 15)]
        assert bool((part == want[r:r + (1 << 15), None]).all()), r
    del gw, part
    torch.cuda.empty_cache()


def test_hidden_gradient_of_more_than_2_32_elements():
    """The last kernel of the backward pass with more than 2^21 work-groups;
    rows from the beginning, either side of the 2^32nd element and the end,
    with the bounds of the smaller sizes' tests."""
    from test_gpu_xent import TINY16, U, close, reference
    M, H, V = (1 << 18) + 300, (1 << 14) + 32, 5
    say(f"xent M={M} H={H} V={V}")
    g = torch.Generator(device=DEV).manual_seed(3)
    h = torch.randn(M, H, generator=g, device=DEV, dtype=torch.bfloat16).mul_(0.25)
    W = torch.randn(V, H, generator=g, device=DEV).mul_(0.02).bfloat16()
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    gl = torch.full((M,), 2.0 ** -18, device=DEV)
    _, lse = L.xent_forward(h, W, y, 1.0)
    dh = L.xent_backward(gl, h, W, y, lse, 1.0, need_weight=False)[0]
    at = (1 << 32) // H
    for r0 in (0, at - 200, M - 400):
        rows = slice(r0, r0 + 400)
        r = reference(h[rows], W, None, y[rows], gl[rows], None, 1.0)
        t = r["dh_tol"]
        close(f"dh {r0}", dh[rows], r["dh"], t + r["h16"] * (r["dh"].abs() + t) * (1 + 4 * U) + 4 * U * r["dh"].abs()
              + TINY16["bf16"])
    del h, dh
    torch.cuda.empty_cache()


def test_row_reduction_of_many_rows():
    """Just over 2^22 rows, one work-group each in the combining kernel: every
    row as in a call of few rows, which the other tests check."""
    M, H, V = (1 << 22) + 5, 32, 40
    say(f"rowreduce M={M}")
    g = torch.Generator(device=DEV).manual_seed(4)
    few = torch.randn(61, H, generator=g, device=DEV).bfloat16()
    W = torch.randn(V, H, generator=g, device=DEV).bfloat16()
    at = torch.arange(M, device=DEV) % 61
    want = L.logits_rowreduce(few, W, 0.5)
    got = L.logits_rowreduce(few[at].contiguous(), W, 0.5)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b[at])
