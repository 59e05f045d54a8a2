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
