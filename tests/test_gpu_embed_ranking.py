"""The embedding gradient's ranking of up to 8192 positions and its border to
the radix sort: every wave's share of the positions, ids repeated across the
waves' and the work-groups' borders, dense and added to a gradient."""
import pytest
import torch

import lm_head_logits_amd as L
from gpu_util import DEV, say
from test_gpu_embed import check_grad, table, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("M", [64, 65, 511, 512, 513, 2047, 2049, 4100, 8191, 8192, 8193])
@pytest.mark.parametrize("how", ["strided", "few", "padded", "outside"])
def test_every_share_counts(M, how, added):
    V, H = 700, 64
    say(f"embed ranking M={M} {how} added={added}")
    if how == "strided":  # one id every 64 positions, and 63 others in between: all shares hold all ids
        ids = (torch.arange(M, device=DEV) * 37) % 64 + 300
    elif how == "few":    # three ids in runs of 100
        ids = (torch.arange(M, device=DEV) // 100) % 3 * 349
    else:
        ids = tokens(M, M, V, how)
    go = table(M + 1, M, H, "bf16")
    base = table(M + 2, V, H, "bf16") if added else None
    got = check_grad(go, ids, V, 0.5, base=base)
    again = L.embed_backward(go, ids, V, 0.5, grad_weight=None if base is None else base.clone())
    assert torch.equal(got, again)


@pytest.mark.parametrize("M", [513, 4100, 8192, 8193])
def test_order_is_that_of_positions(M):
    """The sum of one id's rows in ascending position, over the whole length:
    2^25 first and -2^25 last swallow 1s between them one by one within a tile,
    and what a tile holds alone is exact, so the result is known."""
    V, H = 5, 32
    say("embed ranking order", M)
    go = torch.zeros(M, H, dtype=torch.bfloat16, device=DEV)
    go[0], go[1], go[2] = 2.0 ** 25, 1.0, -2.0 ** 25   # 0 in this order, 1 in any that joins the large ones first
    go[M - 3], go[M - 2], go[M - 1] = 1.0, 2.0, 4.0
    ids = torch.full((M,), 3, device=DEV)
    for gw, want in ((None, 7.0), (torch.ones(V, H, dtype=torch.bfloat16, device=DEV), 8.0)):
        out = L.embed_backward(go, ids, V, grad_weight=gw)
        assert bool((out[3] == want).all())


# a table large enough for its fill to hide the ranking of 16384 positions; one
# position more and a smaller table take the radix sort
@pytest.mark.parametrize("M,V,H", [(8192, 120000, 2080), (16384, 240000, 2080), (16385, 240000, 2080),
                                   (16384, 235000, 2080), (5120, 75000, 2080), (5121, 70000, 2080)])
def test_large_tables(M, V, H):
    say(f"embed ranking M={M} V={V} H={H}")
    ids = tokens(M, M, V, "padded", torch.int32)
    go = table(M + 1, M, H, "f16") * 0.01
    for base in (None, table(M + 2, V, H, "f16")):
        got = check_grad(go, ids, V, 0.5, base=base)
        assert torch.equal(got, L.embed_backward(go, ids, V, 0.5, grad_weight=None if base is None else base.clone()))
        del got
    torch.cuda.empty_cache()


def test_both_sorts_give_the_same_bits():
    """The sums' order is that of (id, position), whichever sort found it."""
    M, H = 3000, 64
    ids = tokens(5, M, 600, "padded")
    go = table(6, M, H, "bf16")
    ranked = L.embed_backward(go, ids, 600, grad_weight=torch.zeros(600, H, dtype=torch.bfloat16, device=DEV))
    small = L.embed_backward(go, ids, 600)        # V H = 38400: the radix sort
    large = L.embed_backward(go, ids, 1 << 20)    # V H = 2^26 < 3000 * 30000, radix; the same rows
    huge = L.embed_backward(go, ids, 1 << 20, grad_weight=torch.zeros(1 << 20, H, dtype=torch.bfloat16, device=DEV))
    assert torch.equal(ranked, small) and torch.equal(large[:600], small) and torch.equal(huge[:600], small)
