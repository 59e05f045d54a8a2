"""embedding's padding_idx is checked where it is given."""
import pytest
import torch

import lm_head_logits_amd as L


@pytest.mark.parametrize("bad", [9, -10, 1 << 40])
def test_a_padding_row_outside_the_table_is_refused(bad):
    ids, W = torch.zeros(4, dtype=torch.int64), torch.zeros(9, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="padding_idx"):
        L.embedding(ids, W, padding_idx=bad)


@pytest.mark.gpu
def test_every_row_may_be_the_padding_row():
    ids = torch.arange(9, device="cuda:0")
    for p in (0, 8, -1, -9):
        W = torch.ones(9, 64, dtype=torch.bfloat16, device="cuda:0", requires_grad=True)
        L.embedding(ids, W, padding_idx=p).sum().backward()
        want = torch.ones(9, 64, device="cuda:0")
        want[p] = 0
        assert torch.equal(W.grad.float(), want)
