"""Limits of the decode-step calls: what they refuse, what they report, and the largest lengths."""

import pytest
import torch

from test_gpu_attention_decode import _setup
from util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [2, 6])
def test_heads_that_are_no_groups_are_refused(fge, heads):
    # with a workspace of the call's own, whose size is asked for before the shapes are checked
    q, cache, table, lens, pp = _setup(fge, [20, 3], 4, 4, 128, 64, 1, prefix=100)
    q = torch.zeros((2, heads, 128), dtype=torch.bfloat16, device=DEV)
    pl = torch.tensor([100], device=DEV, dtype=torch.int32)
    with pytest.raises(fge.FgeError, match="fge_attention_decode failed"):
        fge.attention_decode(q, cache, table, lens)
    with pytest.raises(fge.FgeError, match="fge_attention_decode_shared failed"):
        fge.attention_decode(q, cache, table, lens, prefix_pages=pp, prefix_length=pl)


@pytest.mark.parametrize("t,k", [(65, 2), (4, 1 << 30), (4, 9), (4, -1)])
def test_layers_are_refused_before_memory_is_taken(fge, t, k):
    logits = torch.zeros((t, 8), device=DEV)
    x = torch.zeros((t, 256), dtype=torch.bfloat16, device=DEV)
    banks = [torch.zeros(s, dtype=d, device=DEV) for s, d in
             (((8, 256, 128), torch.uint8), ((8, 2, 256), torch.float32),
              ((8, 256, 64), torch.uint8), ((8, 1, 256), torch.float32))]
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(fge.FgeError, match="fge_moe_layer_decode failed"):
        fge.moe_layer_decode(logits, x, k, 128, *banks)
    assert torch.cuda.max_memory_allocated() - before <= 1 << 17
