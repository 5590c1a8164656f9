"""StackedPrefill writing a prompt's keys and values: what it reports."""

import pytest
import torch

from test_gpu_stack_decode import E, H, HEADS, I, K, KV, PAGE, PAGES, _layers, _model
from util import DEV

pytestmark = pytest.mark.gpu


def _prefill(fge, t, n=2):
    layers = _layers(n)
    return (fge.StackedPrefill(layers, t, H, E, I, K, HEADS, KV, DEV), _model(fge, layers, 4),
            torch.randn((t, H), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV))


def test_a_prompt_slot_past_the_cache_reaches_the_status(fge):
    t = 20
    prefill, decode, h = _prefill(fge, t)
    slots = torch.arange(t, device=DEV)
    assert prefill.status() == 0
    prefill.forward(h.clone())
    prefill.forward(h.clone(), caches=decode.caches, slots=slots)
    assert prefill.status() == 0
    slots[7] = PAGES * PAGE
    prefill.forward(h.clone(), caches=decode.caches, slots=slots)
    assert prefill.status() == fge.ERR_BAD_INDEX


def test_a_key_that_is_not_finite_reaches_the_status(fge):
    t = 5
    prefill, decode, h = _prefill(fge, t, 1)
    h[3, 0] = float("inf")
    prefill.forward(h, caches=decode.caches, slots=torch.arange(t, device=DEV))
    assert prefill.status() == fge.ERR_NONFINITE
