"""A prompt's keys and values: what StackedPrefill reports of writing its own, and a prompt that goes
through StackedDecode, several tokens of a sequence a step."""

import pytest
import torch

import attention_bounds as tight
import decode_ref as ref
from test_gpu_stack_decode import (E, H, HEADS, I, K, KV, PAGE, PAGES, WIDTH, _batch, _layers,
                                   _model)
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


@pytest.mark.parametrize("chunks", [[64, 61], [1, 20, 16]])
def test_a_prompt_in_steps_attends_to_the_tokens_before_each(fge, chunks):
    # rows of a step may be tokens of one sequence: their keys and values are written first, and
    # each row's length ends with its own token
    layers = _layers(1)
    model = _model(fge, layers, 64)
    _, _, table, _ = _batch(fge, model, 64, seed=8)
    pages = table[5]
    h0 = torch.randn((sum(chunks), H), generator=torch.Generator(device=DEV).manual_seed(4),
                     device=DEV)
    begin = 0
    for n in chunks:
        at = torch.arange(begin, begin + n, device=DEV)
        slots = pages.long()[at // PAGE] * PAGE + at % PAGE
        lengths = (at + 1).int()
        rows = pages[None].expand(n, WIDTH).contiguous()
        model.step(h0[begin:begin + n].clone(), slots, rows, lengths)
        assert model.status() == 0
        q = model.qkv[:n, :HEADS * 128].reshape(n, HEADS, 128)
        want = tight.attention(q, model.caches[0], rows, lengths, 128 ** -0.5)
        ref.check_attention(model.attn[:n].view(n, HEADS, 128), None, want, torch.bfloat16)
        k, _ = fge.kv_cache_read(slots, model.caches[0], out_dtype=torch.float32)
        x = model.qkv[:n, HEADS * 128:(HEADS + KV) * 128].reshape(n, KV, 128).float()
        step = x.abs().amax(-1, keepdim=True) / 448.0
        assert ((k - x).abs() <= x.abs() * 2.0 ** -4 + step * 2.0 ** -9).all()
        begin += n
