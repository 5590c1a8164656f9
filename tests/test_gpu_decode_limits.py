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


@pytest.mark.parametrize("places", ["own", "prefix", "tcgen05 prefix"])
@pytest.mark.parametrize("past", [0, 13])
def test_lengths_up_to_the_last_tokens_below_two_to_the_31(fge, places, past):
    # a table of as many pages as are admitted, all of them the same one
    page, d, width = 16, 64, (1 << 27) - 1
    length = width * page - past
    g = torch.Generator(device=DEV).manual_seed(5)
    cache = fge.new_kv_cache(1, page, 1, d, DEV)
    k, v = (torch.randn((page, 1, d), generator=g, device=DEV).to(torch.bfloat16)
            for _ in range(2))
    fge.kv_cache_write(k, v, torch.arange(page, device=DEV), cache)
    b, heads = (8, 8) if places == "tcgen05 prefix" else (1, 4)
    q = torch.randn((b, heads, d), generator=g, device=DEV).to(torch.bfloat16)
    pages = torch.zeros(width, dtype=torch.int32, device=DEV)
    whole = torch.tensor([length], dtype=torch.int32, device=DEV)
    lse = torch.empty((b, heads), device=DEV)
    if places == "own":
        out = fge.attention_decode(q, cache, pages[None], whole, out_dtype=torch.float32, lse=lse)
    else:
        out = fge.attention_decode(q, cache, torch.zeros((b, 1), dtype=torch.int32, device=DEV),
                                   torch.zeros(b, dtype=torch.int32, device=DEV),
                                   prefix_pages=pages, prefix_length=whole,
                                   out_dtype=torch.float32, lse=lse)
    kd, vd = (a.view(torch.float8_e4m3fn).double()[0, 0] * s.double()[0, 0, :, None]
              for a, s in ((cache[0], cache[1]), (cache[2], cache[3])))
    s = q.double() @ kd.T * d ** -0.5
    want = torch.softmax(s, -1) @ vd
    # a run of 2^18 tiles adds to its sums 2^18 times, off by 2^-24 at most each, and to its
    # outputs 2^21 times, off by 2^-23 (sums of matrix instructions are cut off)
    assert (lse.double() - torch.logsumexp(s, -1) - torch.log(torch.tensor(float(width)))).abs().max() \
        <= 2.0 ** -6 + 1e-3
    assert ((out.double() - want).abs() <= (2.0 ** -2 + 2.0 ** -6 + 2.0 ** -11)
            * (torch.softmax(s, -1) @ vd.abs())).all()


@pytest.mark.parametrize("b", [2, 40])          # 16-row and tcgen05 form
@pytest.mark.parametrize("length,code", [(0, 0), (1, 11), (-1, 11), (1 << 30, 11)])
def test_a_prefix_of_no_pages_is_reported(fge, b, length, code):
    q, cache, table, lens, _ = _setup(fge, [20, 3] * (b // 2), 16, 4, 128, 64, 2)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert none.data_ptr() == 0
    ws = fge.new_workspace(fge.workspace_bytes(fge.OP_ATTENTION_DECODE_SHARED, b, 16, 128, 4), DEV)
    want = fge.attention_decode(q, cache, table, lens)
    for pages in (none, torch.empty(4, dtype=torch.int32, device=DEV)[:0]):
        fge.clear_device_status(ws)
        out = fge.attention_decode(q, cache, table, lens, prefix_pages=pages, workspace=ws,
                                   prefix_length=torch.tensor([length], dtype=torch.int32,
                                                              device=DEV))
        assert fge.read_device_status(ws) == code
        # an empty prefix adds nothing, though its outputs are joined: one division later
        assert torch.equal(out, want)


def test_a_status_workspace_that_cannot_hold_the_status_is_refused(fge):
    cache = fge.new_kv_cache(2, 16, 1, 64, DEV)
    x = torch.ones((2, 64), dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(2, device=DEV)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    calls = (lambda w: fge.kv_cache_write(x, x, slots, cache, workspace=w),
             lambda w: fge.kv_cache_read(slots, cache, workspace=w))
    for call in calls:
        for w in (None, ws[:256], ws[16:272]):
            call(w)
        for w, why in ((ws[:255], "workspace"), (ws[:1], "workspace"), (ws[8:], "align")):
            with pytest.raises(fge.FgeError, match=why):
                call(w)
