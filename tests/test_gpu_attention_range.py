"""Single-token attention over the whole range of scores and values: scores that rise and fall
along a sequence, value scales far apart, rows of value zero, tiny queries.  Float32 outputs
against the 64-bit form, within the bounds counted in attention_bounds."""

import math

import pytest
import torch

import attention_bounds as tight
import decode_ref as ref
from test_gpu_attention_decode import _gen, _run, _setup
from util import DEV

pytestmark = pytest.mark.gpu

LAYOUTS = [(16, 4), (32, 2)]            # groups of 4 and of 16 query rows
# (lengths, prefix): undivided sequences, divided ones, a prefix of under 64 query rows a head;
# long enough for several tiles to a block
PLACES = {"undivided": ([1000, 129, 37, 640], None), "divided": ([40000, 700, 1, 3000], None),
          "prefix": ([100, 1, 0], 20000)}


def _check(fge, s, prefix, scale=None, unit=tight.OWN, **more):
    q, cache, table, lens, pp = s
    out, lse, status = _run(fge, q, cache, table, lens, pp, prefix, torch.float32, scale)
    assert status == 0
    r = tight.attention(q, cache, table, lens, q.shape[2] ** -0.5 if scale is None else scale, pp,
                        prefix or 0, unit, **more)
    ref.check_attention(out, lse, r, torch.float32)


def _no_zero_rows(cache):
    """A value in every row: a cache's zero rows have a scale of their own."""
    cache[2][(cache[2] & 0x7F).amax(-1) == 0] = 0x38


def _along(s, prefix):
    """Place of every cached token in its sequence, 0 to 1, as [pages, page]."""
    q, cache, table, lens, pp = s
    page = cache[1].shape[2]
    at = torch.zeros((cache[1].shape[0], page), device=DEV)
    rows = [(table[i], int(lens[i])) for i in range(len(lens))]
    if pp is not None:
        rows.append((pp, prefix))
    for pages, n in rows:
        for j in range((n + page - 1) // page):
            at[int(pages[j])] = (j * page + torch.arange(page, device=DEV)) / n
    return at


@pytest.mark.parametrize("heads,n_kv", LAYOUTS)
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rise,spread", [(64.0, 0.0), (1.0 / 64.0, 0.0), (1.0, 20.0), (8.0, 40.0),
                                         (64.0, -40.0)])
def test_scores_and_values_that_change_along_it(fge, heads, n_kv, place, d, rise, spread):
    # spread < 0: values that fall by 2^(2 spread) along the sequence
    lengths, prefix = PLACES[place]
    s = _setup(fge, lengths, heads, n_kv, d, 64, int(d + spread), prefix, spoil=False)
    cache = s[1]
    _no_zero_rows(cache)
    at = _along(s, prefix)[:, None]
    cache[1].mul_(torch.exp(math.log(rise) * at))
    if spread < 0:
        cache[3].mul_(torch.exp2(-spread * (1 - 2 * at)))
    else:
        cache[3].mul_(torch.exp2(spread * (2 * torch.rand(cache[3].shape, generator=_gen(5),
                                                          device=DEV) - 1)))
    _check(fge, s, prefix)


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up,down", [(20, 20), (40, 28), (60, 40), (120, 90), (300, 100)])
def test_a_large_value_that_loses_its_weight(fge, place, d, up, down):
    # The first token has the largest value; another one, whose score is `up` higher in base 2
    # and whose value is 2^down smaller, takes its weight.  Both lie in the part of the tiles
    # that one warp takes.
    _, prefix = PLACES[place]
    n = {"undivided": 200, "divided": 60000, "prefix": 16384}[place]
    lengths, shared = ([n, 130], None) if prefix is None else ([1, 1], n)
    s = _setup(fge, lengths, 4, 2, d, 64, 17, shared, spoil=False)
    q, cache, table, lens, pp = s
    q.fill_(1.0)
    _no_zero_rows(cache)
    cache[0].zero_()                    # score 0 but for the one token
    cache[1].fill_(1.0)
    cache[3].fill_(2.0 ** -down)
    pages = table[0] if shared is None else pp
    cache[3][int(pages[0]), :, 0] = 1.0
    late = (int(pages[128 // 64]), slice(None), 128 % 64)
    cache[0][late] = 0x38               # 1.0
    cache[1][late] = up * math.log(2.0) / d
    _check(fge, s, shared, scale=1.0)


@pytest.mark.parametrize("heads,n_kv", LAYOUTS)
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("small", [1.0, 2.0 ** -20, 2.0 ** -31, 2.0 ** -60])
def test_rows_of_value_zero_beside_small_values(fge, heads, n_kv, place, d, small):
    # every 13th row is zero and has scale 1 by the cache's rule
    lengths, prefix = PLACES[place]
    s = _setup(fge, lengths, heads, n_kv, d, 64, d, prefix, spoil=False)
    cache = s[1]
    zero = (cache[2] & 0x7F).amax(-1) == 0
    assert zero.any() and (cache[3][zero] == 1.0).all()
    cache[3][~zero] *= small
    _check(fge, s, prefix)


def test_only_rows_of_value_zero(fge):
    s = _setup(fge, [300, 40, 1], 16, 4, 128, 64, 3, spoil=False)
    s[1][2].zero_()
    s[1][3].fill_(1e30)
    out, lse, status = _run(fge, *s[:4], dtype=torch.float32)
    assert status == 0 and not out.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("prefix,b", [(None, 3), (700, 3), (700, 40)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-110, -121, -126])
def test_tiny_queries_and_large_keys(fge, prefix, b, d, power):
    s = _setup(fge, [(97 * i) % 300 for i in range(b)], 16, 4, d, 64, 23, prefix, spoil=False)
    q, cache, table, lens, pp = s
    q.copy_((q.float() * 2.0 ** power).to(torch.bfloat16))
    cache[1].mul_(2.0 ** 118)           # values up to 2^121
    # the row's factor may be subnormal: 2^-129 keeps 20 bits
    _check(fge, s, prefix, scale=0.25 * 2.0 ** (-118 - power),
           unit=tight.TCGEN05 if b * 4 >= 64 else tight.OWN, score_error=2.0 ** -19)


@pytest.mark.parametrize("prefix,b", [(None, 3), (3000, 3), (3000, 40)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-112, -95, -60, 60, 110])
def test_values_of_any_size(fge, prefix, b, d, power):
    # scales from 2^-122 to 2^110, rows of value zero (scale 1) among them
    s = _setup(fge, [(97 * i) % 300 for i in range(b)], 16, 4, d, 64, 31, prefix, spoil=False)
    cache = s[1]
    some = (cache[2] & 0x7F).amax(-1) != 0
    cache[3][some] *= 2.0 ** power
    # the own part's weights are brought up by 2^126 at most: from 2^-118 to 2^8 instead of 2^14
    own = tight.OWN if power > -100 else 2.0 ** -33
    _check(fge, s, prefix, unit=tight.TCGEN05 if b * 4 >= 64 else own)


@pytest.mark.parametrize("d", [64, 128])
def test_tcgen05_prefix_within_the_tight_bounds(fge, d):
    s = _setup(fge, [(11 * i) % 90 for i in range(40)], 16, 4, d, 64, 29, 5000, spoil=False)
    _check(fge, s, 5000, unit=tight.TCGEN05)


def test_tcgen05_prefix_gives_the_same_bits_every_time(fge):
    # full-size runs of the kernel whose values come from TMEM: 384 rows a head, three row-tile
    # pairs, and an odd last one
    for b in (96, 72):
        q, cache, table, lens, pp = _setup(fge, [(31 * i) % 200 for i in range(b)], 16, 4, 128, 64,
                                           b, 9000, spoil=False)
        pl = torch.tensor([9000], device=DEV, dtype=torch.int32)
        lse = torch.empty((b, 16), device=DEV)

        def call():
            return fge.attention_decode(q, cache, table, lens, prefix_pages=pp, prefix_length=pl,
                                        out_dtype=torch.float32, lse=lse)

        want, first = call(), lse.clone()
        for _ in range(50):
            assert torch.equal(call(), want) and torch.equal(lse, first)
