"""Small softmax weights of the e4m3 chunk attention: a few keys far above the rest must not cost the rest its mass.

The queries have RoPE dims alone, so that the logits do not depend on the values, and the values of the many
small keys have a common mean, so that a part of their mass that is lost or added shows.

Tolerance.  Beside what every form of the call has (logits off by d, exp2, n roundings in fp32, the output's
2^-8), a weight w, in the kernel's units where the row's largest stands at 2^4.5 or more, is held as
hi + lo, e4m3 and e5m2, of its fp16 value (tests/test_chunk_weight_split.py):
- It keeps 8 significant bits, 2^-8 of its binade; fp16 adds 2^-11.
- What is left beyond lo's three bits is rounded up or down by thresholds spread over lo's step u, so that the mean is
  right: each weight is off by less than u <= max(2^-2 w, 2^-16), by u / 2 in the root mean square at most, independent
  between keys (or better, the thresholds of 32 keys being spread evenly).  Eight deviations of the sum:
  4 sqrt(sum u^2 v^2).  2^-16 is 2^-20.5 of the row's largest weight P or less.
So with M = sum p |v|

    |out - ref| <= M (2^-8 + 2^-11 + 2d + 2^-21 + n 2^-23) + 4 sqrt(sum (2^-2 p + 2^-20 P)^2 v^2) + 2^-8 |ref|
                   (+ second-order terms, 2 %)
"""
import math

import pytest
import torch

from tests import prefill_reference as P
from tests.test_chunk_gpu import _run

pytestmark = pytest.mark.gpu

SCALE = 0.125


def _tail(lens, gaps, std, sinks, seed=0):
    """One sequence for each length, four query tokens each; head i sees the keys `sinks` at gaps[i] (in nats) above
    the others, whose logits have the deviation std[i]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    h, T = len(gaps), 4 * len(lens)
    bt, pool = P.paging(lens, seed)
    k = torch.randn((pool, 64, 1, 576), generator=g, device="cuda")
    k[..., :512] = 1.0 + 0.5 * k[..., :512]
    k[..., 512:514] = 0.0
    bt = bt.cuda()
    for b, L in enumerate(lens):
        for s in sinks:
            k[bt[b, s // 64].long(), s % 64, 0] = 0.0
            k[bt[b, s // 64].long(), s % 64, 0, 512:514] = 8.0
    q = torch.zeros((T, h, 576), device="cuda")
    whole = torch.tensor(gaps, device="cuda").floor()
    q[..., 512], q[..., 513] = whole, torch.tensor(gaps, device="cuda") - whole
    q[..., 514:] = torch.randn((T, h, 62), generator=g, device="cuda") * (torch.tensor(std, device="cuda") / (SCALE * 62 ** 0.5))[None, :, None]
    cu = torch.arange(0, T + 1, 4, dtype=torch.int32, device="cuda")
    return q.to(P.E4M3), k.to(P.E4M3), bt, cu, torch.tensor(lens, dtype=torch.int32, device="cuda")


def _check(out, lse, q, cache, bt, lens, out_scale=1.0):
    n = [4] * len(lens)
    ref, rl, mag, big = P.chunk(q, cache, bt, n, lens, SCALE, out_scale, True)
    d = (577 * 2.0 ** -24 * big)[..., None]
    keys = max(lens)
    bound = mag * (2.0 ** -8 + 2.0 ** -11 + 2 * d + 2.0 ** -21 + keys * 2.0 ** -23) + 2.0 ** -8 * ref.abs()
    for b, L in enumerate(lens):
        k = P.gather(cache, bt, b, L)[:, 0]
        for i in range(4 * b, 4 * b + 4):
            s = SCALE * (q[i].float().double() @ k.T)
            s[:, L - 3 + i - 4 * b:] = -math.inf
            p = torch.softmax(s, -1)
            u = (0.25 * p + 2.0 ** -20 * p.amax(-1, keepdim=True)) * (p > 0)
            bound[i] += abs(out_scale) * 4 * (u.square() @ k[:, :512].square()).sqrt()
    off = (out.double() - ref).abs()
    worst = (off / (bound * 1.02)).amax((0, 2))
    assert (worst <= 1).all(), "of the bound, by head: " + " ".join("%.2f" % x for x in worst.tolist())
    lb = 2 * d[..., 0] + 2.0 ** -20 + keys * 2.0 ** -24 + 2.0 ** -23 * rl.abs()
    assert ((lse.double() - rl).abs() <= lb).all()


GAPS = [3.0, 5.0, 6.5, 7.5, 8.0, 9.0, 9.5, 10.0, 10.5, 11.0, 11.5, 12.0, 12.5, 13.0, 14.0, 15.0]


@pytest.mark.parametrize("parts", [1, None])
@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_a_long_tail_far_below_one_key(spread, parts):
    """The first key stands above 40,000 equal ones, or ones of unlike logits."""
    lens = [40_003]
    q, cache, bt, cu, L = _tail(lens, GAPS, [spread] * 16, [0], seed=3)
    out, lse = _run(q, cache, bt, cu, L, 1, scale=SCALE, parts=parts)
    _check(out, lse, q, cache, bt, lens)


@pytest.mark.parametrize("sinks", [[777], [20_001], [0, 5000, 29_999], list(range(64, 30_000, 128))])
def test_large_keys_elsewhere(sinks):
    """Large keys inside the sequence, at its end, and one in every tile; and a second sequence with few keys."""
    lens = [30_000, 1000]
    if max(sinks) >= 1000:
        lens[1] = 30_000
    q, cache, bt, cu, L = _tail(lens, GAPS, [0.0, 0.7] * 8, sinks, seed=4)
    out, lse = _run(q, cache, bt, cu, L, 1, scale=SCALE, out_scale=-1.5)
    _check(out, lse, q, cache, bt, lens, -1.5)


@pytest.mark.parametrize("gap", [9.0, 11.0, 13.0])
def test_values_that_alternate_with_the_keys(gap):
    """Values that change their sign with every key, or every 2nd, 4th .. 64th: the rounding follows no such pattern."""
    lens = [30_000]
    q, cache, bt, cu, L = _tail(lens, [gap] * 16, [0.0] * 16, [0], seed=5)
    pos = torch.arange(lens[0], device="cuda")
    v = torch.stack([1.0 - 2.0 * ((pos >> (i % 7)) & 1) for i in range(512)], -1)
    v[0] = 0
    bits = cache.view(torch.uint8)
    bits[bt[0, pos // 64].long(), pos % 64, 0, :512] = v.to(P.E4M3).view(torch.uint8)
    out, lse = _run(q, cache, bt, cu, L, 1, scale=SCALE)
    _check(out, lse, q, cache, bt, lens)
