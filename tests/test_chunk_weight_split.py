"""How the e4m3 chunk attention holds a softmax weight, over every fp16 value and every threshold (CPU).

A restatement of split_e4m3x2 (csrc/chunk_attn.cuh): hi = e4m3(w), then the remainder by way of a sum with 8 hi in
fp16, then a threshold added below the upper byte of that fp16 value, which is e5m2.
"""
import torch


def _split(w):
    """w (n) fp16 -> hi (n), lo (256 thresholds, n), in 64 bits."""
    d = w.double()
    hi = w.float().to(torch.float8_e4m3fn).double()
    rest = (d + 7 * hi).half()                       # one rounding, as the fused product and sum has
    rest = (rest.double() - 8 * hi).half()
    bits = rest.view(torch.int16).int() & 0xffff
    lo = []
    for threshold in range(256):
        b = (bits + threshold) & 0xff00
        lo.append(torch.where(b >= 0x8000, b - 0x10000, b).short().view(torch.float16).double())
    return hi, torch.stack(lo)


def test_every_weight():
    w = torch.arange(0, 0x5f00, dtype=torch.int32).short().view(torch.float16)   # up to 448; the kernel's end at 2^8.5
    hi, lo = _split(w)
    w = w.double()
    held = hi + lo
    binade = 2.0 ** torch.floor(torch.log2(w.clamp(min=2.0 ** -25)))
    large = w >= 2.0 ** -6
    # to the nearest of 8 significant bits, whatever the threshold
    assert torch.equal(held[:, large], held[:1, large].expand(256, -1))
    assert ((held[0] - w).abs() <= 2.0 ** -8 * binade)[large].all()
    assert (((held[0] - w) / w)[large]).mean().abs() <= 2.0 ** -14
    # smaller ones: off by less than a step, right in the mean to 2^-8 of the binade, and exactly where hi is 0
    small = ~large
    assert ((held - w)[:, small].abs() < torch.maximum(w[small] / 4, torch.tensor(2.0 ** -16, dtype=torch.float64))).all()
    off = (held.mean(0) - w).abs()
    assert (off <= 2.0 ** -8 * binade)[small].all()
    assert (off[w < 2.0 ** -10] == 0).all()
    assert (held[:, 0] == 0).all()                    # a masked key's weight stays 0


def test_thresholds_are_spread_evenly():
    """The 32 thresholds of a thread, XORed with any byte, fall into 32 different intervals of 8."""
    thresholds = [sum(((key >> i) & 1) << (7 - i) for i in range(5)) + 4 for key in range(32)]
    for shift in range(256):
        assert sorted((t ^ shift) >> 3 for t in thresholds) == list(range(32))
