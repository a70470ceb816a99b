"""The bounds of cache_bounds tell the kernels' roundings from coarser ones: the
weights' roundings are replayed here on the CPU, with and without a mistake."""
import pytest
import torch

import cache_bounds
from cache_ref import quantise


def _inputs(T, up, i8, d=128):
    """q, K, V and V's scales in 64 bits.  up: key 33 has no weight to speak of
    and a V row 2^up times the others."""
    g = torch.Generator().manual_seed(1)
    q = torch.randn((8, d), generator=g).to(torch.bfloat16).double()
    k = torch.randn((T, d), generator=g).to(torch.bfloat16).double()
    rows = torch.randn((T, d), generator=g).to(torch.bfloat16)
    q[:, 0] = 4
    if not i8:
        return q, k, rows.double(), None
    codes, sv = (t.double() for t in quantise(rows))
    if up:
        k[33] = 0
        k[33, 0] = -1270
        sv[33] *= 2.0 ** up
    return q, k, codes * sv[:, None], sv


def _excess(T, form, up=0, i8=True):
    """Largest error of the replayed form, over its bound."""
    q, k, v, sv = _inputs(T, up, i8)
    seen = torch.ones((8, T), dtype=torch.bool)
    z = q @ k.t() / q.shape[1] ** 0.5
    p = torch.exp(z - z.amax(1, keepdim=True))
    total = p.sum(1, keepdim=True)
    o = torch.zeros((8, v.shape[1]), dtype=torch.float64)
    for t in range(0, T, 128):
        part, rows = p[:, t:t + 128], v[t:t + 128]
        if form == "bf16":
            x = part.to(torch.bfloat16).double()
        elif form == "two bf16 terms":
            hi = part.to(torch.bfloat16)
            x = hi.double() + (part - hi.double()).to(torch.bfloat16).double()
        else:  # integers, in a unit of the tile's V scales or of the row's own terms
            terms = part * sv[t:t + 128]
            if form == "unit of the tile":
                unit = sv[t:t + 128].max() * 2.0 ** -27
            elif form == "unit of the maxima":
                unit = torch.exp2(torch.ceil(torch.log2(part.amax(1, keepdim=True))) - 26 +
                                  torch.floor(torch.log2(sv[t:t + 128].max())))
            else:
                unit = torch.exp2(torch.floor(torch.log2(terms.amax(1, keepdim=True))) - 27)
            x, rows = (terms / unit).round() * unit, rows / sv[t:t + 128, None]
        o += x @ rows
    got = (o / total).to(torch.bfloat16).double()
    bound = cache_bounds.bounds(q, k, v, seen, "split", sv)[0]
    w = cache_bounds.weights(q, k, seen)
    return ((got - w @ v).abs() / bound).max().item()


@pytest.mark.parametrize("T", [40, 130, 701])
def test_bounds_of_the_split_kernel(T):
    assert _excess(T, "two bf16 terms", i8=False) <= 1
    assert _excess(T, "bf16", i8=False) > 1
    assert _excess(T, "unit of the maxima") <= 1
    for up in (0, 16, 20, 24, 28):
        assert _excess(T, "unit of the row", up) <= 1
    for up in (20, 24, 28):
        assert _excess(T, "unit of the tile", up) > 1
