"""Bounds on the attention over pages that count only what a row sees: its
visible keys, each with its weight.  (The plain 64-bit forms are cache_ref's.)

A score is a sum of d fp32 products: off by at most
    e_j = (d + 4) 2^-23 sum_i |q_i k_ji| / sqrt(d)
(the scale factors add two roundings).  Then the weights w_j are off by e_j
relatively, and their sum by sum_j w_j e_j, which is also what lse is off by,
beside the approximations of 2^x and log2 (2^-20)."""
from __future__ import annotations

import torch

from cache_ref import BF16, attend


def reaches(x, kernel, window=0, sinks=0, max_q=None):
    """Whether attention over the batch x takes that kernel, "split" or "chunk", for
    its longest sequence.  (Where both are launched, the split kernel has the
    sequences of at most 16 rows per kv head.)"""
    from block_sparse_long_05_b200 import msa
    taken = msa.attn_paged_kernels(len(x.ns), x.q.shape[0], x.Hq, x.Hkv, x.block, x.table.shape[1],
                                   window, sinks, max_q)
    if len(taken) == 2:
        taken = ("chunk",) if max(x.ns) * x.Hq // x.Hkv > 16 else ("split",)
    return taken == (kernel,)


def visible(n, t, window=0, sinks=0, cap=None, device="cuda"):
    """Keys [n, cap or t] that the n rows at positions t - n .. t - 1 see."""
    i = torch.arange(t - n, t, device=device)[:, None]
    j = torch.arange(t if cap is None else cap, device=device)[None]
    seen = j <= i
    if window:
        seen = seen & ((j > i - window) | (j < sinks))
    return seen


def weights(q, k, seen):
    """Softmax weights [rows, keys] (0 for rows that see nothing)."""
    z = q @ k.t() / q.shape[1] ** 0.5
    z = torch.where(seen, z, torch.full_like(z, -1e300))
    return torch.softmax(z, 1) * seen


def bounds(q, k, v, seen, kernel, sv=None):
    """(bound of out [rows, d], bound of lse [rows]) for q [rows, d], k / v
    [keys, d] in 64 bits.  sv [keys]: the scales of V (int8 pages).

    The chunk kernel rounds each weight (times its V scale) to bf16.

    On int8 pages the split kernel takes q in multiples of 2^-19 of the power of
    two below its row's largest value: what that takes from q_i (nothing, for
    values within 2^12 of the largest) moves a score by its product with k_i.

    The split kernel on bf16 pages takes a weight as two bf16 terms: the first
    leaves at most 2^-7 of it, of which the second misses BF16, below 2^-15.
    On int8 pages the products w_j sv_j of a row and a tile of 128 keys are
    rounded to multiples of 2^(f - 26), where 2^(f - 3) is at most the tile's
    largest one (the row's largest w, rounded down to a power of two, times the
    largest sv, rounded down likewise, over 4): by at most 2^-24 of that, for a
    code of at most 127.  Keys that the row does not see are exact zeros.

    The second product adds 128 keys in fp32 at a time, then keys / 128 such
    sums and their merge.  One rounding to bf16 at the end."""
    w = weights(q, k, seen)
    e = (q.shape[1] + 4) * 2.0 ** -23 * (q.abs() @ k.abs().t()) / q.shape[1] ** 0.5
    if kernel == "split" and sv is not None:
        unit = torch.exp2(torch.floor(torch.log2(q.abs().amax(1, keepdim=True).clamp(min=1e-30))) - 19)
        e = e + (q - (q / unit).round() * unit).abs() @ k.abs().t() / q.shape[1] ** 0.5
    of_sum = (w * e).sum(1)
    wide = w @ v.abs()
    lse = torch.logsumexp(torch.where(seen, q @ k.t() / q.shape[1] ** 0.5, torch.full_like(w, -1e300)), 1)
    t_lse = of_sum + 2.0 ** -20 * (1 + torch.where(seen.any(1), lse.abs(), torch.zeros_like(lse)))
    rel = t_lse + (128 + k.shape[0] / 128 + 16) * 2.0 ** -23
    t_out = (w * e) @ v.abs() + rel[:, None] * wide
    if kernel == "chunk":
        t_out = t_out + BF16 * wide
    elif sv is None:
        t_out = t_out + 2.0 ** -15 * wide
    else:
        t_out = t_out + (seen.sum(1) * 127 * 2.0 ** -24 * (w * sv).amax(1))[:, None]
    return BF16 * (w @ v).abs() + (1 + BF16) * t_out + 1e-30, t_lse


def reference(x, b, at, h, seen, kernel):
    """out, lse and their bounds for head h of sequence b, whose rows begin at
    `at`.  kernel: "split" or "chunk"."""
    G = x.Hq // x.Hkv
    k, v = x.context(b)
    q, kh, vh = x.q[at:at + x.ns[b], h].double(), k[:, h // G], v[:, h // G]
    o, l = attend(q, kh, vh, seen)[:2]
    sv = None
    if x.i8:
        pos = torch.arange(x.ts[b], device=x.q.device)
        sv = x.vs[x.table[b].long()[pos // x.block], h // G, pos % x.block].double()
    return (o, l, *bounds(q, kh, vh, seen, kernel, sv))
