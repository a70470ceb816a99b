"""Plain 64-bit forms of the paged-cache operators, and paged inputs for their
tests.  Everything is looped over sequences and rows of positions, on whatever
device the tensors are."""
from __future__ import annotations

import math

import torch

# A rounding to bf16 is off by at most half a step relative to the value.
BF16 = torch.finfo(torch.bfloat16).eps / 2


class Paged:
    """A batch of contexts in a permuted page store.  ns / ts: new rows and
    context length of each sequence.  Rows of the store that belong to no
    context, and rows past a context's end, hold `poison`."""

    def __init__(self, ns, ts, Hq, Hkv, d, block, i8=False, seed=0, pad_rows=0, pad_pages=2,
                 poison=float("nan"), scale=1.0, device="cuda"):
        self.ns, self.ts, self.block = list(ns), list(ts), block
        self.Hq, self.Hkv, self.d, self.i8 = Hq, Hkv, d, i8
        g = torch.Generator().manual_seed(seed)
        Bt = len(ns)
        per = [-(-t // block) for t in ts]
        self.num_pages = sum(per) + pad_pages
        width = max(max(per), 1) + 1
        perm = torch.randperm(self.num_pages, generator=g)
        self.table = torch.full((Bt, width), -9, dtype=torch.int32)
        at = 0
        for b in range(Bt):
            self.table[b, :per[b]] = perm[at:at + per[b]].to(torch.int32)
            at += per[b]
        cu = [0]
        for n in ns:
            cu.append(cu[-1] + n)
        self.total = cu[-1] + pad_rows
        self.k = [torch.randn((t, Hkv, d), generator=g).mul(scale).to(torch.bfloat16) for t in ts]
        self.v = [torch.randn((t, Hkv, d), generator=g).to(torch.bfloat16) for t in ts]
        self.q = torch.randn((self.total, Hq, d), generator=g).to(torch.bfloat16).to(device)
        shape = (self.num_pages, block, Hkv, d)
        if i8:
            self.kp = torch.full(shape, 77, dtype=torch.int8)
            self.vp = torch.full(shape, 77, dtype=torch.int8)
            self.ks = torch.full((self.num_pages, Hkv, block), poison)
            self.vs = torch.full((self.num_pages, Hkv, block), poison)
        else:
            self.kp = torch.full(shape, poison, dtype=torch.bfloat16)
            self.vp = torch.full(shape, poison, dtype=torch.bfloat16)
            self.ks = self.vs = None
        for b in range(Bt):
            for x, pages, scales in ((self.k[b], self.kp, self.ks), (self.v[b], self.vp, self.vs)):
                codes, sc = quantise(x) if i8 else (x, None)
                for j in range(per[b]):
                    lo, hi = j * block, min((j + 1) * block, ts[b])
                    p = int(self.table[b, j])
                    pages[p, :hi - lo] = codes[lo:hi]
                    if i8:
                        scales[p, :, :hi - lo] = sc[lo:hi].t()
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.kv_len = torch.tensor(ts, dtype=torch.int32)
        for name in ("table", "kp", "vp", "ks", "vs", "cu", "kv_len"):
            t = getattr(self, name)
            if t is not None:
                setattr(self, name, t.to(device))

    def stores(self):
        return (self.kp, self.vp, self.ks, self.vs) if self.i8 else (self.kp, self.vp)

    def step(self):
        return self.table, self.cu, self.kv_len

    def context(self, b):
        """K and V of sequence b as the store holds them, in 64 bits: [t, Hkv, d]."""
        got = []
        for pages, scales in ((self.kp, self.ks), (self.vp, self.vs)):
            rows = []
            for pos in range(0, self.ts[b], self.block):
                p = int(self.table[b, pos // self.block])
                x = pages[p].double()
                if scales is not None:
                    x = x * scales[p].t().double()[:, :, None]
                rows.append(x[:min(self.block, self.ts[b] - pos)])
            got.append(torch.cat(rows) if rows else
                       torch.zeros((0, self.Hkv, self.d), dtype=torch.float64, device=pages.device))
        return got


def quantise(x):
    """Codes and scales of rows x [..., d], by the documented formulas in fp32."""
    x = x.float()
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    tiny = amax < 2.0 ** -100
    # (tensor by tensor: torch turns a division by a plain number into a product)
    most = torch.full_like(amax, 127)
    inv = torch.where(tiny | bad, torch.zeros_like(amax), most / amax)
    codes = torch.where(bad[..., None], torch.zeros_like(x), x * inv[..., None])
    scale = torch.where(tiny, torch.zeros_like(amax), amax / most)
    scale = torch.where(bad, torch.full_like(amax, float("nan")), scale)
    return codes.round().to(torch.int8), scale


def attend(q, k, v, seen):
    """q [rows, d], k / v [keys, d] fp64, seen [rows, keys] -> out, lse, the
    same product with |v| (what a relative error of the weights is taken of),
    and the largest sum of |q_i k_i| / sqrt(d) of each row."""
    z = q @ k.t() / math.sqrt(q.shape[1])
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, 1)
    some = seen.any(1)
    w = torch.where(some[:, None], torch.exp(z - torch.where(some, lse, torch.zeros_like(lse))[:, None]),
                    torch.zeros_like(z))
    lse = torch.where(some, lse, torch.full_like(lse, -math.inf))
    size = (q.abs() @ k.abs().t() / math.sqrt(q.shape[1])).amax(1) if k.shape[0] else torch.zeros_like(lse)
    return w @ v, lse, w @ v.abs(), size


def fixed_point(q, k, v, seen, top_scale):
    """Bound on what fixed-point weights add to the output's error, for int8
    pages.  A weight w_j (relative to the largest of its row so far, hence at
    least w_j relative to the row's largest one, w_top), times its V scale over
    the tile's largest, is rounded to a multiple of 2^-27: the error is at most
    half of that, and at most the weight itself where it rounds to 0.  It
    multiplies code_j and the tile's largest scale, at most top_scale times
    127.  For the context's rows (q [rows, d], seen [rows, keys]): [rows]."""
    z = q @ k.t() / math.sqrt(q.shape[1])
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    top = z.amax(1, keepdim=True) if z.shape[1] else z.sum(1, keepdim=True)
    w = torch.where(seen, torch.exp(z - torch.nan_to_num(top, neginf=0.0)), torch.zeros_like(z))
    e = w.clamp(max=2.0 ** -28).sum(1) * 127 * top_scale
    return e / w.sum(1).clamp(min=1e-300)


def attn(x: Paged, window=0, sinks=0):
    """Reference of attn_paged over the rows 0 .. cu[-1]: out, lse, tol_out, tol_lse."""
    rows = sum(x.ns)
    dev = x.q.device
    G = x.Hq // x.Hkv
    out = torch.zeros((rows, x.Hq, x.d), dtype=torch.float64, device=dev)
    wide = torch.zeros_like(out)
    lse = torch.zeros((rows, x.Hq), dtype=torch.float64, device=dev)
    size = torch.zeros_like(lse)
    fixed = torch.zeros_like(lse)
    at = 0
    for b, (n, t) in enumerate(zip(x.ns, x.ts)):
        k, v = x.context(b)
        top_scale = x.vs.nan_to_num(0).max().item() if x.i8 else 0.0
        i = torch.arange(t - n, t, device=dev)[:, None]
        j = torch.arange(t, device=dev)[None]
        seen = j <= i
        if window:
            seen = seen & ((j > i - window) | (j < sinks))
        for h in range(x.Hq):
            o, l, a, s = attend(x.q[at:at + n, h].double(), k[:, h // G], v[:, h // G], seen)
            out[at:at + n, h], lse[at:at + n, h], wide[at:at + n, h], size[at:at + n, h] = o, l, a, s
            if x.i8:
                fixed[at:at + n, h] = fixed_point(x.q[at:at + n, h].double(), k[:, h // G],
                                                  v[:, h // G], seen, top_scale)
        at += n
    t_out, t_lse = tolerances(out, lse, wide, size, x.d)
    return out, lse, t_out + fixed[..., None], t_lse


def tolerances(out, lse, wide, size, d):
    """Elementwise bounds.  A score is a sum of d fp32 products: off by at most
    (d + 4) 2^-23 of the sum of their magnitudes (the scale factors add two
    roundings), and so is lse, beside the approximations of 2^x and log2
    (2^-20).  A weight is off by that, relatively, and is rounded to bf16; the
    output is rounded once more."""
    score = (d + 4) * 2.0 ** -23 * size
    t_lse = score + 2.0 ** -20 * (1 + torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse)))
    t_out = BF16 * out.abs() + (BF16 + 2 * t_lse)[..., None] * wide * (1 + BF16) + 1e-30
    return t_out, t_lse


def check(got, lse, ref, ref_lse, t_out, t_lse, what=""):
    got, lse = got.double(), lse.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse), empty), f"{what}: rows without keys"
    assert (got[empty] == 0).all(), f"{what}: rows without keys are not zero"
    over = ((got - ref).abs() / t_out).max().item()
    assert over <= 1, f"{what}: out off by {over:.3g} times its bound"
    fine = ~empty
    if fine.any():
        over = ((lse - ref_lse).abs()[fine] / t_lse[fine]).max().item()
        assert over <= 1, f"{what}: lse off by {over:.3g} times its bound"
