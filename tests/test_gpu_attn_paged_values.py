"""Values of V at the ends of their range: infinities on keys that every query
sees, and finite values so large that a weight above 1 would carry them out of
the range of fp32."""
import pytest
import torch

import cache_bounds
import cache_ref
from cache_ref import Paged
from gpu_helpers import lib_ready

pytestmark = pytest.mark.gpu


def _run(x, kernel):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    assert cache_bounds.reaches(x, kernel)
    ws = msa.Workspace.for_cache(x.Hq, x.Hkv, x.d)
    call = msa.attn_paged_i8 if x.i8 else msa.attn_paged
    out, lse = call(x.q, *x.stores(), *x.step(), ws)
    assert msa.device_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("n, kernel", [(1, "split"), (4, "split"), (1000, "chunk")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keys", [1, 2, 700])
def test_infinities_that_every_row_sees(n, kernel, d, keys):
    """A column with an infinity is that infinity, with a NaN or both infinities
    NaN, and the other columns are what they are without them.  With one key
    its weight is 1, a single bf16 term."""
    x = Paged([n], [n - 1 + keys], 4, 2, d, 64)
    k, v = x.context(0)
    seen = cache_bounds.visible(n, x.ts[0])
    want = [cache_bounds.reference(x, 0, 0, h, seen, kernel) for h in range(4)]
    p = int(x.table[0, 0])
    x.vp[p, 0, :, 3] = float("inf")
    x.vp[p, 0, :, 7] = -float("inf")
    x.vp[p, 0, :, 20] = float("nan")
    x.vp[p, 0, :, 40] = float("inf")
    both = keys > 1
    if both:
        x.vp[p, 1, :, 40] = -float("inf")
        if n > 1:
            seen2 = seen[:, 1]
            assert seen2.all()
    out, lse = _run(x, kernel)
    assert (out[..., 3] == float("inf")).all()
    assert (out[..., 7] == -float("inf")).all()
    assert torch.isnan(out[..., 20]).all()
    assert torch.isnan(out[..., 40]).all() if both else (out[..., 40] == float("inf")).all()
    fine = torch.ones(d, dtype=torch.bool)
    fine[[3, 7, 20, 40]] = False
    for h in range(4):
        o, l, t_out, t_lse = want[h]
        cache_ref.check(out[:, h][:, fine], lse[:, h], o[:, fine], l, t_out[:, fine], t_lse, f"head {h}")


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, kernel", [(1, "split"), (2, "split"), (40, "chunk")])
def test_large_values_under_scores_that_climb(n, kernel, i8):
    """V of 2^100 and scores that climb by 20 (29 powers of two) over each context:
    the outputs are below 2^103.  So many contexts that most are walked from the
    first key to the last by one CTA."""
    T, Bt, Hq = 1440, 40, 16
    x = Paged([n] * Bt, [T] * Bt, Hq, 2, 128, 128, i8=i8)
    x.q[..., 0] = 8
    climb = torch.linspace(0, 20 * 128 ** 0.5 / 8, T).to(torch.bfloat16)
    for b in range(Bt):
        for j in range(-(-T // 128)):
            lo, hi = j * 128, min((j + 1) * 128, T)
            p = int(x.table[b, j])
            k = x.k[b][lo:hi] / 4
            k[..., 0] = climb[lo:hi, None]
            if i8:
                codes, sc = cache_ref.quantise(k)
                x.kp[p, :hi - lo], x.ks[p, :, :hi - lo] = codes.cuda(), sc.t().cuda()
                x.vs[p, :, :hi - lo] *= 2.0 ** 100
            else:
                x.kp[p, :hi - lo] = k.cuda()
                x.vp[p, :hi - lo] *= 2.0 ** 100
    out, lse = _run(x, kernel)
    seen = cache_bounds.visible(n, T)
    for b in range(Bt):
        for h in range(Hq):
            at = b * n
            want = cache_bounds.reference(x, b, at, h, seen, kernel)
            cache_ref.check(out[at:at + n, h], lse[at:at + n, h], *want, f"sequence {b} head {h}")
