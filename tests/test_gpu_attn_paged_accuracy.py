"""The split kernel of the attention over pages keeps its weights to 15 bits (bf16
pages) or 23 (int8 pages): the bounds are those of cache_bounds, which reject
weights rounded to bf16 (test_cache_bounds.py)."""
import pytest
import torch

import cache_bounds
import cache_ref
from cache_ref import Paged
from gpu_helpers import lib_ready

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("case", [
    # ns, ts, Hq, Hkv, d, block, window, sinks
    ([1] * 8, [1, 2, 5, 17, 40, 100, 130, 701], 16, 2, 128, 64, 0, 0),
    ([1] * 8, [1, 2, 5, 17, 40, 100, 130, 701], 16, 1, 64, 32, 0, 0),
    ([4, 3, 2], [40, 129, 300], 8, 2, 128, 128, 0, 0),
    ([1, 4], [3000, 260], 8, 2, 64, 64, 50, 4),
    ([30], [200], 8, 2, 128, 64, 0, 0),
    ([1], [20000], 8, 1, 128, 512, 0, 0),
], ids=range(6))
def test_split_kernel_keeps_its_weights(case, i8):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    ns, ts, Hq, Hkv, d, block, window, sinks = case
    x = Paged(ns, ts, Hq, Hkv, d, block, i8=i8, seed=7)
    assert cache_bounds.reaches(x, "split", window, sinks, max(ns))
    ws = msa.Workspace.for_cache(Hq, Hkv, d)
    call = msa.attn_paged_i8 if i8 else msa.attn_paged
    out, lse = call(x.q, *x.stores(), *x.step(), ws, window=window, sinks=sinks, max_q=max(ns))
    assert msa.device_status(ws) == 0
    at = 0
    for b, (n, t) in enumerate(zip(ns, ts)):
        seen = cache_bounds.visible(n, t, window, sinks)
        for h in range(Hq):
            want = cache_bounds.reference(x, b, at, h, seen, "split")
            cache_ref.check(out[at:at + n, h], lse[at:at + n, h], *want, f"sequence {b} head {h}")
        at += n


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("up", [10, 13, 16, 20])
@pytest.mark.parametrize("zero", [False, True])
def test_queries_with_one_large_value(zero, up, i8):
    """One value of q 2^up times the others, in a channel where K is zero or small:
    the others keep their share of the scores, to 20 bits below it on int8 pages."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([1, 3], [300, 129], 8, 2, 128, 64, i8=i8, seed=8)
    x.q[..., 5] *= 2.0 ** up
    x.kp[..., 5] = 0 if zero else (x.kp[..., 5] > 0).to(x.kp.dtype)  # 0 or 1, or NaN's 0 behind the contexts
    assert cache_bounds.reaches(x, "split", max_q=3)
    ws = msa.Workspace.for_cache(8, 2, 128)
    call = msa.attn_paged_i8 if i8 else msa.attn_paged
    out, lse = call(x.q, *x.stores(), *x.step(), ws, max_q=3)
    assert msa.device_status(ws) == 0
    at = 0
    for b, (n, t) in enumerate(zip(x.ns, x.ts)):
        seen = cache_bounds.visible(n, t)
        for h in range(8):
            want = cache_bounds.reference(x, b, at, h, seen, "split")
            cache_ref.check(out[at:at + n, h], lse[at:at + n, h], *want, f"sequence {b} head {h}")
        at += n
