"""V rows of very different sizes on int8 pages: a row of the cache has no
influence on queries that do not see it, or hardly weigh it, however large its
scale is.  The bounds count visible, weighted terms only (cache_bounds)."""
import pytest
import torch

import cache_bounds
import cache_ref
from cache_ref import Paged
from gpu_helpers import lib_ready

pytestmark = pytest.mark.gpu

# rows of one sequence, and the kernel that takes them (G 2, 2 kv heads, 700 keys and more)
ROWS = [(1, "split"), (4, "split"), (7, "split"), (1000, "chunk")]


def _check(x, kernel, ws=None):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    assert cache_bounds.reaches(x, kernel)
    ws = ws or msa.Workspace.for_cache(x.Hq, x.Hkv, x.d)
    out, lse = msa.attn_paged_i8(x.q, *x.stores(), *x.step(), ws)
    assert msa.device_status(ws) == 0
    at = 0
    for b, (n, t) in enumerate(zip(x.ns, x.ts)):
        seen = cache_bounds.visible(n, t)
        for h in range(x.Hq):
            want = cache_bounds.reference(x, b, at, h, seen, kernel)
            cache_ref.check(out[at:at + n, h], lse[at:at + n, h], *want, f"sequence {b} head {h}")
        at += n


def _at(x, b, j):
    return int(x.table[b, j // x.block]), j % x.block


@pytest.mark.parametrize("n, kernel", ROWS)
@pytest.mark.parametrize("up", [8, 20, 24, 28, 60])
def test_a_large_row_with_negligible_weight(n, kernel, up):
    """One V row 2^up times the others, on a key that no query weighs: its
    score lies some hundreds below the others'."""
    x = Paged([n], [n + 700], 4, 2, 128, 64, i8=True)
    x.q[..., 0] = 4
    p, r = _at(x, 0, 333)
    x.kp[p, r] = 0
    x.kp[p, r, :, 0] = -127
    x.ks[p, :, r] = 10.0
    x.vs[p, :, r] *= 2.0 ** up
    _check(x, kernel)


@pytest.mark.parametrize("n, kernel", ROWS[1:])
@pytest.mark.parametrize("up", [8, 20, 28, 60])
def test_a_large_row_that_earlier_rows_do_not_see(n, kernel, up):
    x = Paged([n], [n + 700], 4, 2, 128, 64, i8=True)
    p, r = _at(x, 0, n + 699)
    x.vs[p, :, r] *= 2.0 ** up
    _check(x, kernel)


@pytest.mark.parametrize("n, kernel", ROWS)
@pytest.mark.parametrize("down", [10, 30, 60])
def test_a_first_token_that_takes_the_weight(n, kernel, down):
    """The first key takes all but 2^-30 or so of the weight and its V row is
    zero, or 2^down times smaller than the others: the small weights make up the
    output, and stand in other tiles as well as in its own."""
    for zero in (False, True):
        x = Paged([n], [n + 700], 4, 2, 128, 64, i8=True)
        x.q[..., 0] = 4
        p, r = _at(x, 0, 0)
        x.kp[p, r] = 0
        x.kp[p, r, :, 0] = 127
        x.ks[p, :, r] = 0.55          # a score of 4 * 127 * 0.55 / sqrt(128) = 24.7
        x.vs[p, :, r] *= 0.0 if zero else 2.0 ** -down
        _check(x, kernel)


@pytest.mark.parametrize("n, kernel", ROWS)
def test_scales_of_all_sizes(n, kernel):
    """Scales from 2^-40 to 2^40, and zeros."""
    x = Paged([n, n], [n + 700, n + 350], 4, 2, 64, 32, i8=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    e = torch.randint(-40, 41, x.vs.shape, generator=g, device="cuda")
    x.vs.mul_(torch.exp2(e.float()))
    x.vs[torch.rand(x.vs.shape, generator=g, device="cuda") < 0.1] = 0
    _check(x, kernel)


@pytest.mark.parametrize("Hq", [2, 16])
def test_sparse_decode_with_a_large_row(Hq):
    """The sparse branch: a large V row of negligible weight among the selected
    blocks, 8 and 16 query rows."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    T = 1000
    x = Paged([1], [T], Hq, 1, 128, 64, i8=True)
    x.q[..., 0] = 4
    ids = torch.tensor([[[1, 3, 4, 15]]], dtype=torch.int32, device="cuda")
    p, r = _at(x, 0, 200)
    x.kp[p, r] = 0
    x.kp[p, r, :, 0] = -127
    x.ks[p, :, r] = 10.0
    x.vs[p, :, r] *= 2.0 ** 28
    ws = msa.Workspace.for_cache(Hq, 1, 128)
    out, lse = msa.sparse_attn_paged_i8(x.q[:, None], *x.stores(), x.table, T, ids, ws)
    assert msa.device_status(ws) == 0
    seen = torch.isin(torch.arange(T, device="cuda") // 64, ids[0, 0])[None]
    for h in range(Hq):
        want = cache_bounds.reference(x, 0, 0, h, seen, "split")
        cache_ref.check(out[0, :, h], lse[0, :, h], *want, f"head {h}")
