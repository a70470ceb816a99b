"""The paged cache written and read back (msa_kv_append*, msa_kv_gather*)
against the documented formulas: codes, scales and copies are equal bit for
bit, and everything that no row maps to stays as it was."""
import pytest
import torch

from cache_ref import Paged, quantise
from gpu_helpers import lib_ready

pytestmark = pytest.mark.gpu

BAD_IDS = 6


def _ws(Hq=8, Hkv=8, d=128):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    return msa.Workspace.for_cache(Hq, Hkv, d)


def _new_rows(x, pad, stride_extra, seed=3):
    """New rows k, v of x's contexts as parts of one wide projection output."""
    g = torch.Generator().manual_seed(seed)
    width = x.Hkv * x.d
    wide = torch.randn((x.total, 2 * width + stride_extra), generator=g).to(torch.bfloat16).cuda()
    k = wide[:, :width].unflatten(1, (x.Hkv, x.d))
    v = wide[:, width:2 * width].unflatten(1, (x.Hkv, x.d))
    if not stride_extra and not pad:
        k, v = k.contiguous(), v.contiguous()
    return k, v


def _expect(x, k, v, k_idx, xpages):
    """The stores after the append, row by row of positions."""
    kp, vp = x.kp.clone(), x.vp.clone()
    ks, vs = (x.ks.clone(), x.vs.clone()) if x.i8 else (None, None)
    xp = xpages.clone() if xpages is not None else None
    at = 0
    for b, (n, t) in enumerate(zip(x.ns, x.ts)):
        for pos in range(t - n, t):
            if pos >= 0:
                p, r = int(x.table[b, pos // x.block]), pos % x.block
                for rows, pages, scales in ((k, kp, ks), (v, vp, vs)):
                    if x.i8:
                        pages[p, r], scales[p, :, r] = quantise(rows[at])
                    else:
                        pages[p, r] = rows[at]
                if xp is not None:
                    xp[p, r] = k_idx[at]
            at += 1
    return kp, vp, ks, vs, xp


def _same(a, b, what):
    if a is None:
        return
    if a.is_floating_point():
        assert torch.equal(torch.isnan(a), torch.isnan(b)), f"{what}: NaN places"
        a, b = a.nan_to_num(), b.nan_to_num()
    assert torch.equal(a, b), what


CASES = [
    # ns, ts, Hkv, d, block, d_idx, pad, stride_extra
    ([1], [1], 1, 64, 32, 0, 0, 0),
    ([1] * 7, [1, 128, 129, 5, 640, 300, 77], 8, 128, 128, 128, 0, 0),
    ([33, 0, 70, 1], [33, 40, 199, 200], 2, 64, 64, 64, 5, 8),
    ([257, 300], [1000, 300], 3, 128, 512, 64, 1, 16),
    ([40, 2], [7, 9], 4, 128, 32, 128, 0, 0),   # more rows than positions
    ([5] * 300, [17] * 300, 2, 64, 32, 64, 3, 0),
]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_append_and_gather(case, i8):
    from block_sparse_long_05_b200 import msa
    ns, ts, Hkv, d, block, d_idx, pad, extra = case
    ws = _ws()
    x = Paged(ns, ts, Hkv, Hkv, d, block, i8=i8, pad_rows=pad, poison=1.5)
    k, v = _new_rows(x, pad, extra)
    index, xp, k_idx = {}, None, None
    if d_idx:
        k_idx = torch.randint(-3, 4, (x.total, d_idx + 8)).to(torch.bfloat16).cuda()[:, :d_idx]
        xp = torch.full((x.num_pages, block, d_idx), 9.0, dtype=torch.bfloat16, device="cuda")
        index = dict(k_idx=k_idx, k_idx_pages=xp)
    want = _expect(x, k, v, k_idx, xp)
    call = msa.kv_append_i8 if i8 else msa.kv_append
    call(k, v, *x.stores(), *x.step(), ws, **index)
    assert msa.device_status(ws) == 0
    for got, exp, what in zip((x.kp, x.vp, x.ks, x.vs, xp), want, ("k", "v", "ks", "vs", "index")):
        _same(got, exp, what)

    gk = torch.full((x.total, Hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    gv = gk.clone()
    read = msa.kv_gather_i8 if i8 else msa.kv_gather
    read(*x.stores(), *x.step(), x.total, ws, k=gk, v=gv)
    assert msa.device_status(ws) == 0
    at = 0
    for b, (n, t) in enumerate(zip(ns, ts)):
        kk, vv = x.context(b)
        for i in range(n):
            pos = t - n + i
            for got, ctx in ((gk, kk), (gv, vv)):
                want_row = torch.zeros_like(ctx[:1])[0] if pos < 0 else ctx[pos]
                assert torch.equal(got[at], want_row.float().to(torch.bfloat16)), (b, pos)
            at += 1
    assert (gk[at:] == 5).all() and (gv[at:] == 5).all(), "rows behind the last sequence"


@pytest.mark.parametrize("i8", [False, True])
def test_gather_into_outputs_that_begin_on_16_bytes(i8):
    """Outputs that begin on 16 bytes but not on 32 get the same rows."""
    from block_sparse_long_05_b200 import msa
    ws = _ws()
    x = Paged([77, 50], [130, 60], 2, 2, 64, 32, i8=i8)
    read = msa.kv_gather_i8 if i8 else msa.kv_gather
    k, v = read(*x.stores(), *x.step(), x.total, ws)
    for off_k, off_v in ((8, 0), (0, 8), (8, 24)):
        bufs = [torch.full((x.total * 2 * 64 + 32,), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        outs = [b[o:o + k.numel()].view(k.shape) for b, o in zip(bufs, (off_k, off_v))]
        read(*x.stores(), *x.step(), x.total, ws, k=outs[0], v=outs[1])
        assert msa.device_status(ws) == 0
        assert torch.equal(outs[0], k) and torch.equal(outs[1], v)
        for b, o in zip(bufs, (off_k, off_v)):
            assert (b[:o] == 5).all() and (b[o + k.numel():] == 5).all(), "around the output"


def test_quantised_rows_that_are_special():
    """Zero rows, rows near the smallest values, single large values, and rows
    with an infinity or a NaN; a row's error is at most half a step."""
    from block_sparse_long_05_b200 import msa
    ws = _ws()
    x = Paged([64], [64], 2, 2, 128, 64, i8=True, poison=0.0)
    k, v = _new_rows(x, 0, 0)
    k[0] = 0
    k[1] = 1e-38
    k[2] = 2.0 ** -99
    k[3, 0, 5] = 3e38
    k[4, 1, 7] = float("inf")
    k[5, 0, 127] = float("nan")
    k[6, 0, 0] = -float("inf")
    k[7] = -1
    v[8] = -0.0
    want = _expect(x, k, v, None, None)
    msa.kv_append_i8(k, v, *x.stores(), *x.step(), ws)
    assert msa.device_status(ws) == 0
    for got, exp, what in zip((x.kp, x.vp, x.ks, x.vs), want, ("k", "v", "ks", "vs")):
        _same(got, exp, what)
    gk, gv = msa.kv_gather_i8(*x.stores(), *x.step(), 64, ws)
    for row, head in ((4, 1), (5, 0), (6, 0)):
        assert torch.isnan(gk[row, head]).all()
    fine = torch.isfinite(k).all(-1) & (k.abs().amax(-1) >= 2.0 ** -100)
    # half a step of the code, the rounding of inv (2^-23 of the value) and of the bf16 result
    step = k.double().abs().amax(-1, keepdim=True) / 254
    bound = step + k.double().abs() * 2.0 ** -22 + gk.double().abs() * 2.0 ** -8
    assert ((gk.double() - k.double()).abs() <= bound)[fine].all()
    assert (gk[0] == 0).all() and (gk[1] == 0).all()


def test_missing_pages_are_skipped_and_reported():
    from block_sparse_long_05_b200 import msa
    ws = _ws()
    for i8 in (False, True):
        x = Paged([100, 3], [100, 50], 2, 2, 64, 32, i8=i8, poison=2.0)
        x.table[0, 1] = x.num_pages + 4
        x.table[1, 1] = -3  # rows 47..49 of sequence 1: positions 47, 48, 49 are in page 1
        k, v = _new_rows(x, 0, 0)
        before = [t.clone() for t in x.stores()]
        append = msa.kv_append_i8 if i8 else msa.kv_append
        append(k, v, *x.stores(), *x.step(), ws)
        assert msa.device_status(ws) == BAD_IDS
        assert msa.device_status(ws) == 0
        for j in (0, 2, 3):
            p, rows = int(x.table[0, j]), min(32, 100 - 32 * j)
            assert not torch.equal(x.kp[p, :rows], before[0][p, :rows])
        touched = {int(x.table[0, j]) for j in (0, 2, 3)}
        for p in set(range(x.num_pages)) - touched:
            for now, was in zip(x.stores(), before):
                assert torch.equal(now[p], was[p])
        read = msa.kv_gather_i8 if i8 else msa.kv_gather
        gk, gv = read(*x.stores(), *x.step(), x.total, ws)
        assert msa.device_status(ws) == BAD_IDS
        assert (gk[32:64] == 0).all() and (gv[32:64] == 0).all() and (gk[100:] == 0).all()
        # a context that its page-table row cannot hold
        x = Paged([4], [60], 2, 2, 64, 32, i8=i8, poison=2.0)
        before = [t.clone() for t in x.stores()]
        long = torch.tensor([4000], dtype=torch.int32, device="cuda")
        append(k[:4], v[:4], *x.stores(), x.table, x.cu, long, ws)
        assert msa.device_status(ws) == BAD_IDS
        assert all(torch.equal(a, b) for a, b in zip(before, x.stores()))


def test_store_rows_past_32_bits():
    """The last pages of stores of more than 2^31 values, and more than 2^32 bytes."""
    from block_sparse_long_05_b200 import msa
    ws = _ws()
    Hkv, d, block = 8, 128, 512
    pages = (1 << 31) // (block * Hkv * d) + 8
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3 * block], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([3 * block], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((3 * block, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((3 * block, Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    kp = torch.zeros((pages, block, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    msa.kv_append(k, v, kp, vp, table, cu, kv_len, ws)
    for j in range(3):
        assert torch.equal(kp[int(table[0, j])], k[j * block:(j + 1) * block])
        assert torch.equal(vp[int(table[0, j])], v[j * block:(j + 1) * block])
    gk, gv = msa.kv_gather(kp, vp, table, cu, kv_len, 3 * block, ws)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    del kp, vp
    torch.cuda.empty_cache()
