"""Attention over the paged cache (msa_attn_paged*, msa_sparse_attn_paged_i8)
against a plain 64-bit form.  Rows of the stores that no query may use hold
NaN, page tables are permuted, and the bounds are those of cache_ref."""
import pytest
import torch

import cache_ref
from cache_ref import Paged
from gpu_helpers import lib_ready

pytestmark = pytest.mark.gpu

BAD_IDS = 6


def _run(x, ws, **how):
    from block_sparse_long_05_b200 import msa
    call = msa.attn_paged_i8 if x.i8 else msa.attn_paged
    return call(x.q, *x.stores(), *x.step(), ws, **how)


def _both(x, window=0, sinks=0, **how):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    ws = msa.Workspace.for_cache(x.Hq, x.Hkv, x.d)
    out, lse = _run(x, ws, window=window, sinks=sinks, **how)
    st = msa.device_status(ws)
    assert st == 0, msa.status_string(st)
    rows = sum(x.ns)
    cache_ref.check(out[:rows], lse[:rows], *cache_ref.attn(x, window, sinks))
    return out, lse


CASES = [
    # ns, ts, Hq, Hkv, d, block, window, sinks
    ([1], [1], 1, 1, 64, 32, 0, 0),
    ([1], [4001], 8, 2, 64, 64, 0, 0),
    ([1, 1, 1], [1, 63, 4097], 16, 2, 128, 128, 0, 0),
    ([1] * 5, [64, 65, 127, 2000, 1], 48, 1, 128, 32, 0, 0),       # 48 heads of one kv head
    ([2, 3, 0, 1], [2, 700, 55, 129], 15, 3, 128, 64, 0, 0),        # 5 heads per kv head
    ([1], [20000], 8, 1, 128, 512, 0, 0),                           # one row over many runs
    ([1, 1], [900, 1800], 8, 2, 128, 128, 100, 0),
    ([1, 1], [900, 1800], 8, 2, 64, 64, 100, 5),
    ([1, 4], [5, 3000], 8, 2, 128, 32, 1, 0),                       # a window of the key itself
    ([3], [700], 8, 8, 128, 128, 64, 200),                          # more sinks than window
    ([1] * 300, [(7 * i) % 200 + 1 for i in range(300)], 4, 2, 64, 32, 0, 0),
    # chunks
    ([5], [5], 4, 4, 64, 64, 0, 0),
    ([65], [65], 8, 1, 128, 128, 0, 0),
    ([129, 1, 200], [400, 77, 200], 8, 2, 128, 128, 0, 0),
    ([333], [1500], 8, 2, 64, 32, 0, 0),
    ([260], [260], 16, 2, 128, 512, 0, 0),
    ([300, 40], [1024, 40], 12, 4, 128, 64, 0, 0),                  # 3 heads per kv head
    ([500], [900], 8, 2, 128, 128, 70, 3),
    ([700, 2], [700, 500], 4, 2, 64, 64, 256, 130),
    ([257], [2048], 8, 1, 128, 128, 1000, 64),
    ([150], [150], 4, 1, 128, 32, 1, 1),
    ([20, 64], [9, 64], 8, 2, 128, 64, 0, 0),                       # rows before position 0
    ([20, 64], [9, 64], 8, 2, 64, 64, 16, 2),
    ([700], [0], 8, 2, 64, 64, 0, 0),                               # no context at all
]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_matches_plain_form(case, i8):
    ns, ts, Hq, Hkv, d, block, window, sinks = case
    _both(Paged(ns, ts, Hq, Hkv, d, block, i8=i8, seed=len(ns)), window, sinks)


@pytest.mark.parametrize("i8", [False, True])
def test_large_scores(i8):
    # scores of several hundred: one key takes nearly all the weight
    _both(Paged([1, 200], [3000, 900], 8, 2, 128, 128, i8=i8, scale=30.0))


@pytest.mark.parametrize("max_q", [0, 1, 5, 400, 100000])
def test_hint_changes_no_result(max_q):
    _both(Paged([400, 1, 5], [800, 333, 100], 8, 2, 128, 64), max_q=max_q)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n", [1, 70])
def test_padded_batch_strides_and_given_outputs(n, i8):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([n, 1], [500, 80], 8, 2, 128, 64, i8=i8, pad_rows=9)
    wide = torch.zeros((x.total, 10, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = x.q
    x.q = wide[:, :8]
    out = torch.full((x.total, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.total, 8), 3.0, device="cuda")
    ws = msa.Workspace.for_cache(8, 2, 128)
    _run(x, ws, out=out, lse=lse)
    assert msa.device_status(ws) == 0
    cache_ref.check(out[:n + 1], lse[:n + 1], *cache_ref.attn(x))
    assert (out[n + 1:] == 3).all() and (lse[n + 1:] == 3).all()


def test_no_rows():
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([1], [40], 4, 2, 64, 32)
    ws = msa.Workspace.for_cache(4, 2, 64)
    out, lse = msa.attn_paged(x.q[:0], *x.stores(), x.table, torch.zeros_like(x.cu), x.kv_len, ws)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    msa.kv_append(torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda"),
                  torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda"), *x.stores(),
                  x.table, torch.zeros_like(x.cu), x.kv_len, ws)
    assert msa.device_status(ws) == 0


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, count", [(1, 900), (9, 300), (260, 24)])
def test_many_rows_without_keys(n, count, i8):
    """Long runs of row tiles that see nothing, with contexts between them."""
    ts = [0 if b % 7 else n + 130 for b in range(count)]
    ts[-1] = 0
    _both(Paged([n] * count, ts, 4, 2, 64, 64, i8=i8))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, Hkv", [(1, 2), (70, 3), (300, 5), (40, 6)])
def test_contexts_that_share_pages(n, Hkv, i8):
    """Several contexts with the same first pages, and one page twice in a table."""
    x = Paged([n, 5, n], [500, 450, 700], 2 * Hkv, Hkv, 64, 64, i8=i8)
    x.table[1, :5] = x.table[0, :5]
    x.table[2, 1] = x.table[2, 0]
    _both(x)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n", [1, 150])
def test_missing_pages(n, i8):
    """Keys of a page that does not exist are left out and reported."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([n], [500], 8, 2, 128, 64, i8=i8)
    ws = msa.Workspace.for_cache(8, 2, 128)
    gone = x.table.clone()
    gone[0, 2], gone[0, 4] = x.num_pages, -1
    good, x.table = x.table, gone
    out, lse = _run(x, ws)
    assert msa.device_status(ws) == BAD_IDS
    x.table = good
    k, v = x.context(0)
    j = torch.arange(500, device="cuda")[None]
    i = torch.arange(500 - n, 500, device="cuda")[:, None]
    seen = (j <= i) & (j // 64 != 2) & (j // 64 != 4)
    for h in range(8):
        o, l, a, s = cache_ref.attend(x.q[:, h].double(), k[:, h // 4], v[:, h // 4], seen)
        cache_ref.check(out[:, h], lse[:, h], o, l, *cache_ref.tolerances(o, l, a, s, 128))


def test_context_longer_than_its_table():
    from block_sparse_long_05_b200 import msa
    lib_ready()
    for n in (1, 150):
        x = Paged([n], [640], 8, 2, 128, 64)
        ws = msa.Workspace.for_cache(8, 2, 128)
        x.table = x.table[:, :10].contiguous()
        x.kv_len = torch.tensor([700], dtype=torch.int32, device="cuda")
        out, lse = _run(x, ws)
        assert msa.device_status(ws) == BAD_IDS
        k, v = x.context(0)
        j = torch.arange(640, device="cuda")[None]
        i = torch.arange(700 - n, 700, device="cuda")[:, None]
        for h in range(8):
            o, l, a, s = cache_ref.attend(x.q[:, h].double(), k[:, h // 4], v[:, h // 4], j <= i)
            cache_ref.check(out[:, h], lse[:, h], o, l, *cache_ref.tolerances(o, l, a, s, 128))


def test_dead_rows_of_shared_tiles():
    """Keys that the batch's rows cannot see hold NaN and infinities: past the
    context, and before the window of a single token."""
    x = Paged([1], [777], 8, 2, 128, 64)
    for pos in range(0, 777 - 100):
        if pos >= 3:
            p = int(x.table[0, pos // 64])
            x.kp[p, pos % 64] = float("nan")
            x.vp[p, pos % 64] = float("inf")
    from block_sparse_long_05_b200 import msa
    lib_ready()
    ws = msa.Workspace.for_cache(8, 2, 128)
    out, lse = _run(x, ws, window=100, sinks=3)
    assert msa.device_status(ws) == 0
    k, v = x.context(0)
    keep = torch.cat([torch.arange(3), torch.arange(677, 777)]).cuda()
    for h in range(8):
        kk, vv = k[keep, h // 4], v[keep, h // 4]
        o, l, a, s = cache_ref.attend(x.q[:, h].double(), kk, vv,
                                      torch.ones((1, 103), dtype=torch.bool, device="cuda"))
        cache_ref.check(out[:, h], lse[:, h], o, l, *cache_ref.tolerances(o, l, a, s, 128))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n", [1, 3, 100, 600])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_pages_before_the_window_may_be_gone(n, i8, block):
    """A page with no key in any row's window (nor a sink) is not looked up."""
    window, sinks, T = 150, 5, 1500
    x = Paged([n], [T], 8, 2, 128, block, i8=i8)
    first = T - n - window + 1  # the first key that the first row sees
    for j in range(1 + (sinks - 1) // block, max(first, 0) // block):
        x.table[0, j] = -1 if j % 2 else x.num_pages + 7
    keep = x.table.clone()
    good = Paged([n], [T], 8, 2, 128, block, i8=i8)
    x.table = good.table
    want = cache_ref.attn(x, window, sinks)
    x.table = keep
    from block_sparse_long_05_b200 import msa
    lib_ready()
    ws = msa.Workspace.for_cache(8, 2, 128)
    out, lse = _run(x, ws, window=window, sinks=sinks)
    assert msa.device_status(ws) == 0
    cache_ref.check(out, lse, *want)


@pytest.mark.parametrize("n", [1, 6, 300])
def test_rows_without_sound_scales(n):
    """A cached row that was not finite when it was written (scale NaN) reaches the
    queries that see it, and no others; a bad V row leaves lse as it is."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    T, j = 700, 650 if n > 100 else 700 - (n + 1) // 2
    for bad in ("v", "k"):
        x = Paged([n], [T], 8, 2, 128, 64, i8=True)
        want = cache_ref.attn(x)
        getattr(x, bad + "s")[int(x.table[0, j // 64]), :, j % 64] = float("nan")
        ws = msa.Workspace.for_cache(8, 2, 128)
        out, lse = _run(x, ws)
        assert msa.device_status(ws) == 0
        sees = torch.arange(T - n, T, device="cuda") >= j
        assert torch.isnan(out[sees]).all()
        if (~sees).any():
            cache_ref.check(out[~sees], lse[~sees], *(t[~sees] for t in want))
        if bad == "v":
            assert ((lse - want[1]).abs() <= want[3]).all()
        else:
            assert torch.isnan(lse[sees]).all()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n", [2, 300])
def test_keys_of_later_tokens_may_be_anything(n, i8):
    """K of a token that a query may not see has no influence, whatever it holds."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([n], [500], 8, 2, 128, 64, i8=i8)
    want = cache_ref.attn(x)
    p, r = int(x.table[0, 499 // 64]), 499 % 64
    if i8:
        x.ks[p, :, r] = float("inf")
    else:
        x.kp[p, r] = float("nan")
    ws = msa.Workspace.for_cache(8, 2, 128)
    out, lse = _run(x, ws)
    cache_ref.check(out[:-1], lse[:-1], *(t[:-1] for t in want))


@pytest.mark.parametrize("i8", [False, True])
def test_scores_that_leap(i8):
    """Scores that rise by hundreds from one key tile to the next: the weights'
    reference is raised again and again, in every row apart."""
    x = Paged([1, 300], [1400, 1400], 8, 2, 128, 128, i8=i8, scale=0.0)
    g = torch.Generator().manual_seed(9)
    for b in range(2):
        grow = torch.linspace(0, 60, 1400)[:, None, None]
        k = (torch.randn((1400, 2, 128), generator=g) * grow).to(torch.bfloat16)
        for j in range(-(-1400 // 128)):
            lo, hi = j * 128, min((j + 1) * 128, 1400)
            p = int(x.table[b, j])
            if i8:
                codes, sc = cache_ref.quantise(k[lo:hi])
                x.kp[p, :hi - lo], x.ks[p, :, :hi - lo] = codes.cuda(), sc.t().cuda()
            else:
                x.kp[p, :hi - lo] = k[lo:hi].cuda()
    _both(x)


def test_repeats_bit_for_bit():
    from block_sparse_long_05_b200 import msa
    lib_ready()
    for ns, ts in (([1, 1, 1], [9000, 31, 2500]), ([300, 20], [4000, 900])):
        x = Paged(ns, ts, 16, 2, 128, 128)
        ws = msa.Workspace.for_cache(16, 2, 128)
        first = _run(x, ws)
        for _ in range(3):
            again = _run(x, ws)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_other_stream_and_captured_steps():
    """A captured step follows the lengths and pages that its buffers hold when
    it is replayed; two steps on two streams do not share a workspace."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    for n in (1, 100):
        x = Paged([n, n], [900, 300], 8, 2, 128, 64)
        y = Paged([n, n], [100, 1200], 8, 2, 128, 64, seed=5)
        want_x, want_y = cache_ref.attn(x), cache_ref.attn(y)
        wx, wy = (msa.Workspace.for_cache(8, 2, 128) for _ in range(2))
        sx, sy = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(3):
            ox = _run(x, wx, stream=sx)
            oy = _run(y, wy, stream=sy)
        sx.synchronize()
        sy.synchronize()
        cache_ref.check(*ox, *want_x)
        cache_ref.check(*oy, *want_y)
        # one captured step over buffers that then take the other batch's contents
        pages = max(x.num_pages, y.num_pages)
        width = max(x.table.shape[1], y.table.shape[1])
        q = x.q.clone()
        kp = torch.zeros((pages, 64, 2, 128), dtype=torch.bfloat16, device="cuda")
        vp = torch.zeros_like(kp)
        table = torch.zeros((2, width), dtype=torch.int32, device="cuda")
        kv_len = x.kv_len.clone()
        out = torch.empty((2 * n, 8, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((2 * n, 8), device="cuda")
        ws = msa.Workspace.for_cache(8, 2, 128)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            msa.attn_paged(q, kp, vp, table, x.cu, kv_len, ws, out=out, lse=lse)
        for z, want in ((x, want_x), (y, want_y), (x, want_x)):
            q.copy_(z.q)
            kp[:z.num_pages], vp[:z.num_pages] = z.kp, z.vp
            table[:, :z.table.shape[1]] = z.table
            kv_len.copy_(z.kv_len)
            graph.replay()
            torch.cuda.synchronize()
            cache_ref.check(out, lse, *want)
        assert msa.device_status(ws) == 0
        del graph


def test_outputs_made_on_a_given_stream():
    """Outputs of a call on a given stream do not take memory that work queued on
    the current stream still uses."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([1, 200], [300, 900], 8, 2, 128, 64)
    ws = msa.Workspace.for_cache(8, 2, 128)
    want = [t.clone() for t in _run(x, ws)]
    side = torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        kept = torch.full_like(want[0], 3.0)
        busy = torch.full((1 << 27,), 1.0, device="cuda")
        for _ in range(20):
            busy += 1
        copy = kept + busy[0].to(torch.bfloat16) * 0  # reads `kept` late
        shape = kept.shape
        del kept  # its memory is free for the current stream only
        got = _run(x, ws, stream=side)
        torch.cuda.synchronize()
        assert got[0].shape == shape
        assert (copy == 3).all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert msa.device_status(ws) == 0


def test_store_past_32_bits():
    """Keys at the end of stores of more than 2^31 codes."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    Hkv, d, block = 8, 128, 512
    x = Paged([1, 100], [1500, 1024], 16, Hkv, d, block, i8=True)
    pages = (1 << 31) // (block * Hkv * d) + x.num_pages
    shift = pages - x.num_pages
    big = []
    for t in (x.kp, x.vp):
        y = torch.zeros((pages, block, Hkv, d), dtype=torch.int8, device="cuda")
        y[shift:] = t
        big.append(y)
    for t in (x.ks, x.vs):
        y = torch.zeros((pages, Hkv, block), device="cuda")
        y[shift:] = t
        big.append(y)
    ws = msa.Workspace.for_cache(16, Hkv, d)
    table = torch.where(x.table >= 0, x.table + shift, x.table)
    out, lse = msa.attn_paged_i8(x.q, *big, table, x.cu, x.kv_len, ws)
    assert msa.device_status(ws) == 0
    cache_ref.check(out, lse, *cache_ref.attn(x))
    del big
    torch.cuda.empty_cache()


def test_binding_refusals():
    """Types, shapes and strides that the binding refuses, before any launch."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([2], [100], 8, 2, 128, 64, i8=True)
    ws = msa.Workspace.for_cache(8, 2, 128)

    def attend(**ch):
        a = dict(q=x.q, kp=x.kp, vp=x.vp, ks=x.ks, vs=x.vs, table=x.table, cu=x.cu, kv_len=x.kv_len)
        how = {k: ch.pop(k) for k in list(ch) if k in ("out", "lse", "window", "max_q")}
        a.update(ch)
        return msa.attn_paged_i8(*a.values(), ws, **how)

    good = attend()
    for ch in (dict(q=x.q.float()), dict(q=x.q[0]), dict(q=x.q[:, :, :64]), dict(q=x.q.transpose(0, 1)),
               dict(kp=x.kp.float()), dict(kp=x.kp[:, ::2]), dict(vp=x.vp[1:]), dict(ks=x.ks[:, :1]),
               dict(vs=x.vs.double()), dict(table=x.table.long()), dict(table=x.table[0]),
               dict(table=x.table[:, ::2]), dict(cu=x.cu[:1]), dict(kv_len=x.cu), dict(kv_len=x.kv_len.cpu()),
               dict(out=good[0].float()), dict(out=good[0][:1]), dict(lse=good[1][:, :4]), dict(window=1 << 40)):
        with pytest.raises(ValueError):
            attend(**ch)
    for ch in (dict(window=-1), dict(max_q=-3)):
        with pytest.raises(msa.MSAError):
            attend(**ch)
    assert msa.device_status(ws) == 0


# ------------------------------------------------------------------ sparse branch
@pytest.mark.parametrize("case", [
    # Bt, T, Hq, Hkv, d, block, K
    (3, 1000, 8, 2, 64, 64, 4),
    (2, 4096, 16, 2, 128, 128, 8),
    (2, 5000, 16, 4, 128, 512, 4),
    (2, 50, 8, 8, 64, 64, 4),          # fewer blocks than K
    (1, 2000, 4, 1, 64, 32, 31),       # an odd number of 32-key blocks
    (1, 2001, 40, 1, 128, 32, 8),      # 40 heads per kv head
    (70, 300, 6, 2, 128, 128, 2),      # 3 heads per kv head
])
def test_sparse_decode_i8(case):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    Bt, T, Hq, Hkv, d, block, K = case
    x = Paged([1] * Bt, [T] * Bt, Hq, Hkv, d, block, i8=True, seed=K)
    N = -(-T // block)
    g = torch.Generator().manual_seed(K)
    ids = torch.full((Bt, 1, K), -1, dtype=torch.int32)
    for b in range(Bt):
        if b % 5 == 4:
            continue  # nothing selected
        m = min(K, N)
        ids[b, 0, :m] = torch.randperm(N, generator=g)[:m].sort().values.to(torch.int32)
    ids = ids.cuda()
    ws = msa.Workspace.for_cache(Hq, Hkv, d)
    out, lse = msa.sparse_attn_paged_i8(x.q[:, None], *x.stores(), x.table, T, ids, ws)
    assert msa.device_status(ws) == 0
    G = Hq // Hkv
    for b in range(Bt):
        k, v = x.context(b)
        blocks = torch.arange(T, device="cuda") // block
        seen = torch.isin(blocks, ids[b, 0])[None]
        for h in range(Hq):
            o, l, a, s = cache_ref.attend(x.q[b:b + 1, h].double(), k[:, h // G], v[:, h // G], seen)
            cache_ref.check(out[b, :, h], lse[b, :, h], o, l, *cache_ref.tolerances(o, l, a, s, d), f"{b} {h}")


def test_sparse_decode_i8_bad_ids():
    from block_sparse_long_05_b200 import msa
    lib_ready()
    x = Paged([1], [1000], 8, 2, 64, 64, i8=True)
    ws = msa.Workspace.for_cache(8, 2, 64)
    good = torch.tensor([[[1, 3, 15, -1]]], dtype=torch.int32, device="cuda")
    want = msa.sparse_attn_paged_i8(x.q[:, None], *x.stores(), x.table, 1000, good, ws)
    assert msa.device_status(ws) == 0
    bad = torch.tensor([[[1, 3, 15, 16]]], dtype=torch.int32, device="cuda")
    got = msa.sparse_attn_paged_i8(x.q[:, None], *x.stores(), x.table, 1000, bad, ws)
    assert msa.device_status(ws) == BAD_IDS
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ together
def test_serving_run():
    """Prompt, chunk and single tokens through append, attention and the sparse
    branch, and the cache read back for the contiguous calls: on bf16 pages and
    on int8 ones, each step against the plain form over what the cache holds."""
    from block_sparse_long_05_b200 import msa
    lib_ready()
    Hq, Hkv, d, block, K, d_idx = 8, 2, 128, 64, 4, 64
    ws = msa.Workspace.for_cache(Hq, Hkv, d)
    for i8 in (False, True):
        x = Paged([0, 0], [640, 640], Hq, Hkv, d, block, i8=i8, poison=float("nan"))
        if i8:
            x.ks.fill_(float("nan"))
            x.vs.fill_(float("nan"))
        else:
            x.kp.fill_(float("nan"))
            x.vp.fill_(float("nan"))
        xp = torch.full((x.num_pages, block, d_idx), 50.0, dtype=torch.bfloat16, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(2)
        lens, index = [0, 0], [[], []]
        for ns in ([300, 17], [100, 250], [1, 1], [1, 1]):
            lens = [a + n for a, n in zip(lens, ns)]
            x.ns, x.ts, x.total = ns, lens, sum(ns)
            x.cu = torch.tensor([0, ns[0], sum(ns)], dtype=torch.int32, device="cuda")
            x.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
            qkv = torch.randn((x.total, Hq + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
            x.q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            k_idx = torch.randint(-3, 4, (x.total, d_idx), generator=g, device="cuda").to(torch.bfloat16)
            for b in range(2):
                index[b].append(k_idx[x.cu[b]:x.cu[b + 1]])
            append = msa.kv_append_i8 if i8 else msa.kv_append
            append(k, v, *x.stores(), *x.step(), ws, k_idx=k_idx, k_idx_pages=xp)
            out, lse = _run(x, ws, max_q=max(ns))
            assert msa.device_status(ws) == 0
            cache_ref.check(out, lse, *cache_ref.attn(x), f"step {ns}")
            out, lse = _run(x, ws, window=64, sinks=4, max_q=max(ns))
            cache_ref.check(out, lse, *cache_ref.attn(x, 64, 4), f"window step {ns}")
        # the first sequence's sparse decode step over the same pages
        T = lens[0]
        q_idx = torch.randint(-3, 4, (1, 1, d_idx), generator=g, device="cuda").to(torch.bfloat16)
        mws = msa.Workspace.for_shape(1, 1, T, Hq, Hkv, d, d_idx, block, K)
        ids = msa.index_topk_paged(q_idx, xp, x.table[:1], T, K, mws)
        flat = torch.cat(index[0])[None].contiguous()
        assert torch.equal(ids, msa.index_topk(q_idx, flat, block, K, mws))
        q1 = x.q[:1][None].contiguous()
        cu1 = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        read = msa.kv_gather_i8 if i8 else msa.kv_gather
        kk, vv = read(*x.stores(), x.table[:1], cu1, x.kv_len[:1], T, ws)
        want, wlse = msa.sparse_attn(q1, kk[None], vv[None], ids, block, mws)
        if i8:
            got, glse = msa.sparse_attn_paged_i8(q1, *x.stores(), x.table[:1], T, ids, ws)
        else:
            got, glse = msa.sparse_attn_paged(q1, *x.stores(), x.table[:1], T, ids, mws)
        assert msa.device_status(ws) == 0 and msa.device_status(mws) == 0
        # the contiguous call reads rows rounded to bf16 and rounds its weights:
        # three relative errors of 2^-8 on terms whose weighted size is below max |v|
        bound = 4 * cache_ref.BF16 * vv.float().abs().max().item()
        assert (got.float() - want).abs().max().item() <= bound
        # scores move by at most 2^-8 of the sum of |q_i k_i| / sqrt(d)
        size = (q1[0, 0].float().abs().max() * kk.float().abs().sum(-1).max() / d ** 0.5).item()
        assert (glse - wlse).abs().max().item() <= cache_ref.BF16 * size
