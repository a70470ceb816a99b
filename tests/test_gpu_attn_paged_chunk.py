"""The chunk kernel of the attention over pages where it can go wrong.  Each case
first makes sure that its step reaches that kernel (small steps go to the split
kernel whatever their rows)."""
import pytest
import torch

import cache_bounds
import cache_ref
from cache_ref import Paged
from gpu_helpers import lib_ready

pytestmark = pytest.mark.gpu

BAD_IDS = 6


def _run(x, ws, window=0, sinks=0, **how):
    from block_sparse_long_05_b200 import msa
    assert cache_bounds.reaches(x, "chunk", window, sinks, how.get("max_q"))
    call = msa.attn_paged_i8 if x.i8 else msa.attn_paged
    return call(x.q, *x.stores(), *x.step(), ws, window=window, sinks=sinks, **how)


def _ws(x):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    return msa.Workspace.for_cache(x.Hq, x.Hkv, x.d)


def _compare(x, out, lse, window=0, sinks=0, context=None, what=""):
    """Every sequence against the 64-bit form.  context: (K, V) of each, if the
    store no longer holds them as they count."""
    at = 0
    G = x.Hq // x.Hkv
    for b, (n, t) in enumerate(zip(x.ns, x.ts)):
        k, v = context[b] if context else x.context(b)
        seen = cache_bounds.visible(n, t, window, sinks)
        for h in range(x.Hq):
            _head(x.q[at:at + n, h], k[:, h // G], v[:, h // G], seen, out[at:at + n, h],
                  lse[at:at + n, h], f"{what} sequence {b} head {h}")
        at += n


def _head(q, k, v, seen, out, lse, what):
    if not len(q):
        return
    o, l = cache_ref.attend(q.double(), k, v, seen)[:2]
    cache_ref.check(out, lse, o, l, *cache_bounds.bounds(q.double(), k, v, seen, "chunk"), what)


CASES = [
    # ns, ts, Hq, Hkv, d, block, window, sinks
    ([600, 1, 700], [900, 77, 700], 8, 2, 128, 128, 0, 0),
    ([1500], [1900], 8, 2, 128, 128, 70, 3),
    ([1500, 2], [1500, 500], 4, 2, 64, 64, 256, 130),
    ([1500], [0], 8, 2, 64, 64, 0, 0),                       # no context at all
    ([620, 64], [300, 64], 8, 2, 128, 64, 0, 0),             # rows before position 0
    ([620, 64], [300, 64], 8, 2, 64, 64, 16, 2),
    ([900], [900], 15, 3, 128, 64, 0, 0),                    # 5 heads per kv head
    ([2, 800], [2, 1000], 48, 1, 128, 32, 0, 0),             # 48 heads of one kv head
    ([1300], [1300], 8, 8, 64, 32, 1, 0),                    # a window of the key itself
    ([1111], [1111], 4, 2, 128, 512, 300, 5000),             # more sinks than keys
]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_matches_plain_form(case, i8):
    from block_sparse_long_05_b200 import msa
    ns, ts, Hq, Hkv, d, block, window, sinks = case
    x = Paged(ns, ts, Hq, Hkv, d, block, i8=i8, seed=len(ns))
    ws = _ws(x)
    out, lse = _run(x, ws, window, sinks)
    assert msa.device_status(ws) == 0
    _compare(x, out, lse, window, sinks)


@pytest.mark.parametrize("i8", [False, True])
def test_padded_batch_strides_and_given_outputs(i8):
    from block_sparse_long_05_b200 import msa
    n = 601
    x = Paged([n, 1], [1500, 80], 8, 2, 128, 64, i8=i8, pad_rows=9)
    wide = torch.zeros((x.total, 10, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:9] = x.q
    x.q = wide[:, 1:9]
    out = torch.full((x.total, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.total, 8), 3.0, device="cuda")
    ws = _ws(x)
    _run(x, ws, out=out, lse=lse)
    assert msa.device_status(ws) == 0
    _compare(x, out, lse)
    assert (out[n + 1:] == 3).all() and (lse[n + 1:] == 3).all()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_missing_pages(i8, block):
    """Keys of a page that does not exist are left out and reported."""
    from block_sparse_long_05_b200 import msa
    n, T = 700, 1400
    x = Paged([n], [T], 8, 2, 128, block, i8=i8)
    ws = _ws(x)
    gone = [2, 4, T // block]
    good, x.table = x.table, x.table.clone()
    x.table[0, gone[0]], x.table[0, gone[1]], x.table[0, gone[2]] = x.num_pages, -1, -2 ** 31
    out, lse = _run(x, ws)
    assert msa.device_status(ws) == BAD_IDS
    x.table = good
    k, v = x.context(0)
    there = ~torch.isin(torch.arange(T, device="cuda") // block, torch.tensor(gone, device="cuda"))
    for h in range(8):
        _head(x.q[:, h], k[:, h // 4], v[:, h // 4], cache_bounds.visible(n, T) & there, out[:, h],
              lse[:, h], f"head {h}")


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("kv_len", [1281, 1500, 1279 + 800])
def test_context_longer_than_its_table(i8, kv_len):
    from block_sparse_long_05_b200 import msa
    n, cap = 800, 1280
    x = Paged([n], [cap], 8, 2, 128, 64, i8=i8)
    x.table = x.table[:, :cap // 64].contiguous()
    x.kv_len = torch.tensor([kv_len], dtype=torch.int32, device="cuda")
    ws = _ws(x)
    out, lse = _run(x, ws)
    assert msa.device_status(ws) == BAD_IDS
    k, v = x.context(0)
    for h in range(8):
        _head(x.q[:, h], k[:, h // 4], v[:, h // 4], cache_bounds.visible(n, kv_len, cap=cap),
              out[:, h], lse[:, h], f"head {h}")


@pytest.mark.parametrize("window, sinks", [(0, 0), (333, 0), (333, 5)])
def test_rows_without_sound_scales(window, sinks):
    """A cached row that was not finite when it was written (scale NaN) reaches the
    queries that see it, and no others; a bad V row leaves lse as it is."""
    from block_sparse_long_05_b200 import msa
    n, T = 700, 1400
    for j in (2, 650, 1100, T - 1):
        for bad in ("v", "k"):
            x = Paged([n], [T], 8, 2, 128, 64, i8=True)
            context = [x.context(0)]
            getattr(x, bad + "s")[int(x.table[0, j // 64]), :, j % 64] = float("nan")
            ws = _ws(x)
            out, lse = _run(x, ws, window, sinks)
            assert msa.device_status(ws) == 0
            seen = cache_bounds.visible(n, T, window, sinks)
            sees = seen[:, j]
            assert torch.isnan(out[sees]).all()
            k, v = context[0]
            for h in range(8):
                if (~sees).any():
                    _head(x.q[~sees, h], k[:, h // 4], v[:, h // 4], seen[~sees], out[~sees, h],
                          lse[~sees, h], f"{bad} {j} head {h}")
                if bad == "v" and sees.any():
                    l = cache_ref.attend(x.q[sees, h].double(), k[:, h // 4], v[:, h // 4], seen[sees])[1]
                    t = cache_bounds.bounds(x.q[sees, h].double(), k[:, h // 4], v[:, h // 4],
                                            seen[sees], "chunk")[1]
                    assert ((lse[sees, h] - l).abs() <= t).all()
            if bad == "k":
                assert torch.isnan(lse[sees]).all()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_keys_of_later_tokens_may_be_anything(i8, value):
    """K of a token that a query may not see has no influence, whatever it holds."""
    from block_sparse_long_05_b200 import msa
    n, T = 700, 1400
    for j in (T - n + 1, T - 300, T - 1):
        x = Paged([n], [T], 8, 2, 128, 64, i8=i8)
        k, v = x.context(0)
        p, r = int(x.table[0, j // 64]), j % 64
        if i8:
            x.ks[p, :, r] = value
        else:
            x.kp[p, r] = value
        ws = _ws(x)
        out, lse = _run(x, ws)
        assert msa.device_status(ws) == 0
        m = n - (T - j)  # rows before token j
        seen = cache_bounds.visible(n, T)[:m]
        for h in range(8):
            _head(x.q[:m, h], k[:, h // 4], v[:, h // 4], seen, out[:m, h], lse[:m, h], f"{j} head {h}")


@pytest.mark.parametrize("i8", [False, True])
def test_dead_rows_of_tiles_that_are_read(i8):
    """Keys that no row of the step sees hold NaN and infinities: past the
    contexts (as in every case), and between the sinks and the first window."""
    from block_sparse_long_05_b200 import msa
    n, T, window, sinks = 700, 1400, 100, 3
    x = Paged([n], [T], 8, 2, 128, 64, i8=i8)
    context = [x.context(0)]
    for pos in range(sinks, T - n - window + 1):
        p, r = int(x.table[0, pos // 64]), pos % 64
        if i8:
            x.ks[p, :, r], x.vs[p, :, r] = float("nan"), float("inf")
        else:
            x.kp[p, r], x.vp[p, r] = float("nan"), float("inf")
    ws = _ws(x)
    out, lse = _run(x, ws, window, sinks)
    assert msa.device_status(ws) == 0
    _compare(x, out, lse, window, sinks, context)


@pytest.mark.parametrize("i8", [False, True])
def test_other_streams_and_captured_steps(i8):
    """A captured step (the chunk kernel, its merge, and the split kernel behind
    them) follows the lengths and pages that its buffers hold when it is replayed,
    down to steps without a row for the chunk kernel; two steps on two streams do
    not share a workspace."""
    from block_sparse_long_05_b200 import msa
    batches = [Paged(ns, ts, 8, 2, 128, 64, i8=i8, seed=s) for s, (ns, ts) in enumerate([
        ([600, 1, 299], [2900, 300, 900]), ([300, 300, 300], [301, 2999, 1500]),
        ([898, 1, 1], [898, 40, 2000]), ([1, 2, 3], [2000, 1, 1500])])]
    x, y = batches[:2]
    wx, wy = _ws(x), _ws(y)
    sx, sy = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        ox = _run(x, wx, stream=sx)
        oy = _run(y, wy, stream=sy)
    sx.synchronize()
    sy.synchronize()
    _compare(x, *ox)
    _compare(y, *oy)
    rows, pages = 900, max(z.num_pages for z in batches)
    width = max(z.table.shape[1] for z in batches)
    g = Paged([900, 0, 0], [64 * (width - 1), 0, 0], 8, 2, 128, 64, i8=i8)
    g.q = torch.zeros((rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    for name in ("kp", "vp", "ks", "vs"):
        if getattr(x, name) is not None:
            shape = (pages, *getattr(x, name).shape[1:])
            setattr(g, name, torch.zeros(shape, dtype=getattr(x, name).dtype, device="cuda"))
    g.table = torch.zeros((3, width), dtype=torch.int32, device="cuda")
    out = torch.empty((rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((rows, 8), device="cuda")
    ws = _ws(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(g, ws, out=out, lse=lse)
    for z in (*batches, x, *reversed(batches)):
        g.q[:z.total] = z.q
        for name in ("kp", "vp", "ks", "vs"):
            if getattr(z, name) is not None:
                getattr(g, name)[:z.num_pages] = getattr(z, name)
        g.table[:, :z.table.shape[1]] = z.table
        g.cu.copy_(z.cu)
        g.kv_len.copy_(z.kv_len)
        out.fill_(3)
        lse.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        _compare(z, out, lse)
        assert (out[z.total:] == 3).all() and (lse[z.total:] == 3).all()
    assert msa.device_status(ws) == 0
    del graph


def test_outputs_made_on_a_given_stream():
    """Outputs of a call on a given stream do not take memory that work queued on
    the current stream still uses."""
    from block_sparse_long_05_b200 import msa
    x = Paged([1, 700], [300, 1900], 8, 2, 128, 64)
    ws = _ws(x)
    want = [t.clone() for t in _run(x, ws)]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        kept = torch.full_like(want[0], 3.0)
        busy = torch.full((1 << 27,), 1.0, device="cuda")
        for _ in range(20):
            busy += 1
        copy = kept + busy[0].to(torch.bfloat16) * 0  # reads `kept` late
        del kept  # its memory is free for the current stream only
        got = _run(x, ws, stream=side)
        torch.cuda.synchronize()
        assert (copy == 3).all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert msa.device_status(ws) == 0


@pytest.mark.parametrize("i8", [False, True])
def test_a_run_of_long_steps(i8):
    """Prompts and chunks through append and attention, dense and in a window,
    each step against the plain form over what the cache holds."""
    from block_sparse_long_05_b200 import msa
    Hq, Hkv, d, block = 8, 2, 128, 64
    x = Paged([0, 0], [2100, 2100], Hq, Hkv, d, block, i8=i8)
    ws = _ws(x)
    for t in (x.stores()[2:] if i8 else x.stores()):
        t.fill_(float("nan"))
    g = torch.Generator(device="cuda").manual_seed(2)
    lens = [0, 0]
    for ns in ([900, 17], [100, 1250], [700, 1], [333, 800]):
        lens = [a + n for a, n in zip(lens, ns)]
        x.ns, x.ts, x.total = ns, lens, sum(ns)
        x.cu = torch.tensor([0, ns[0], sum(ns)], dtype=torch.int32, device="cuda")
        x.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        qkv = torch.randn((x.total, Hq + 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
        x.q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        append = msa.kv_append_i8 if i8 else msa.kv_append
        append(k, v, *x.stores(), *x.step(), ws)
        for window, sinks in ((0, 0), (64, 4)):
            out, lse = _run(x, ws, window, sinks, max_q=max(ns))
            assert msa.device_status(ws) == 0
            _compare(x, out, lse, window, sinks, what=f"step {ns}")
