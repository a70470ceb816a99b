"""A window over a context that is longer than its page-table row: the sinks,
and the keys of the window that the table holds, are attended all the same."""
import pytest
import torch

import cache_bounds
import cache_ref
from cache_ref import Paged, attend, tolerances
from gpu_helpers import lib_ready

pytestmark = pytest.mark.gpu

BAD_IDS = 6


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n", [1, 3, 600])
@pytest.mark.parametrize("kv_len", [641, 700, 900, 4000, 100000])
@pytest.mark.parametrize("sinks", [0, 4, 200, 5000])
def test_window_of_a_context_longer_than_its_table(n, kv_len, sinks, i8):
    from block_sparse_long_05_b200 import msa
    lib_ready()
    cap, window = 640, 100
    x = Paged([n], [cap], 8, 2, 128, 64, i8=i8)
    x.table = x.table[:, :10].contiguous()
    x.kv_len = torch.tensor([kv_len], dtype=torch.int32, device="cuda")
    assert cache_bounds.reaches(x, "chunk" if n == 600 else "split", window, sinks)
    ws = msa.Workspace.for_cache(8, 2, 128)
    call = msa.attn_paged_i8 if i8 else msa.attn_paged
    out, lse = call(x.q, *x.stores(), *x.step(), ws, window=window, sinks=sinks)
    assert msa.device_status(ws) == BAD_IDS
    seen = cache_bounds.visible(n, kv_len, window, sinks, cap=cap)
    k, v = x.context(0)
    for h in range(8):
        o, l, a, s = attend(x.q[:, h].double(), k[:, h // 4], v[:, h // 4], seen)
        cache_ref.check(out[:, h], lse[:, h], o, l, *tolerances(o, l, a, s, 128), f"head {h}")
