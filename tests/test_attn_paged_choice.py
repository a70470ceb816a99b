"""msa_attn_paged_kernels: which kernels a step of attention over pages takes."""
import pytest


@pytest.fixture(scope="module")
def msa():
    from block_sparse_long_05_b200 import build, msa
    build.build_library()
    return msa


@pytest.mark.parametrize("step, kernels", [
    # Bt, total, Hq, Hkv, block, page_stride, window, sinks, max_q
    ((1, 1, 8, 2, 64, 63, 0, 0, None), ("split",)),                  # one token
    ((32, 32, 64, 8, 128, 256, 0, 0, 1), ("split",)),                # a decode step
    ((32, 32, 64, 8, 128, 256, 0, 0, None), ("split", "chunk")),     # the same, its rows unknown
    ((1, 2048, 32, 8, 128, 256, 0, 0, 2048), ("chunk",)),            # a chunk by itself
    ((6, 2215, 64, 8, 512, 24, 0, 0, 701), ("split", "chunk")),      # a mixed batch
    ((1, 64, 32, 8, 128, 4, 0, 0, 64), ("split",)),                  # a small step of many rows
    ((1, 64, 32, 8, 128, 1024, 0, 0, 64), ("chunk",)),               # behind a wide table
    ((1, 64, 32, 8, 128, 1024, 128, 4, 64), ("split",)),             # in a window
    ((1, 64, 32, 8, 128, 1024, 2 ** 31 - 1, 2 ** 31 - 1, 64), ("chunk",)),
    ((1, 0, 8, 2, 64, 63, 0, 0, None), ()),
    ((0, 4, 8, 2, 64, 63, 0, 0, None), ()),
    ((1, 4, 7, 2, 64, 63, 0, 0, None), ()),
    ((1, 4, 8, 0, 64, 63, 0, 0, None), ()),
    ((1, 4, 8, 2, 0, 63, 0, 0, None), ()),
    ((1, 4, 8, 2, 64, 0, 0, 0, None), ()),
    ((1, 4, 8, 2, 64, 63, -1, 0, None), ()),
    ((1, 4, 8, 2, 64, 63, 0, -1, None), ()),
    ((1, 4, 8, 2, 64, 63, 0, 0, -1), ()),
    ((1, 4, 8, 2, 48, 63, 0, 0, None), ()),                          # no such block
    ((1, 2 ** 31 - 1, 2 ** 31 - 1, 1, 128, 2 ** 31 - 1, 0, 0, None), ()),
    ((1, 64, 32, 8, 128, 2 ** 31 - 1, 0, 0, None), ()),
    ((1, 2 ** 30, 1, 1, 128, 8, 0, 0, None), ()),
    ((2 ** 24, 64, 32, 8, 128, 8, 0, 0, None), ()),
    ((1, 2 ** 26, 32, 8, 128, 8, 0, 0, None), ()),
])
def test_choice(msa, step, kernels):
    *sizes, max_q = step
    assert msa.attn_paged_kernels(*sizes, max_q=max_q) == kernels
