"""Refusals of the paged-cache calls, on the host before any CUDA call, and
the checks of their Python binding."""
import pytest
import torch

OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 1 << 20  # never dereferenced: every case fails on the host
ODD = FAKE + 8  # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    from block_sparse_long_05_b200 import build, msa
    build.build()
    return msa.load_library()


def _call(fn, names, base, **change):
    args = dict(base, **change)
    assert set(args) == set(names.split())
    return fn(*(args[n] for n in names.split()))


STEP = dict(table=FAKE, stride=16, pages=64, cu=FAKE, kv_len=FAKE)
TAIL = dict(ws=FAKE, ws_bytes=1 << 30, stream=None)


def _step_refusals(call):
    for name in ("table", "cu", "kv_len"):
        assert call(**{name: None}) == ARG
        assert call(**{name: FAKE + 2}) == ARG
    assert call(stride=0) == ARG
    assert call(pages=0) == ARG
    assert call(Bt=0) == ARG
    assert call(total=-1) == ARG
    assert call(Hkv=0) == ARG
    assert call(d=96) == UNSUPPORTED
    assert call(block=48) == UNSUPPORTED
    assert call(block=0) == ARG
    assert call(pages=1 << 25, block=64) == UNSUPPORTED     # 2^31 rows
    assert call(stride=1 << 24, block=64) == UNSUPPORTED    # 2^30 positions
    assert call(total=1 << 30) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 128) == WORKSPACE
    assert call(ws_bytes=64) == WORKSPACE


def test_append_refusals(lib):
    names = ("k ks v vs k_idx xs kp vp xp table stride pages cu kv_len Bt total Hkv d d_idx block "
             "ws ws_bytes stream")
    base = dict(k=FAKE, ks=256, v=FAKE, vs=256, k_idx=None, xs=0, kp=FAKE, vp=FAKE, xp=None, Bt=2,
                total=8, Hkv=2, d=128, d_idx=0, block=64, **STEP, **TAIL)
    names8 = names.replace("vp xp", "vp sk sv xp")
    for fn, nm, b in ((lib.msa_kv_append, names, base),
                      (lib.msa_kv_append_i8, names8, dict(base, sk=FAKE, sv=FAKE))):
        call = lambda **ch: _call(fn, nm, b, **ch)  # noqa: E731
        _step_refusals(call)
        for name in ("k", "v", "kp", "vp"):
            assert call(**{name: None}) == ARG
            assert call(**{name: ODD}) == ARG
        assert call(ks=255) == ARG and call(ks=252) == ARG and call(vs=260) == ARG
        assert call(k_idx=FAKE) == ARG and call(xp=FAKE) == ARG
        assert call(k_idx=FAKE, xp=FAKE, d_idx=96, xs=96) == UNSUPPORTED
        assert call(k_idx=FAKE, xp=FAKE, d_idx=64, xs=60) == ARG
        assert call(k_idx=ODD, xp=FAKE, d_idx=64, xs=64) == ARG
        assert call(total=1 << 25, Hkv=64, ks=8192, vs=8192) == UNSUPPORTED
        assert call(total=0) == OK
    assert _call(lib.msa_kv_append_i8, names8, dict(base, sk=None, sv=FAKE)) == ARG
    assert _call(lib.msa_kv_append_i8, names8, dict(base, sk=FAKE, sv=FAKE + 4)) == ARG


def test_gather_refusals(lib):
    names = "kp vp table stride pages cu kv_len k v Bt total Hkv d block ws ws_bytes stream"
    base = dict(kp=FAKE, vp=FAKE, k=FAKE, v=FAKE, Bt=2, total=8, Hkv=2, d=128, block=64, **STEP,
                **TAIL)
    names8 = names.replace("kp vp", "kp vp sk sv")
    for fn, nm, b in ((lib.msa_kv_gather, names, base),
                      (lib.msa_kv_gather_i8, names8, dict(base, sk=FAKE, sv=FAKE))):
        call = lambda **ch: _call(fn, nm, b, **ch)  # noqa: E731
        _step_refusals(call)
        for name in ("k", "v", "kp", "vp"):
            assert call(**{name: None}) == ARG
            assert call(**{name: ODD}) == ARG
        assert call(total=0) == OK
    assert _call(lib.msa_kv_gather_i8, names8, dict(base, sk=FAKE, sv=None)) == ARG


def test_attn_refusals(lib):
    names = ("q qs kp vp table stride pages cu kv_len out lse Bt total max_q Hq Hkv d block window "
             "sinks ws ws_bytes stream")
    base = dict(q=FAKE, qs=1024, kp=FAKE, vp=FAKE, out=FAKE, lse=FAKE, Bt=2, total=8, max_q=0, Hq=8,
                Hkv=2, d=128, block=64, window=0, sinks=0, **STEP, **TAIL)
    names8 = names.replace("kp vp", "kp vp sk sv")
    for fn, nm, b in ((lib.msa_attn_paged, names, base),
                      (lib.msa_attn_paged_i8, names8, dict(base, sk=FAKE, sv=FAKE))):
        call = lambda **ch: _call(fn, nm, b, **ch)  # noqa: E731
        _step_refusals(call)
        for name in ("q", "kp", "vp", "out"):
            assert call(**{name: None}) == ARG
            assert call(**{name: ODD}) == ARG
        assert call(lse=None) == ARG and call(lse=FAKE + 2) == ARG
        assert call(Hq=7) == ARG and call(Hq=0) == ARG
        assert call(window=-1) == ARG and call(sinks=-1) == ARG and call(max_q=-1) == ARG
        assert call(qs=1023) == ARG and call(qs=1020) == ARG
        assert call(ws_bytes=1 << 16) == WORKSPACE
        assert call(total=0) == OK
    assert _call(lib.msa_attn_paged_i8, names8, dict(base, sk=None, sv=FAKE)) == ARG


def test_sparse_i8_refusals(lib):
    names = ("q kp vp sk sv table stride pages ids out lse Bt T Hq Hkv d block K ws ws_bytes stream")
    base = dict(q=FAKE, kp=FAKE, vp=FAKE, sk=FAKE, sv=FAKE, table=FAKE, stride=16, pages=64,
                ids=FAKE, out=FAKE, lse=FAKE, Bt=2, T=1000, Hq=8, Hkv=2, d=128, block=64, K=4,
                **TAIL)
    call = lambda **ch: _call(lib.msa_sparse_attn_paged_i8, names, base, **ch)  # noqa: E731
    for name in ("q", "kp", "vp", "sk", "sv", "out"):
        assert call(**{name: None}) == ARG
        assert call(**{name: ODD}) == ARG
    for name in ("table", "ids", "lse"):
        assert call(**{name: None}) == ARG
        assert call(**{name: FAKE + 2}) == ARG
    assert call(stride=15) == ARG                   # fewer entries than blocks
    assert call(K=0) == ARG and call(K=33) == UNSUPPORTED
    assert call(T=0) == ARG and call(Bt=0) == ARG and call(Hq=9) == ARG
    assert call(d=80) == UNSUPPORTED and call(block=96) == UNSUPPORTED
    assert call(T=1 << 30, stride=1 << 26) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(ws_bytes=1 << 12) == WORKSPACE


def test_workspace_size(lib):
    for d in (64, 128):
        n = lib.msa_cache_workspace_size(8, 2, d)
        assert n > 0 and n % 256 == 0
    assert lib.msa_cache_workspace_size(8, 3, 128) == 0
    assert lib.msa_cache_workspace_size(0, 1, 128) == 0
    assert lib.msa_cache_workspace_size(8, 2, 96) == 0


def test_binding_checks(lib):
    """The compiled binding refuses tensors that are not CUDA tensors, and arguments
    that are no tensors at all, before any call."""
    from block_sparse_long_05_b200 import msa

    class Ws:
        ptr, nbytes, device_index = FAKE, 1 << 30, 0

    pages = torch.zeros((4, 32, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    codes, scales = pages.to(torch.int8), torch.zeros((4, 2, 32))
    for call in (lambda: msa.kv_append(pages[0], pages[0], pages, pages, i, i, i, Ws),
                 lambda: msa.kv_append_i8(pages[0], pages[0], codes, codes, scales, scales, i, i, i, Ws),
                 lambda: msa.kv_gather(pages, pages, i, i, i, 4, Ws),
                 lambda: msa.kv_gather_i8(codes, codes, scales, scales, i, i, i, 4, Ws),
                 lambda: msa.attn_paged(pages[0], pages, pages, i, i, i, Ws),
                 lambda: msa.attn_paged_i8(pages[0], codes, codes, scales, scales, i, i, i, Ws),
                 lambda: msa.sparse_attn_paged_i8(pages[:1], codes, codes, scales, scales, i, 9, i, Ws)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="must be a tensor"):
        msa.attn_paged(pages[0], None, pages, i, i, i, Ws)
    with pytest.raises(ValueError, match="negative"):
        msa.kv_gather(pages, pages, i, i, i, -1, Ws)
    with pytest.raises((ValueError, TypeError)):
        msa.kv_gather(pages, pages, i, i, i, "4", Ws)


def test_binding_fails_loudly_if_missing(tmp_path):
    from block_sparse_long_05_b200 import msa
    saved, msa._fast = msa._fast, None
    try:
        with pytest.raises(RuntimeError, match="missing"):
            msa.load_binding(str(tmp_path / "_msa_torch.so"))
    finally:
        msa._fast = saved
