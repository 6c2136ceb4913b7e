"""Refusals of the serving-step calls, without a GPU: bad arguments return an
error on the host before any launch, empty calls return at once."""

import ctypes

import pytest

I32MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def mla():
    import __graft_entry__
    try:
        __graft_entry__.build()
    except RuntimeError as e:  # pragma: no cover - needs nvcc
        pytest.skip("cannot build: %s" % e)
    import mla_latent_kv_append_gb300 as m
    return m


A = 0x10000          # an aligned address that nothing dereferences on the host

PLAN = dict(ctx=A, new=A, req=A, batch=2, table=A, rows=4, max_pages=3, free=A, free_len=5, free_range=A + 64, num_pages=9,
            n=7, block_table=A, q_start=A, seq_lens=A, positions=A, token_req=A, slot=A, free_head=A, err=None, stream=None)


@pytest.mark.parametrize("bad", [
    {"batch": -1}, {"batch": 4097}, {"n": -1}, {"rows": 0}, {"rows": 65537}, {"max_pages": 0}, {"max_pages": I32MAX // 64 + 1},
    {"num_pages": 0}, {"num_pages": I32MAX // 64 + 1}, {"free_len": -1}, {"ctx": None}, {"new": A + 2}, {"req": None},
    {"table": None}, {"free": None}, {"free_range": None}, {"block_table": None}, {"q_start": None}, {"seq_lens": A + 1},
    {"positions": None}, {"token_req": None}, {"slot": None}, {"free_head": None}, {"err": A + 2},
    {"free_head": A + 64}, {"free_head": A + 68}], ids=str)
def test_plan_refuses(mla, bad):
    assert mla.lib.mla_plan_chunks(*(PLAN | bad).values()) == 1


def test_plan_empty(mla):
    assert mla.lib.mla_plan_chunks(*(PLAN | {"batch": 0, "ctx": None}).values()) == 0


ROPE = dict(q=A, qt=192 * 16, qh=192, k=A, kt=576, pos=A, axes=2, axis=None, freq=A, n=5, heads=16, il=1, inv=0, amp=1.0,
            qo=A, qot=1024, qoh=64, ko=A, kot=64, stream=None)


@pytest.mark.parametrize("bad", [
    {"n": -1}, {"heads": -1}, {"heads": 129}, {"axes": 0}, {"axes": 5}, {"amp": float("nan")}, {"amp": float("inf")}, {"il": 2},
    {"inv": -1}, {"k": None}, {"ko": None}, {"axis": bytes([2] * 32)}, {"qt": 4}, {"qh": -8}, {"kt": 7}, {"qot": 1028},
    {"qoh": 12}, {"kot": 1}, {"pos": None}, {"pos": A + 2}, {"freq": None}, {"q": None}, {"q": A + 8}, {"qo": A + 2},
    {"k": A + 8}, {"qoh": 32}, {"qot": 512, "qoh": 64}, {"qot": 64, "qoh": 64}, {"kot": 32}, {"kot": 0}], ids=str)
def test_rope_refuses(mla, bad):
    assert mla.lib.mla_rope(*(ROPE | bad).values()) == 1


def test_rope_empty(mla):
    assert mla.lib.mla_rope(*(ROPE | {"n": 0, "pos": None}).values()) == 0
    assert mla.lib.mla_rope(*(ROPE | {"heads": 0, "k": None, "ko": None, "q": None}).values()) == 0


def chunk(mla, cache=None, **bad):
    a = dict(qn=A, qnt=192 * 16, qnh=192, qp=A, qpt=192 * 16, qph=192, w_uk=A, w_uv=A, table=A, max_pages=4, start=A,
             lens=A, batch=2, n=10, heads=16, max_new=9, kv=0, scale=0.07, ws=A, ws_bytes=1 << 40, o=A, err=None, stream=None) | bad
    c = cache or mla._CacheLayer(8, 1, 1, 0, A, None)
    return mla.lib.mla_chunk_attention(ctypes.byref(c), *a.values())


@pytest.mark.parametrize("bad", [
    {"batch": -1}, {"batch": 4097}, {"n": -1}, {"heads": 8}, {"heads": 24}, {"heads": 144}, {"max_new": -1}, {"max_new": 0},
    {"max_new": 11}, {"kv": -1}, {"kv": (1 << 23) + 1}, {"kv": 1 << 31}, {"scale": 0.0}, {"scale": float("nan")}, {"scale": float("inf")},
    {"max_pages": 0}, {"max_pages": I32MAX // 64 + 1}, {"qnt": -8}, {"qnh": 4}, {"qpt": 2}, {"qph": 100}, {"qn": None},
    {"qn": A + 8}, {"qp": None}, {"w_uk": None}, {"w_uv": A + 4}, {"table": None}, {"start": None}, {"lens": A + 1},
    {"ws": None}, {"ws": A + 16}, {"ws_bytes": 0}, {"o": None}, {"o": A + 8}, {"err": A + 1},
    {"n": I32MAX // 16 + 1, "max_new": 1}], ids=str)
def test_chunk_refuses(mla, bad):
    assert chunk(mla, **bad) == 1


@pytest.mark.parametrize("layer", [(0, 1, 1, 0, A), (8, 9, 1, 0, A), (8, 4, 0, 0, A), (8, 1, 2, 0, A), (8, 1, 1, 1, A),
                                   (8, 1, 1, 0, None), (8, 1, 1, 0, A + 128), (8, 8, 0, 0, A)], ids=str)
def test_chunk_refuses_cache_descriptors(mla, layer):
    assert chunk(mla, cache=mla._CacheLayer(*layer, None)) == 1


def test_chunk_empty(mla):
    assert chunk(mla, batch=0) == 0
    assert chunk(mla, n=0, max_new=0, qn=None, ws=None, ws_bytes=0) == 0


def test_chunk_workspace_sizes(mla):
    f = mla.mla_chunk_workspace_bytes
    assert f(4, 10, 16, 1) > 0
    for bad in [(-1, 10, 16, 1, 0), (4097, 10, 16, 1, 0), (4, -1, 16, 1, 0), (4, 10, 15, 1, 0), (4, 10, 16, 11, 0),
                (4, 10, 16, 1, -1), (4, 300, 16, 300, (1 << 23) + 1)]:
        assert f(*bad) == 0
    # 512 bytes per token and head for the expanded keys and values, at the largest too
    assert f(4, 300, 16, 300, 1 << 23) >= 512 * 16 << 23
    # larger bounds never need less
    assert f(4, 20, 16, 1) >= f(4, 10, 16, 1)
    assert f(4, 300, 16, 300, 1024) >= f(4, 300, 16, 300, 512) >= f(4, 300, 16, 1, 0)


def test_bindings_refuse_host_tensors(mla):
    torch = pytest.importorskip("torch")
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    h = lambda *n: torch.zeros(n, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        mla.mla_plan_chunks(i(2), i(2), i(2), i(4, 3), i(5), i(2), 9, i(2, 3), i(3), i(2), i(7), i(7), i(7), i(1))
    with pytest.raises(ValueError):
        mla.mla_rope(h(5, 16, 64), h(5, 64), i(5), torch.zeros(32), h(5, 16, 64), h(5, 64))
    with pytest.raises(ValueError):
        mla.mla_chunk_attention(None, h(5, 16, 128), h(5, 16, 64), h(16, 128, 512), h(16, 512, 128), i(2, 3), i(3), i(2),
                                torch.zeros(1 << 10, dtype=torch.uint8), h(5, 16, 128), max_new=4)
    with pytest.raises(ValueError):
        mla._err(i(1))
