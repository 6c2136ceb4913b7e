"""Refusals of the calls behind a step's attention, without a GPU: bad
arguments return an error on the host before any launch, empty calls return at
once, and the bindings refuse host tensors and tensors on different GPUs."""

import ctypes
import types

import pytest
import torch

from tests.test_step_devices import Tensor, half

I32MAX = 2 ** 31 - 1
A = 0x100000         # aligned addresses, far apart, that nothing dereferences on the host


@pytest.fixture(scope="module")
def mla():
    import __graft_entry__
    try:
        __graft_entry__.build()
    except RuntimeError as e:  # pragma: no cover - needs nvcc
        pytest.skip("cannot build: %s" % e)
    import mla_latent_kv_append_gb300 as m
    return m


VERIFY = dict(p=A, pr=1000, q=A, qr=1000, kind=0, vocab=1000, drafts=A, start=A, batch=2, rows=6, ua=A, us=A, lens=A, acc=A,
              tokens=A, width=4, kept=A, err=None, stream=None)


@pytest.mark.parametrize("bad", [
    {"batch": -1}, {"batch": 4097}, {"rows": -1}, {"vocab": 0}, {"vocab": (1 << 22) + 1, "pr": 1 << 30, "qr": 1 << 30}, {"width": 0},
    {"kind": -1}, {"kind": 3}, {"p": None}, {"p": A + 2}, {"kind": 1, "p": A + 1}, {"q": A + 2}, {"pr": 999}, {"qr": 999}, {"pr": -1},
    {"drafts": None}, {"start": None}, {"ua": None}, {"us": A + 2}, {"acc": None}, {"tokens": None}, {"lens": None}, {"kept": None},
    {"kept": A + 1}, {"err": A + 2}, {"pr": 2 ** 62, "rows": I32MAX}], ids=str)
def test_verify_refuses(mla, bad):
    assert mla.lib.mla_verify_drafts(*(VERIFY | bad).values()) == 1


def test_verify_empty(mla):
    assert mla.lib.mla_verify_drafts(*(VERIFY | {"batch": 0, "start": None}).values()) == 0


def mass(mla, cache=None, **bad):
    a = dict(q=A, qp=A, lse=A, table=A, max_pages=4, start=A, lens=A, counted=None, batch=2, n=10, heads=16, max_new=9, scale=0.07,
             decay=1.0, ws=A, ws_bytes=1 << 40, mass=A, err=None, stream=None) | bad
    c = cache or mla._CacheLayer(8, 1, 1, 0, A, None)
    return mla.lib.mla_token_mass(ctypes.byref(c), *a.values())


@pytest.mark.parametrize("bad", [
    {"batch": -1}, {"batch": 4097}, {"n": -1}, {"heads": 8}, {"heads": 24}, {"heads": 144}, {"max_new": -1}, {"max_new": 0},
    {"max_new": 11}, {"scale": 0.0}, {"scale": float("nan")}, {"scale": float("inf")}, {"decay": -0.5}, {"decay": float("nan")},
    {"decay": float("inf")}, {"max_pages": 0}, {"max_pages": I32MAX // 64 + 1}, {"q": None}, {"q": A + 8}, {"qp": A + 4},
    {"lse": None}, {"table": None}, {"start": A + 2}, {"lens": None}, {"counted": A + 1}, {"mass": None}, {"mass": A + 2}, {"ws": None},
    {"ws": A + 128}, {"ws_bytes": 0}, {"err": A + 1}, {"n": I32MAX // 16 + 1, "max_new": 1}], ids=str)
def test_mass_refuses(mla, bad):
    assert mass(mla, **bad) == 1


LAYERS = [(0, 1, 1, 0, A), (8, 9, 1, 0, A), (8, 4, 0, 0, A), (8, 1, 2, 0, A), (8, 1, 1, 1, A), (8, 1, 1, 0, None), (8, 1, 1, 0, A + 128),
          (8, 8, 0, 0, A)]


@pytest.mark.parametrize("layer", LAYERS, ids=str)
def test_cache_descriptors(mla, layer):
    assert mass(mla, cache=mla._CacheLayer(*layer, None)) == 1
    assert move(mla, cache=mla._CacheLayer(*layer, None)) == 1


def test_mass_empty_and_workspace(mla):
    assert mass(mla, batch=0) == 0
    assert mass(mla, n=0, max_new=0, q=None, ws=None) == 0
    f = mla.mla_mass_workspace_bytes
    assert 0 < f(4, 10, 16, 1) <= f(4, 20, 16, 1) <= f(4, 20, 64, 20)
    for bad in [(-1, 10, 16, 1), (4097, 10, 16, 1), (4, -1, 16, 1), (4, 10, 15, 1), (4, 10, 144, 1), (4, 10, 16, 11), (4, 10, 16, -1),
                (4, I32MAX // 16 + 1, 16, 1)]:
        assert f(*bad) == 0


SELECT = dict(mass=A, num_pages=9, table=A, max_pages=4, lens=A, keep=A + 64, batch=2, sinks=1, recent=1, kept=A, max_keep=5,
              kept_lens=A + 128, err=None, stream=None)


@pytest.mark.parametrize("bad", [
    {"batch": -1}, {"batch": 4097}, {"sinks": -1}, {"recent": -1}, {"max_keep": 0}, {"max_pages": 0}, {"max_pages": (1 << 24) + 1},
    {"num_pages": 0}, {"num_pages": I32MAX // 64 + 1}, {"mass": None}, {"table": A + 1}, {"lens": None}, {"keep": None}, {"kept": None},
    {"kept_lens": None}, {"kept_lens": A}, {"kept_lens": A + 64}, {"err": A + 3}], ids=str)
def test_select_refuses(mla, bad):
    assert mla.lib.mla_select_tokens(*(SELECT | bad).values()) == 1


def test_select_empty(mla):
    assert mla.lib.mla_select_tokens(*(SELECT | {"batch": 0, "mass": None}).values()) == 0


B = 0x1000           # bytes between the arrays below
RELEASE = dict(old=A, new=A + B, req=A + 2 * B, batch=2, table=A + 3 * B, page_table=A + 4 * B, rows=4, max_pages=3, free=A + 5 * B,
               free_len=5, range=A + 6 * B, num_pages=9, move=1, out=A + 7 * B, lens_out=A + 8 * B, range_out=A + 9 * B, err=None,
               stream=None)


@pytest.mark.parametrize("bad", [
    {"batch": -1}, {"batch": 4097}, {"move": 2}, {"move": -1}, {"rows": 0}, {"rows": 65537}, {"max_pages": 0},
    {"max_pages": I32MAX // 64 + 1}, {"num_pages": 0}, {"num_pages": I32MAX // 64 + 1}, {"free_len": -1}, {"old": None}, {"new": A + 2},
    {"req": None}, {"table": None}, {"page_table": None}, {"free": None}, {"range": None}, {"out": None}, {"lens_out": None},
    {"range_out": A + 1}, {"err": A + 2},
    {"lens_out": A}, {"lens_out": A + B + 4}, {"out": A + 3 * B}, {"out": A + 3 * B - 4}, {"range_out": A + 6 * B}, {"range_out": A + 6 * B + 4},
    {"out": A + 5 * B + 16}, {"range_out": A + 8 * B + 4}, {"page_table": A + 3 * B}, {"free": A + 2 * B}], ids=str)
def test_release_refuses(mla, bad):
    assert mla.lib.mla_release_pages(*(RELEASE | bad).values()) == 1


def test_release_empty(mla):
    assert mla.lib.mla_release_pages(*(RELEASE | {"batch": 0, "old": None}).values()) == 0


def move(mla, cache=None, **bad):
    a = dict(src=A, lens=A, kept=A, max_keep=5, new=A, dst=A, max_pages=4, batch=2, mass=None, err=None, stream=None) | bad
    c = cache or mla._CacheLayer(8, 1, 1, 0, A, None)
    return mla.lib.mla_move_tokens(ctypes.byref(c), *a.values())


@pytest.mark.parametrize("bad", [
    {"batch": -1}, {"batch": 4097}, {"max_keep": 0}, {"max_pages": 0}, {"max_pages": I32MAX // 64 + 1}, {"src": None}, {"lens": None},
    {"kept": A + 2}, {"new": None}, {"dst": None}, {"mass": A + 2}, {"err": A + 1}], ids=str)
def test_move_refuses(mla, bad):
    assert move(mla, **bad) == 1


def test_move_empty(mla):
    assert move(mla, batch=0, src=None) == 0


# ---------------------------------------------------------------------------

def real(*shape):
    return Tensor(*shape, dtype=torch.float32)


def calls(mla):
    cache = types.SimpleNamespace(pool=Tensor(1 << 20, dtype=torch.uint8), c_struct=mla._CacheLayer, num_pages=9)
    return {
        "mla_verify_drafts": dict(target_probs=real(6, 100), draft_probs=real(6, 100), drafts=Tensor(6), row_start=Tensor(3),
                                  u_accept=real(6), u_sample=real(2), accepted=Tensor(2), tokens=Tensor(2, 4), seq_lens=Tensor(2),
                                  kept_lens=Tensor(2), dev_err=Tensor(1)),
        "mla_token_mass": dict(cache=cache, q_lat=real(5, 16, 512), q_pe=half(5, 16, 64), lse=real(5, 16), block_table=Tensor(2, 3),
                               q_start=Tensor(3), seq_lens=Tensor(2), workspace=Tensor(1 << 20, dtype=torch.uint8), mass=real(576),
                               max_new=4, counted=Tensor(2), dev_err=Tensor(1)),
        "mla_select_tokens": dict(mass=real(576), block_table=Tensor(2, 3), seq_lens=Tensor(2), keep_lens=Tensor(2), kept=Tensor(2, 7),
                                  kept_lens=Tensor(2), dev_err=Tensor(1)),
        "mla_release_pages": dict(old_lens=Tensor(2), new_lens=Tensor(2), req=Tensor(2), block_table=Tensor(2, 3),
                                  page_table=Tensor(4, 3), free_pages=Tensor(5), free_range=Tensor(2), num_pages=9,
                                  new_table=Tensor(2, 3), lens_out=Tensor(2), free_range_out=Tensor(2), move=True, dev_err=Tensor(1)),
        "mla_move_tokens": dict(cache=cache, src_table=Tensor(2, 3), seq_lens=Tensor(2), kept=Tensor(2, 7), lens=Tensor(2),
                                dst_table=Tensor(2, 3), mass=real(576), dev_err=Tensor(1)),
    }


NAMES = ["mla_verify_drafts", "mla_token_mass", "mla_select_tokens", "mla_release_pages", "mla_move_tokens"]


@pytest.mark.parametrize("name", NAMES)
def test_one_tensor_on_another_gpu(mla, monkeypatch, name):
    made = []
    monkeypatch.setattr(mla, "_step", lambda *args: made.append(args))
    getattr(mla, name)(**calls(mla)[name])
    assert len(made) == 1                                 # all on one GPU: launched
    for k, v in calls(mla)[name].items():
        if not isinstance(v, Tensor) and k != "cache":
            continue
        args = calls(mla)[name]
        (args[k].pool if k == "cache" else args[k]).index = 1
        with pytest.raises(ValueError):
            getattr(mla, name)(**args)
    assert len(made) == 1


@pytest.mark.parametrize("name", NAMES)
def test_another_type_or_shape(mla, monkeypatch, name):
    made = []
    monkeypatch.setattr(mla, "_step", lambda *args: made.append(args))
    for k, v in calls(mla)[name].items():
        if not isinstance(v, Tensor) or k == "workspace":
            continue
        args = calls(mla)[name]
        args[k].dtype = torch.float64
        with pytest.raises(ValueError):
            getattr(mla, name)(**args)
        if k == "dev_err":
            continue
        args = calls(mla)[name]
        args[k].shape = args[k].shape[:-1] + (args[k].shape[-1] + 65,)
        free = {"mla_verify_drafts": ("tokens",), "mla_token_mass": ("block_table",), "mla_select_tokens": ("block_table", "kept")}
        if k in free.get(name, ("kept", "free_pages")):   # any width will do
            continue
        with pytest.raises(ValueError):
            getattr(mla, name)(**args)
    assert not made


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors(mla, name):
    args = {k: torch.zeros(v.shape, dtype=v.dtype) if isinstance(v, Tensor) and k != "workspace" else v
            for k, v in calls(mla)[name].items()}
    with pytest.raises(ValueError):
        getattr(mla, name)(**args)


def test_arguments_that_go_together(mla):
    a = calls(mla)["mla_verify_drafts"]
    with pytest.raises(ValueError):
        mla.mla_verify_drafts(**(a | {"kept_lens": None}))
    a = calls(mla)["mla_release_pages"]
    for k in ("req", "page_table"):
        with pytest.raises(ValueError):
            mla.mla_release_pages(**(a | {k: None}))
