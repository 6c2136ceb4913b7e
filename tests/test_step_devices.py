"""The serving-step bindings refuse tensors on different GPUs, checked without
one: stand-in tensors say where they lie, and nothing is launched."""

import types

import pytest
import torch


@pytest.fixture(scope="module")
def mla():
    import __graft_entry__
    try:
        __graft_entry__.build()
    except RuntimeError as e:  # pragma: no cover - needs nvcc
        pytest.skip("cannot build: %s" % e)
    import mla_latent_kv_append_gb300 as m
    return m


class Tensor:
    """A contiguous CUDA tensor's attributes, without its memory."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.int32):
        self.shape, self.dtype, self.index = shape, dtype, 0

    device = property(lambda self: "cuda:%d" % self.index)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def stride(self):
        n, out = 1, []
        for s in reversed(self.shape):
            out.insert(0, n)
            n *= s
        return tuple(out)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return 1 << 20

    def element_size(self):
        return 1

    def data_ptr(self):
        return 0x10000


def half(*shape):
    return Tensor(*shape, dtype=torch.bfloat16)


def plan():
    names = ("ctx_lens", "new_lens", "req", "page_table", "free_pages", "free_range", "block_table", "q_start", "seq_lens",
             "positions", "token_req", "slot", "free_head", "dev_err")
    shapes = ((2,), (2,), (2,), (4, 3), (5,), (2,), (2, 3), (3,), (2,), (7,), (7,), (7,), (1,), (1,))
    return {k: Tensor(*s) for k, s in zip(names, shapes)} | {"num_pages": 9}


def rope():
    return {"q_pe": half(5, 16, 64), "k_pe": half(5, 64), "positions": Tensor(5), "inv_freq": Tensor(32, dtype=torch.float32),
            "q_out": half(5, 16, 64), "k_out": half(5, 64)}


def chunk(mla):
    return {"cache": types.SimpleNamespace(pool=Tensor(1 << 20, dtype=torch.uint8), c_struct=mla._CacheLayer),
            "q_nope": half(5, 16, 128), "q_pe": half(5, 16, 64), "w_uk": half(16, 128, 512), "w_uv": half(16, 512, 128),
            "block_table": Tensor(2, 3), "q_start": Tensor(3), "seq_lens": Tensor(2), "workspace": Tensor(1 << 20, dtype=torch.uint8),
            "o": half(5, 16, 128), "dev_err": Tensor(1), "max_new": 4}


@pytest.mark.parametrize("name", ["mla_plan_chunks", "mla_rope", "mla_chunk_attention"])
def test_one_tensor_on_another_gpu(mla, monkeypatch, name):
    calls = []
    monkeypatch.setattr(mla, "_step", lambda *args: calls.append(args))
    make = {"mla_plan_chunks": plan, "mla_rope": rope, "mla_chunk_attention": lambda: chunk(mla)}[name]
    getattr(mla, name)(**make())
    assert len(calls) == 1                                # all on one GPU: launched
    tensors = [k for k, v in make().items() if isinstance(v, Tensor)] + (["cache"] if "cache" in make() else [])
    assert len(tensors) >= 6
    for k in tensors:
        args = make()
        (args[k].pool if k == "cache" else args[k]).index = 1
        with pytest.raises(ValueError):
            getattr(mla, name)(**args)
    assert len(calls) == 1
