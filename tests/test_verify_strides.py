"""mla_verify_drafts' binding and the strides of dimensions of one entry, which
mean nothing and which PyTorch leaves as a view made them (no GPU)."""

import pytest
import torch

from tests.test_stay_refusals import mla, real  # noqa: F401  (a fixture)
from tests.test_step_devices import Tensor


class Strided(Tensor):
    def __init__(self, shape, strides):
        super().__init__(*shape, dtype=torch.float32)
        self.strides = strides

    def stride(self):
        return self.strides


def call(mla, monkeypatch, target, draft):  # noqa: F811
    made = []
    monkeypatch.setattr(mla, "_step", lambda *args: made.append(args))
    n, one = target.shape[0], Tensor(1)
    mla.mla_verify_drafts(target, draft, Tensor(n), Tensor(2), real(n), real(1), one, Tensor(1, 4))
    (args,) = made
    return args[4], args[6]                                # the rows' strides as the library gets them


@pytest.mark.parametrize("shape,strides,row", [
    ((1, 100), (1, 1), 100),                               # a column, transposed
    ((1, 100), (0, 1), 100),                               # expanded
    ((1, 100), (7000, 1), 100),
    ((3, 100), (128, 1), 128),
    ((3, 1), (100, 100), 100),                             # one column of a wider matrix
    ((3, 1), (1, 5), 1),
    ((1, 1), (0, 0), 1),
])
def test_any_stride_of_one_entry(mla, monkeypatch, shape, strides, row):  # noqa: F811
    t = Strided(shape, strides)
    assert call(mla, monkeypatch, t, None) == (row, 0)
    assert call(mla, monkeypatch, t, Strided(shape, strides)) == (row, row)


@pytest.mark.parametrize("strides", [(1, 3), (200, 2)])
def test_rows_apart_are_refused(mla, monkeypatch, strides):  # noqa: F811
    for target, draft in ((Strided((3, 100), strides), None), (real(3, 100), Strided((3, 100), strides))):
        with pytest.raises(ValueError):
            call(mla, monkeypatch, target, draft)
