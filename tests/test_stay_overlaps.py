"""Lengths written over lengths that other blocks still read are refused, also
where the arrays only overlap in part (no GPU: before any launch)."""

import pytest

from tests.test_stay_refusals import A, SELECT, VERIFY, mla  # noqa: F401  (a fixture)

FAR = 0x10000


@pytest.mark.parametrize("off", [-4, 4, -12, 12])
@pytest.mark.parametrize("of", ["lens", "keep"])
def test_select(mla, of, off):  # noqa: F811
    a = SELECT | {"batch": 4, "lens": A + FAR, "keep": A + 2 * FAR}
    assert mla.lib.mla_select_tokens(*(a | {"kept_lens": a[of] + off}).values()) == 1


@pytest.mark.parametrize("off", [-4, 4, -12, 12])
def test_verify(mla, off):  # noqa: F811
    a = VERIFY | {"batch": 4, "lens": A + FAR}
    assert mla.lib.mla_verify_drafts(*(a | {"kept": a["lens"] + off}).values()) == 1
