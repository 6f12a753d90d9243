"""Rotary positions in place, without a GPU: outputs that start where their inputs do, but are laid out in another way or moved
by slots, are refused before anything is launched."""
import ctypes

import pytest

import test_abi_long_cache as base
from test_abi_long_cache import api  # noqa: F401

APART = dict(q_out=1 << 20, k_out=2 << 20, v_out=3 << 20)
SAME, OTHER = [512, 128, 64], [512, 64, 128]


@pytest.mark.parametrize("kw,strides", [
    (dict(q_out=base.P16), [*SAME, *SAME, *SAME, *OTHER, *SAME, *SAME]),
    (dict(k_out=base.P16, slot=None), [*SAME, *SAME, *SAME, *SAME, *OTHER, *SAME]),
    (dict(v_out=base.P16, slot=None), [*SAME, *SAME, *SAME, *SAME, *SAME, *OTHER]),
    (dict(k_out=base.P16), [*SAME] * 6),
    (dict(v_out=base.P16), [*SAME] * 6),
], ids=str)
def test_refused(api, kw, strides):  # noqa: F811
    heads = base._heads(api, strides=strides, **{**APART, **kw})
    assert api.library_handle().kv_qk_norm_rope(ctypes.byref(heads), None, None) == -1

