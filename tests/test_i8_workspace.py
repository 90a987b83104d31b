"""Workspace of the 8-bit products: asked for only where a kernel may use it."""
import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_abi import L  # noqa: F401  (the built library as a fixture)
from tests.test_abi_i8_rope import _item, _linear


@pytest.mark.parametrize("k", [64, 448, 512])
@pytest.mark.parametrize("m", [0, 1, 8, 9, 300, 16238])
def test_short_k_needs_no_workspace(L, m, k):
    assert te.i8_workspace(m, k, 1536) == 0


def test_a_call_of_short_k_goes_without(L):
    # m = 0 looks at the arguments and has nothing to launch; a long k of many
    # tokens is still refused before any launch
    assert _linear(L, m=0, ws=None, nb=0)[0] == te.TE_OK
    assert _linear(L, m=300, k=576, ldx=576, item=_item(k=576), ws=None, nb=0)[0] == te.TE_EWORKSPACE
    assert te.i8_workspace(300, 576, 64) >= 2 * 300 * 576
