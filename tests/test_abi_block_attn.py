"""Refusals of the block's attention step that need no descriptor (no GPU needed)."""
import ctypes

import transformer_encoder_forward_gb300 as te
from tests.test_abi import FAKE, L, _call  # noqa: F401  (the built library as a fixture)


def _block(L, a):
    return _call(L, "te_encoder_block_attn_fwd", None, ctypes.byref(a), FAKE, FAKE, None, FAKE, 1, FAKE, 0, None)


def test_a_table_without_its_plan_is_refused(L):
    """Not taken as attention without a bias."""
    st, msg = _block(L, te.te_block_attn(-1, -1, 0, None, FAKE, 8))
    assert st == te.TE_EINVAL and "plan" in msg
    # and without either the descriptor is looked at
    st, msg = _block(L, te.te_block_attn(-1, -1, 0, None, None, 0))
    assert st == te.TE_EINVAL and "plan" not in msg
