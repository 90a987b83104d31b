"""Choosing a kernel of the 8-bit products by hand: what is no choice, and calls
that a chosen kernel does not take, are refused on the host."""
import ctypes

import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_abi import L, _call  # noqa: F401  (the built library as a fixture)
from tests.test_abi_i8_rope import FAKE, _item, _linear


@pytest.fixture(autouse=True)
def the_rule_again(L):
    yield
    te.i8_choose(None)


@pytest.mark.parametrize("choice", [(-1, 8, 1), (4, 8, 1), (te.TE_I8_FEW, 64, 1), (te.TE_I8_FEW, 8, 3), (te.TE_I8_FEW, 8, 0),
                                    (te.TE_I8_MIDDLING, 8, 1), (te.TE_I8_MIDDLING, 256, 1), (te.TE_I8_MIDDLING, 64, 16),
                                    (te.TE_I8_MIDDLING, 64, 3), (te.TE_I8_RESIDENT, 64, 1), (te.TE_I8_RESIDENT, 128, 2),
                                    (te.TE_I8_LARGE, 192, 1), (te.TE_I8_LARGE, 0, 1)])
def test_what_is_no_choice_is_refused(L, choice):
    with pytest.raises(te.TEError) as e:
        te.i8_choose(choice)
    assert e.value.status == te.TE_EINVAL


@pytest.mark.parametrize("choice,m,k", [((te.TE_I8_FEW, 8, 2), 9, 512), ((te.TE_I8_FEW, 16, 1), 17, 512),
                                        ((te.TE_I8_FEW, 8, 1), 4, 512), ((te.TE_I8_FEW, 16, 4), 4, 512),
                                        ((te.TE_I8_FEW, 32, 2), 4, 512), ((te.TE_I8_MIDDLING, 16, 8), 40, 896),
                                        ((te.TE_I8_MIDDLING, 16, 2), 40, 128), ((te.TE_I8_MIDDLING, 16, 1), 1 << 20, 512),
                                        ((te.TE_I8_RESIDENT, 128, 1), 300, 576), ((te.TE_I8_LARGE, 0, 0), 300, 512),
                                        ((te.TE_I8_LARGE, 0, 0), 8, 1024)])
def test_a_call_that_the_chosen_kernel_does_not_take(L, choice, m, k):
    te.i8_choose(choice)
    st, msg = _linear(L, m=m, k=k, ldx=k, item=_item(k=k))
    assert st == te.TE_ESHAPE and "chosen" in msg
    with pytest.raises(te.TEError):
        te.i8_choice_of(m, k, [64])


def test_the_choice_is_a_threads_own(L):
    import threading
    te.i8_choose((te.TE_I8_LARGE, 0, 0))
    seen = []
    t = threading.Thread(target=lambda: seen.append(te.i8_choice_of(5, 512, [64])[0]))
    t.start()
    t.join()
    assert seen == [te.TE_I8_FEW]
    te.i8_choose(None)
    assert te.i8_choice_of(5, 512, [64])[:2] == (te.TE_I8_FEW, 8)


def test_choice_of_rejects_bad_sizes(L):
    for m, k, ns, gated in ((0, 64, [64], 0), (5, 100, [64], 0), (5, 65600, [64], 0), (5, 64, [40], 0), (5, 64, [], 0),
                            (5, 64, [32] * 5, 0), (5, 64, [32, 32], 1)):
        with pytest.raises(te.TEError) as e:
            te.i8_choice_of(m, k, ns, gated)
        assert e.value.status == te.TE_ESHAPE
    c = te.te_i8_choice()
    assert _call(L, "te_i8_choice_of", 5, 64, None, 1, 0, ctypes.byref(c))[0] == te.TE_EINVAL
    assert FAKE


def test_the_marshalling_module_calls_nothing_before_it_is_bound(L):
    import os
    import subprocess
    import sys
    from tests.test_abi import ROOT
    script = """
import torch
from transformer_encoder_forward_gb300 import _marshal
try:
    _marshal.quant_rows(1, 2, 3, None)
except RuntimeError as e:
    print(e)
for bad in ((1, 2), (0, 0, 0, 0, 0), (1, 2, 3, 4, "5")):
    try:
        _marshal.bind(*bad)
    except (TypeError, ValueError):
        print("refused")
"""
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split("\n")[:4] == ["the library's functions have not been bound"] + ["refused"] * 3
