"""The binding's copies of the header's names and numbers are the header's."""
import os
import re

import pytest

from gated_delta_rule_gate_gb300 import _native as N

HEADER = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn.h")).read()
NUMBERS = {n: int(v.rstrip("u"), 0) for n, v in
           re.findall(r"^\s*(?:#define )?(GDN_[A-Z0-9_]+)\s*(?:=\s*)?(0x[0-9a-f]+u?|\d+)\b", HEADER, re.M)}


@pytest.mark.parametrize("prefix,copy", [("GDN_ACT_", N.ACTIVATIONS), ("GDN_RULE_", N.RULES),
                                         ("GDN_INPUT_SCALE_", N.INPUT_SCALES)])
def test_names(prefix, copy):
    assert {n[len(prefix):].lower(): v for n, v in NUMBERS.items() if n.startswith(prefix)} == copy


def test_numbers():
    assert NUMBERS["GDN_ADAMW_BLOCK"] == N.ADAMW_BLOCK and NUMBERS["GDN_SCAN_CHUNK"] == N.SCAN_CHUNK
    for prefix in ("DTYPE_", "FLAG_", "DEVERR_"):
        theirs = {n[len("GDN_"):]: v for n, v in NUMBERS.items() if n.startswith("GDN_" + prefix)}
        assert theirs == {n: getattr(N, n) for n in dir(N) if n.startswith(prefix)} and theirs


def test_activations_reach_the_library_by_the_same_names():
    """The names that gdn_glu takes, as it lists them where it is given another."""
    import torch

    import gated_delta_rule_gate_gb300 as gdn
    from layer_standins import Standin
    x, w = (Standin(s, dtype=torch.float16) for s in ((20, 24), (16, 24)))
    with pytest.raises(ValueError) as e:
        gdn.gdn_glu(x, w, w, activation="")
    assert str(e.value).split(" of ")[1].split(", ") == list(N.ACTIVATIONS)
