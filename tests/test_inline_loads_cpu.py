"""Inline PTX that reads memory says so to the compiler, which otherwise may move or drop the stores it reads."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_19_gb300", "csrc")


def statements(text):
    """The asm statements of a source, each from `asm` to its closing parenthesis."""
    for m in re.finditer(r"\basm\b(\s+volatile)?\s*\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        yield text[m.start():at]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_loads_are_ordered_with_plain_stores(path):
    with open(path) as f:
        text = f.read()
    for s in statements(text):
        if re.search(r"\b(ld\.(volatile\.|relaxed\.|acquire\.)?(global|shared)|ldmatrix)", s):
            assert "volatile" in s.split("(")[0] and '"memory"' in s, s


def test_the_scan_sees_them():
    with open(os.path.join(CSRC, "fa_cache_ptx.cuh")) as f:
        assert sum("ld.global" in s for s in statements(f.read())) == 2
    assert list(statements('x; asm volatile("a (%0;" : "=r"(v) : "l"(p(1)));')) == ['asm volatile("a (%0;" : "=r"(v) : "l"(p(1)))']
