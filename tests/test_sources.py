"""Forms that the kernels' sources keep away from."""
import glob
import os
import re

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "bwd_ssm_conv_gb300", "csrc", "*.cu*")))
# a loop without braces of its own behind `if constexpr`: nvcc 13.0.88 drops the loop after a discarded one
# where that has a `#pragma unroll`
LOOP = re.compile(r"if constexpr \([^\n]*\)[ \t]*\n?[ \t]*(while|for|do)\b")


def _behind(text):
    return LOOP.search(re.sub(r"//[^\n]*", "", text))


def test_loops_behind_if_constexpr_have_braces():
    assert SOURCES
    for bad in ("if constexpr (P > 1)\n  while (n > 0) n--;", "if constexpr (P > f(1)) for (;;) n--;",
                "if constexpr (P > 1)  // why\n  do n--; while (n);"):
        assert _behind(bad)
    assert not _behind("if constexpr (P > 1) {\n  while (n > 0) n--;\n}")
    for path in SOURCES:
        with open(path) as f:
            found = _behind(f.read())
        assert not found, (path, found.group(0))
