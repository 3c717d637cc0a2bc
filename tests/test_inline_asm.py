"""Inline assembly of the kernels names what it overwrites (text check, no GPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "scoring_exact_top_amd", "csrc")


def _blocks():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", open(path).read(), flags=re.S):
            yield os.path.basename(path), m.group(1)


def test_m0_is_declared():
    found = 0
    for name, text in _blocks():
        code = re.match(r'\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', text).group(1)
        if re.search(r"\bm0\b", code):
            found += 1
            assert text.count('"m0"') == 1, "%s: %s" % (name, code)
    assert found >= 2
