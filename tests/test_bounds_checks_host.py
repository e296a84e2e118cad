"""The debug-bounds build checks the indexes of accesses: a condition that compares sizes
with one another, or with zero, is true whatever an index is, and checks nothing."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mamba_ssd_forward_gb300", "csrc")
# sizes and strides, by the names that these files give them
SIZES = {"rows", "cols", "D", "d", "L", "n", "ld", "ps", "zs", "ws", "V", "K", "N", "M", "team",
         "side", "parts", "count", "words", "runs", "a", "g", "qu", "in"}


def conditions(name):
    src = open(os.path.join(CSRC, name)).read()
    for m in re.finditer(r"SSD_IN_BOUNDS\(", src):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(src[at], 0)
            at += 1
        yield src[m.end():at - 1].rsplit(",", 2)


@pytest.mark.parametrize("name", ["add_norm.cu", "vocab_loss.cu", "orthogonalize.cu",
                                  "layer_colsum.cu"])
def test_every_check_bounds_an_index_from_above(name):
    seen = list(conditions(name))
    assert seen
    for cond, err, site in seen:
        for part in re.split(r"&&|\|\|", cond):
            if part.strip().startswith("!"):  # (a case that the check is not for)
                continue
            assert re.search(r"[^<]<=?[^<]", part), (name, site, part)
            index = re.split(r"<=?", part)[0]
            names = set(re.findall(r"[A-Za-z_]\w*", index))
            assert names - SIZES, (name, site, part)


def test_a_site_is_one_files():
    """What ssd_device_error reports says where to look."""
    files = {}
    for name in ("add_norm.cu", "vocab_loss.cu", "orthogonalize.cu"):
        for *_, site in conditions(name):
            assert files.setdefault(int(site), name) == name and int(site) >= 500
