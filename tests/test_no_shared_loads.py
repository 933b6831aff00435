"""Every CTA loads its own tiles: no source holds a tensor load that writes the
shared memory of several CTAs of a cluster at once.  Such a load is only sound on
this GPU's own memory, which an operand's address does not promise, and the same
library serves every replica of a run on several GPUs.  (The tensor cores' commits
to both CTAs of a pair arrive at barriers and move no data.)"""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "dense_fp32_matrix_03_gb300", "csrc", "*.*")))
STATEMENT = re.compile(r"cp\.async\.bulk[^;]*", re.S)


def statements(text):
    """The bulk copies of a source, strings that follow each other joined."""
    return STATEMENT.findall(re.sub(r'"\s*"', "", text))


def test_the_copies_are_found():
    found = sum(len(statements(open(p).read())) for p in SOURCES)
    assert found > 5
    split = '"cp.async.bulk.tensor.3d.shared::cluster.global.tile"\n    ".multi' + 'cast::cluster [%0];"'
    assert any("multi" + "cast" in s for s in statements(split))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_reaches_several_ctas(path):
    assert not [s for s in statements(open(path).read()) if "multi" + "cast" in s]
