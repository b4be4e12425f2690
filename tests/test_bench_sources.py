"""The hash that ties bench.py's quoted DRAM traffic to the sources: it covers everything that
the decode step is compiled from, and changes with each of them."""

import os
import re
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join("linear_attention_decode_replay_b200", "csrc")


def compiled_into_the_step():
    """Its translation units, and what they include from the same folder."""
    found = [f for f in os.listdir(os.path.join(ROOT, CSRC))
             if re.fullmatch(r"replay_(api|small|kernels_\w+)\.cu", f)]
    for f in found:  # grows as includes are met
        with open(os.path.join(ROOT, CSRC, f)) as fh:
            found += [h for h in re.findall(r'#include "(\w[\w.]*)"', fh.read()) if h not in found]
    return sorted(found)


def test_the_hash_covers_the_decode_step():
    import bench

    assert sorted(bench.DECODE_SOURCES) == compiled_into_the_step()


@pytest.mark.parametrize("name", compiled_into_the_step())
def test_the_hash_changes_with_each_source(name, tmp_path, monkeypatch):
    import bench

    shutil.copytree(os.path.join(ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.kernel_sources_hash()
    with open(tmp_path / CSRC / name, "a") as f:
        f.write("// changed\n")
    assert bench.kernel_sources_hash() != before
