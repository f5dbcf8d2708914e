"""The sources that key the committed DRAM traffic: all that the dominant kernel's code is made of."""
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

CSRC = os.path.join(ROOT, "rank_sum_reduce_gb300", "csrc")


def test_every_included_device_source_is_in_the_key():
    """Launch declarations (car_launch.h) hold no device code."""
    todo, seen = ["fused_tma.cu"], set()
    while todo:
        f = todo.pop()
        if f not in seen:
            seen.add(f)
            with open(os.path.join(CSRC, f)) as fh:
                todo += re.findall(r'#include "([^"]+)"', fh.read())
    assert seen - {"car_launch.h"} == set(bench.KERNEL_SOURCES)


def test_the_key_follows_every_source(monkeypatch, tmp_path):
    d = tmp_path / "rank_sum_reduce_gb300" / "csrc"
    d.mkdir(parents=True)
    for f in bench.KERNEL_SOURCES:
        (d / f).write_text("int x;\n")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    keys = {bench.kernel_source_hash()}
    for f in bench.KERNEL_SOURCES:
        (d / f).write_text("int y;\n")
        keys.add(bench.kernel_source_hash())
    assert len(keys) == 1 + len(bench.KERNEL_SOURCES)
