"""The recorded DRAM traffic of the attention call holds for the sources it was taken
on, and every file that is compiled into the kernel counts as one."""
import hashlib
import os
import re

import bench

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_diffusion_speculative_attn_gb300", "csrc")


def test_every_header_of_the_kernel_counts():
    todo, seen = ["block_attn.cu"], set()
    while todo:
        f = todo.pop()
        if f in seen:
            continue
        seen.add(f)
        with open(os.path.join(CSRC, f)) as fh:
            todo += [i for i in re.findall(r'^#include "([^"]+)"', fh.read(), re.M)
                     if not i.startswith("..")]  # (the public header: declarations)
    assert seen == {os.path.basename(f) for f in bench.ATTN_SOURCES}


def test_traffic_is_of_its_sources(monkeypatch):
    name, n = bench.ATTN_TRAFFIC["workload"], bench.ATTN_TRAFFIC["bytes_per_call"]
    h = hashlib.sha256()
    for f in bench.ATTN_SOURCES:
        with open(os.path.join(bench.ROOT, f), "rb") as fh:
            h.update(fh.read())
    now = dict(bench.ATTN_TRAFFIC, sources_sha256=h.hexdigest())
    monkeypatch.setattr(bench, "ATTN_TRAFFIC", now)
    assert bench.attn_traffic(name) == n
    assert bench.attn_traffic("another workload") is None
    monkeypatch.setattr(bench, "ATTN_TRAFFIC", dict(now, sources_sha256="0" * 64))
    assert bench.attn_traffic(name) is None
