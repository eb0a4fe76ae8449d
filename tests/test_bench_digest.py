"""The digest that ties the bench's DRAM traffic figure to the kernel sources it
was taken on: it follows the kernels that the bench launches, and no others."""

from __future__ import annotations

import os

import bench


def test_digest_follows_the_benched_sources(tmp_path, monkeypatch):
    csrc = tmp_path / "varlen_flashattention_backward_gb300" / "csrc"
    os.makedirs(csrc)
    (csrc / "bwd.cu").write_text("a")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    first = bench.source_digest()
    (csrc / "paged_x.cu").write_text("b")
    assert bench.source_digest() == first
    (csrc / "bwd.cu").write_text("c")
    assert bench.source_digest() != first


def test_paged_sources_stand_alone():
    # What the digest leaves out is included by nothing that it covers.
    csrc = os.path.join(bench.ROOT, "varlen_flashattention_backward_gb300", "csrc")
    for name in os.listdir(csrc):
        if not name.startswith("paged"):
            with open(os.path.join(csrc, name)) as f:
                assert '#include "paged' not in f.read()
