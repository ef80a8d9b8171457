"""The build's dependencies, on the CPU: a source is compiled again when a header that it names changes."""
import os
import re

import pytest

pytest.importorskip("torch")
from sparse_attention_indexer_gb300 import build as M  # noqa: E402


def test_every_header_that_a_source_names_is_a_dependency(monkeypatch):
    deps = {}

    def stale(target, names):
        deps[os.path.basename(target)] = {os.path.basename(n) for n in names}
        return False

    def run(*a, **kw):
        raise AssertionError("nothing is out of date")

    monkeypatch.setattr(M, "_stale", stale)
    monkeypatch.setattr(M.subprocess, "run", run)
    M.build()

    def named(path):
        out = set()
        for name in re.findall(r'#include "([^"]+)"', open(path).read()):
            at = next(p for p in (os.path.join(M.CSRC, name), os.path.join(M.ROOT, "include", name)) if os.path.exists(p))
            out |= {os.path.basename(at)} | named(at)
        return out

    for src in M.SOURCES:
        missing = named(os.path.join(M.CSRC, src)) - deps[src.replace(".cu", ".o")]
        assert not missing, (src, missing)
