"""Host checks of bench.py: which sources the stored HBM counters are tied to."""
import json
import os
import re
import shutil

import bench


def included(name, found):
    """name and every project header that it includes, directly or through others."""
    if name not in found:
        found.append(name)
        with open(os.path.join(bench.CSRC, name)) as f:
            for header in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                included(header, found)
    return found


def test_the_hash_covers_every_source_of_the_grouped_gemm():
    assert sorted(bench.GEMM_SRC) == sorted(included("grouped_gemm.hip", []))


def test_an_edit_of_any_of_them_changes_it(tmp_path):
    for name in bench.GEMM_SRC:
        for n in bench.GEMM_SRC:
            shutil.copy(os.path.join(bench.CSRC, n), tmp_path / n)
        assert bench.source_hash(folder=str(tmp_path)) == bench.source_hash()
        with open(tmp_path / name, "a") as f:
            f.write("// one more line\n")
        assert bench.source_hash(folder=str(tmp_path)) != bench.source_hash()


def test_counters_of_other_sources_are_not_reported(tmp_path, monkeypatch):
    stored = tmp_path / "traffic.json"
    monkeypatch.setattr(bench, "TRAFFIC_FILE", str(stored))
    for key, want in ((bench.source_hash(), 7), ("0" * 16, None)):
        stored.write_text(json.dumps({"layer": {"bytes_per_launch": 7, "kernel_source_sha256_16": key}}))
        assert bench.stored_traffic("layer") == want
        assert bench.stored_traffic("another") is None
