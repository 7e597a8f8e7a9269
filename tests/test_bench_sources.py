"""The bench pairs its times with committed traces and counters as long as the sources of the kernels
that it times are those they were taken from; sources of other operators do not part them."""
import os
import shutil

import pytest

import bench


@pytest.fixture
def csrc(tmp_path, monkeypatch):
    for name in os.listdir(bench.CSRC):
        if name.endswith((".hip", ".hpp")):
            shutil.copy(os.path.join(bench.CSRC, name), tmp_path)
    monkeypatch.setattr(bench, "CSRC", str(tmp_path))
    return tmp_path


def _changes(path):
    before = bench.kernel_source_hash()
    path.write_text(path.read_text() + "// changed\n")
    return bench.kernel_source_hash() != before


def test_estimators_sources_count(csrc):
    for name in ("est_vtrace.hip", "rlscan_kernel.hpp", "rlscan_launch.hpp", "rlscan_plan.hpp", "rlscan_tmdma.hpp"):
        assert _changes(csrc / name), name
    assert _changes(csrc / "est_gae.hip")


def test_other_operators_sources_do_not(csrc):
    for name in ("la_backward.hip", "la_forward.hip", "la_step.hip", "log_probs.hip", "sample_actions.hip",
                 "policy_api.hip", "rlscan_api.hip", "rlscan_la.hpp", "rlscan_logits.hpp"):
        assert not _changes(csrc / name), name
