"""The package imports, and all its names can be taken, without torch: only calls need it."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_names_without_torch():
    # a None entry makes `import torch` raise ImportError
    r = _python("""
import sys
sys.modules["torch"] = None
from linear_recurrence_scan_reverse_amd import *
import linear_recurrence_scan_reverse_amd as rl
assert all(callable(globals()[n]) for n in rl.__all__)
for call in (lambda: linear_attention(1, 2, 3, 4), lambda: linear_attention_step(1, 2, 3, 4, 5),
             lambda: linear_attention_backward(1, 2, 3, 4, 5), lambda: sample_actions(1, 2),
             lambda: action_log_probs(1, 2), lambda: action_log_probs_backward(1, 2, 3, 4, 5, 6)):
    try:
        call()
    except ImportError:
        continue
    raise AssertionError("a call without torch")
""")
    assert r.returncode == 0, r.stderr


def test_names_do_not_load_torch():
    r = _python("""
import sys
from linear_recurrence_scan_reverse_amd import *
assert "torch" not in sys.modules
try:
    sample_actions([1.0], None)
except TypeError:
    assert "torch" in sys.modules
""")
    assert r.returncode == 0, r.stderr
