"""One definition for every name: the library's sources are compiled one by one and linked together, so a struct,
kernel or function of one name in one namespace must not be two things in two of them."""
from __future__ import annotations

import collections
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_recurrence_scan_reverse_amd", "csrc")

OPENS = re.compile(r"^(?:inline )?namespace (\w*) ?{")
CLOSES = re.compile(r"^}  // namespace")
TYPE = re.compile(r"^(?:struct|class|union|enum(?: class)?) (\w+)[^;]*{")
# a definition at the left edge that begins with no word that keeps it to its file
FUNCTION = re.compile(r"^(?!static|extern|using|typedef|template|struct|class|namespace|constexpr|return|#|/|\s)"
                      r"[\w:<>*& ,()\"]*?\b(\w+)\([^;]*$")


def definitions(path):
    """(namespaces, name) of what the file gives to the others, but for what has no linkage."""
    spaces, found = [], set()
    with open(path) as f:
        lines = f.read().split("\n")
    for line in lines:
        opened = OPENS.match(line)
        if opened:
            spaces.append(opened.group(1))
        elif CLOSES.match(line):
            spaces.pop()
        elif "" not in spaces:  # an unnamed namespace keeps its names
            for pattern in (TYPE, FUNCTION):
                m = pattern.match(line)
                if m and m.group(1) not in ("__launch_bounds__", "__attribute__"):
                    found.add((tuple(spaces), m.group(1)))
            m = re.match(r"^__global__ .*?\b(\w+_kernel)\(", line)
            if m:
                found.add((tuple(spaces), m.group(1)))
    return found


def test_every_name_has_one_definition():
    where = collections.defaultdict(list)
    for path in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
        for name in definitions(path):
            where[name].append(os.path.basename(path))
    assert (("rlscan", "gr"), "forward_kernel") in where and (("rlscan", "nr"), "Head") in where
    assert (("rlscan", "embed"), "SumArgs") in where and (("rlscan", "gr"), "make_plan") in where
    twice = {"::".join(n[0] + (n[1],)): files for n, files in where.items() if len(files) > 1}
    assert not twice, twice
