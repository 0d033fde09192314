"""A warp whose lanes each test a barrier may get different answers, the barrier's completion
coming in between; what such a test decides holds warp synchronisation (barriers, votes, one
lane's arrival for all).  So kernels act on a vote over the lanes' answers only, never on a
lane's own.  A divergence cannot be brought about at will, so the sources are looked at."""
import pathlib
import re

import gated_deltanet_recurrence_02_gb300 as package

SOURCES = sorted((pathlib.Path(package.__file__).parent / "csrc").glob("*.cu"))


def test_lanes_act_on_a_vote():
    calls, alone = 0, []
    for path in SOURCES:
        text = re.sub(r"//[^\n]*", "", path.read_text())
        for m in re.finditer(r"\bmbar_test_wait\(", text):
            calls += 1
            if not re.search(r"__(all|any)_sync\(\w+,\s*!?$", text[:m.start()]):
                alone.append(f"{path.name}:{text[:m.start()].count(chr(10)) + 1}")
    assert calls >= 3 and not alone, f"a lane's own answer decides at {alone}"
