"""The counter summaries under profiles/ say how they were measured."""
import glob
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_traffic_summaries_hold_their_command():
    files = glob.glob(os.path.join(ROOT, "profiles", "traffic_*.json"))
    assert files
    for f in files:
        with open(f) as h:
            assert "rocprofv3" in json.load(h)["command"], f


def test_summary_without_a_command_is_refused():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--summarize-counters", "none.csv", "none.csv"],
                       cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 2 and "--command" in r.stderr
