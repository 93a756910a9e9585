"""The benchmark's distillation command: one JSON line over the four
operators and the AdamW step that takes their gradient."""

from __future__ import annotations

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bench(args):
    return subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *args], capture_output=True, text=True,
                          timeout=300, cwd=ROOT)


def test_bench_distill_line():
    r = _bench(["--distill", "--steps", "3", "--warmup", "1"])
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [ln for ln in r.stdout.splitlines() if ln.strip()]
    assert len(lines) == 1
    d = json.loads(lines[0])
    assert d["steps"] == 3 and d["warmup"] == 1 and d["n_gpus"] == 1 and d["value"] > 0
    assert d["config"]["workload"] == "dense800m" and d["config"]["vocab"] == 32000
    assert set(d["kernels"]) == {"logprobs", "mx4_quant", "mx4_matmul", "distill", "adamw"}
    for name, k in d["kernels"].items():
        assert 0 < k["frac"] < 1, name
    assert 0 < d["roofline"]["frac"] < 1
    assert d["loss_mean"] >= 0.0
    r = _bench(["--distill", "--workload", "large_n5", "--steps", "1"])
    assert r.returncode == 2 and "LM head" in r.stderr
