"""The binding's first calls from several threads at once: each is a call like any other."""
import os
import subprocess
import sys

import pytest

import fine_grained_moe_gate_b200 as moe

PROGRAM = """
import sys, threading
import torch
import fine_grained_moe_gate_b200 as moe
sys.setswitchinterval(float(sys.argv[1]))
n, errors, codes = 8, [], []
start = threading.Barrier(n)
sh = moe.MoEShape(0, 64, 16, 2, 128, 0, 128, moe.MOE_BF16)
opts = moe.MoERouteOpts(7, 1, 1, 1, 1, 1.0)  # no such score: refused before anything reaches a device

def call():
    start.wait()
    try:
        moe.moe_route_logits(None, None, sh, opts, None, None, None, stream=0)
    except moe.MoEError as e:
        codes.append(e.status)
    except BaseException as e:
        errors.append(repr(e))

threads = [threading.Thread(target=call) for _ in range(n)]
for t in threads: t.start()
for t in threads: t.join()
print(errors, codes)
sys.exit(0 if not errors and codes == [1] * n else 1)
"""


@pytest.mark.parametrize("interval", ["0.005", "1e-6"])
def test_first_calls_from_several_threads(interval):
    if not os.path.exists(moe.LIB_PATH):
        from fine_grained_moe_gate_b200 import build
        build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", PROGRAM, interval], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
