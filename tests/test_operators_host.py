"""What the Python entry points do on the host around a call: no GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# At one line event of a first call, another thread makes its first call too.
TWO_THREADS = r"""
import importlib, sys
import torch
import bandwidth_bound_block_amd as qmv

class OnGpu(torch.Tensor):
    is_cuda = True

def first_call():
    t = torch.zeros(4).as_subclass(OnGpu)
    assert qmv._type_of(t, "x") == qmv.X_F32
    assert qmv._scratch(None, "workspace", 16, torch.zeros(1), None).numel() >= 16

for at in range(1, 200):
    importlib.reload(qmv)
    seen = 0
    def trace(frame, event, arg):
        global seen
        if frame.f_code.co_filename != qmv.__file__:
            return None
        if event == "line":
            seen += 1
            if seen == at:
                sys.settrace(None)
                first_call()
        return trace
    sys.settrace(trace)
    first_call()
    sys.settrace(None)
    if seen < at:
        break
print("lines", at)
assert 5 < at < 199
"""


def test_first_calls_of_two_threads():
    r = subprocess.run([sys.executable, "-c", TWO_THREADS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
