"""What the Python entry points do on the host around a call: no GPU."""
import contextlib
import inspect
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

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


# ------------------------------------------------------- tensors and streams
# Stand-ins: CPU tensors that say they are on a GPU, streams that are a name,
# a library whose calls succeed without doing anything.
class OnGpu(torch.Tensor):
    is_cuda = True
    pool = None

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.recorded = getattr(self, "recorded", []) + [s]


class Stand:
    def __init__(self, monkeypatch, qmv):
        self.main, self.side = SimpleNamespace(cuda_stream=11), SimpleNamespace(cuda_stream=22)
        self.current, self.made, self.calls = self.main, [], []
        empty = torch.empty

        def made(*a, **k):
            t = empty(*a, **k).as_subclass(OnGpu)
            t.pool = self.current
            self.made.append(t)
            return t

        @contextlib.contextmanager
        def entered(s):
            before, self.current = self.current, s
            yield
            self.current = before

        class Lib:
            def __getattr__(lib, name):
                if name.endswith("_bytes"):
                    return lambda *a: 64
                return lambda *a: self.calls.append((name, a[-1])) or 0
        monkeypatch.setattr(qmv, "_lib", Lib())
        monkeypatch.setattr(torch, "empty", made)
        monkeypatch.setattr(torch.cuda, "stream", entered)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: self.current.cuda_stream, raising=False)


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def raw(n):
    return gpu(n, dtype=torch.uint8)


def ids(*shape):
    return gpu(*shape, dtype=torch.int32)


def i8(*shape):
    return gpu(*shape, dtype=torch.int8)


def plan_of(q):
    return q.GroupPlan(raw(64), 6, 4)


MOE = (4 * 8 * 36, 4, 8, 64)          # stride, experts, rows, columns
CALLS = {
    "qmv_q8_0": lambda q, s: q.qmv_q8_0(raw(8 * 68), 8, 64, gpu(2, 64), stream=s),
    "qmv_q4_0": lambda q, s: q.qmv_q4_0(raw(8 * 36), 8, 64, gpu(64), stream=s),
    "qmv_q4_1": lambda q, s: q.qmv_q4_1(raw(8 * 40), 8, 64, gpu(64), stream=s),
    "qmv_q4_k": lambda q, s: q.qmv_q4_k(raw(8 * 144), 8, 256, gpu(256), stream=s),
    "qmv_q6_k": lambda q, s: q.qmv_q6_k(raw(8 * 210), 8, 256, gpu(256), stream=s),
    "qmv_matvec_path": lambda q, s: q.qmv_matvec_path("q4_0", raw(8 * 36), 8, 64, gpu(64), q.PATH_FMA, stream=s),
    "qmv_matvec_xt": lambda q, s: q.qmv_matvec_xt("q4_0", raw(8 * 36), 8, 64, gpu(3, 64, dtype=torch.float16), stream=s),
    "qmv_i8_requant": lambda q, s: q.qmv_i8_requant(i8(8, 16), i8(2, 16), ids(8), ids(8), stream=s),
    "qmv_i8_requant_lut": lambda q, s: q.qmv_i8_requant_lut(i8(8, 16), i8(2, 16), ids(8), ids(8), i8(256), stream=s),
    "qmv_moe": lambda q, s: q.qmv_moe("q4_0", raw(4 * MOE[0]), *MOE, ids(3, 2), gpu(3, 64), stream=s),
    "qmv_moe_xt": lambda q, s: q.qmv_moe_xt("q4_0", raw(4 * MOE[0]), *MOE, ids(3, 2), gpu(3, 64), stream=s),
    "qmv_moe_swiglu": lambda q, s: q.qmv_moe_swiglu("q4_0", raw(8 * MOE[0]), *MOE, ids(3, 2), gpu(3, 64), stream=s),
    "qmv_moe_swiglu_xt": lambda q, s: q.qmv_moe_swiglu_xt("q4_0", raw(8 * MOE[0]), *MOE, ids(3, 2), gpu(3, 64), stream=s),
    "qmv_moe_combine": lambda q, s: q.qmv_moe_combine("q4_0", raw(4 * MOE[0]), *MOE, ids(3, 2), gpu(3, 2), gpu(3, 2, 64),
                                                      stream=s),
    "qmv_group_plan": lambda q, s: q.qmv_group_plan(ids(6), 4, stream=s),
    "qmv_moe_grouped": lambda q, s: q.qmv_moe_grouped("q4_0", raw(4 * MOE[0]), *MOE, plan_of(q), 2, gpu(3, 64), stream=s),
    "qmv_moe_grouped_swiglu": lambda q, s: q.qmv_moe_grouped_swiglu("q4_0", raw(8 * MOE[0]), *MOE, plan_of(q), 2, gpu(3, 64),
                                                                    stream=s),
    "qmv_moe_weighted_sum": lambda q, s: q.qmv_moe_weighted_sum(gpu(3, 2, 8), gpu(3, 2), stream=s),
    "qmv_lora": lambda q, s: q.qmv_lora("q4_0", raw(8 * 36), 8, 64, gpu(3, 64), gpu(2, 4, 64), gpu(2, 8, 4), gpu(2), ids(3),
                                        stream=s),
    "qmv_spec_verify": lambda q, s: q.qmv_spec_verify(gpu(2, 4, 9), gpu(2, 3, 9), ids(2, 3), ids(2), gpu(2, 3), gpu(2), stream=s),
    "qmv_dequant": lambda q, s: q.qmv_dequant("q4_0", raw(8 * 36), 8, 64, stream=s),
}


@pytest.fixture()
def stand(monkeypatch):
    import bandwidth_bound_block_amd as qmv
    return Stand(monkeypatch, qmv), qmv


def test_every_entry_point_with_outputs_is_here():
    import bandwidth_bound_block_amd as qmv
    with_stream = {n for n in qmv.__all__ if n.startswith("qmv_") and "stream" in inspect.signature(getattr(qmv, n)).parameters}
    assert with_stream - {"qmv_chain", "qmv_chain_noalloc", "qmv_stream_read"} == set(CALLS)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_new_tensors_come_from_the_pool_of_the_calls_stream(stand, name):
    """A block of the current stream's pool may still be in use by work queued there, which another stream does not wait
    for, and goes back to that pool while the other stream still writes it."""
    st, qmv = stand
    out = CALLS[name](qmv, st.side)
    assert st.made and all(t.pool is st.side for t in st.made)
    assert st.current is st.main
    assert all(getattr(s, "value", s) == 22 for _, s in st.calls)
    # what is returned is read on the current stream too (after a wait), and does not go back before that
    for t in out if isinstance(out, tuple) else (out.buffer if isinstance(out, qmv.GroupPlan) else out,):
        assert st.main in t.recorded


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("given", [False, True])
def test_nothing_is_recorded_on_the_current_stream(stand, name, given):
    st, qmv = stand
    CALLS[name](qmv, st.main if given else None)
    assert st.made and all(t.pool is st.main and not hasattr(t, "recorded") for t in st.made)
    assert all(getattr(s, "value", s) == 11 for _, s in st.calls)


@pytest.mark.parametrize("name", ["qmv_moe_grouped", "qmv_moe_grouped_swiglu"])
def test_a_plan_read_on_another_stream_is_kept_for_it(stand, name):
    st, qmv = stand
    f = getattr(qmv, name)

    def product(plan, s):
        f("q4_0", raw(8 * MOE[0]), *MOE, plan, 2, gpu(3, 64), stream=s)
    plan = qmv.qmv_group_plan(ids(3, 2), 4)
    product(plan, None)
    assert not hasattr(plan.buffer, "recorded")
    product(plan, st.side)
    assert plan.buffer.recorded == [st.side]
    plan = qmv.qmv_group_plan(ids(3, 2), 4, stream=st.side)
    before = list(plan.buffer.recorded)
    product(plan, st.side)
    assert plan.buffer.recorded == before
    product(plan, None)
    assert plan.buffer.recorded == before + [st.main]
    given = raw(64)
    plan = qmv.qmv_group_plan(ids(3, 2), 4, plan=given)      # whose pool it is from is not known
    product(plan, None)
    assert given.recorded == [st.main]
