"""Argument errors of the grouped products, the adapters and the verification:
every call here is refused on the host before anything is launched (no GPU)."""
import re
import os

import pytest

EINVAL, EALIGN, EUNSUPPORTED = 1, 2, 3
A = 0x10000          # a fake, aligned, never dereferenced device address


@pytest.fixture(scope="module")
def qmv():
    import bandwidth_bound_block_amd as q
    return q


def check(qmv, name, good, changes):
    """good: argument names and values in order; changes: (changed arguments, code, word of the message)."""
    f = getattr(qmv.lib(), name)
    for change, code, word in changes:
        args = dict(good)
        assert set(change) <= set(args), change
        args.update(change)
        assert f(*args.values()) == code, (name, change, qmv.last_error())
        assert word in qmv.last_error(), (name, change, qmv.last_error())


def test_new_entry_points_are_declared_and_bound(qmv):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "qmv.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(qmv_\w+)\s*\(", src))
    new = {"qmv_group_plan", "qmv_moe_grouped", "qmv_moe_grouped_swiglu", "qmv_moe_weighted_sum", "qmv_lora", "qmv_spec_verify"}
    assert new <= names
    for n in new:
        assert n in qmv.__all__ and callable(getattr(qmv, n)) and getattr(qmv.lib(), n).argtypes


def test_size_functions(qmv):
    L = qmv.lib()
    assert L.qmv_group_plan_bytes(0, 4) == 0 and L.qmv_group_plan_bytes(4, 0) == 0
    assert L.qmv_group_plan_bytes(4, 1025) == 0 and L.qmv_group_plan_bytes((1 << 24) + 1, 4) == 0
    assert L.qmv_group_plan_bytes(1, 1) > 0
    # more items or groups never need less
    last = 0
    for n in (1, 7, 8, 100, 5000, 1 << 20, 1 << 24):
        b = L.qmv_group_plan_bytes(n, 8)
        assert b >= last + (4 if last else 0) and b >= 4 * n
        last = b
    assert L.qmv_lora_workspace_bytes(0, 1, 1) == 0 and L.qmv_lora_workspace_bytes(1, 129, 1) == 0
    assert L.qmv_lora_workspace_bytes(1, 1, 1025) == 0 and L.qmv_lora_workspace_bytes(1, 1, 1) > 0
    assert L.qmv_spec_verify_workspace_bytes(0, 1, 1) == 0 and L.qmv_spec_verify_workspace_bytes(1, 65, 1) == 0
    assert L.qmv_spec_verify_workspace_bytes(1, 1, (1 << 22) + 1) == 0
    assert L.qmv_spec_verify_workspace_bytes(65535, 64, 1 << 22) > 1 << 32


def test_group_plan_errors(qmv):
    need = qmv.lib().qmv_group_plan_bytes(10, 4)
    good = dict(ids=A, n=10, groups=4, plan=A, bytes=need, stream=None)
    check(qmv, "qmv_group_plan", good, [
        (dict(ids=0), EINVAL, "null"), (dict(plan=0), EINVAL, "null"),
        (dict(n=0), EINVAL, "n_items"), (dict(n=-1), EINVAL, "n_items"), (dict(n=(1 << 24) + 1), EINVAL, "n_items"),
        (dict(groups=0), EINVAL, "n_groups"), (dict(groups=1025), EINVAL, "n_groups"),
        (dict(bytes=need - 1), EINVAL, "bytes"),
        (dict(ids=A + 2), EALIGN, "aligned"), (dict(plan=A + 8), EALIGN, "aligned"),
    ])


@pytest.mark.parametrize("name,mul", [("qmv_moe_grouped", 1), ("qmv_moe_grouped_swiglu", 2)])
def test_grouped_errors(qmv, name, mul):
    good = dict(fmt=1, W=A, stride=mul * 8 * 36, E=4, rows=8, cols=64, plan=A, tokens=5, top_k=2, x=A, xt=2, xs=64, xslot=0,
                y=A, yt=0, stream=None)
    check(qmv, name, good, [
        (dict(fmt=9), EUNSUPPORTED, "format"),
        (dict(W=0), EINVAL, "null"), (dict(plan=0), EINVAL, "null"), (dict(x=0), EINVAL, "null"), (dict(y=0), EINVAL, "null"),
        (dict(xt=3), EINVAL, "x_type"), (dict(yt=-1), EINVAL, "output type"),
        (dict(E=0), EINVAL, "n_experts"), (dict(E=1025), EINVAL, "n_experts"),
        (dict(rows=0), EINVAL, "n_rows"), (dict(cols=48), EINVAL, "multiple of 32"), (dict(cols=0), EINVAL, "multiple"),
        (dict(fmt=3, cols=224, stride=1 << 20), EINVAL, "multiple of 256"),
        (dict(tokens=0), EINVAL, "n_tokens"), (dict(top_k=0), EINVAL, "top_k"), (dict(top_k=1025), EINVAL, "top_k"),
        (dict(tokens=(1 << 23) + 1), EINVAL, "n_tokens"),
        (dict(stride=mul * 8 * 36 - 4), EINVAL, "expert_stride_bytes"),
        (dict(xs=63), EINVAL, "x_stride_token"), (dict(xslot=63), EINVAL, "x_stride_slot"),
        (dict(W=A + 2), EALIGN, "aligned"), (dict(stride=mul * 8 * 36 + 1), EALIGN, "multiple of 2"),
        (dict(fmt=2, stride=mul * 8 * 40 + 2), EALIGN, "multiple of 4"), (dict(fmt=3, cols=256, xs=256, stride=(1 << 20) + 8), EALIGN, "multiple of 16"),
        (dict(fmt=3, cols=256, xs=256, W=A + 4, stride=1 << 20), EALIGN, "16-byte"),
        (dict(plan=A + 4), EALIGN, "plan"), (dict(x=A + 1), EALIGN, "aligned"), (dict(y=A + 2), EALIGN, "aligned"),
    ])


def test_weighted_sum_errors(qmv):
    good = dict(y=A, yt=0, w=A, tokens=5, top_k=2, rows=8, out=A, ot=2, stream=None)
    check(qmv, "qmv_moe_weighted_sum", good, [
        (dict(y=0), EINVAL, "null"), (dict(w=0), EINVAL, "null"), (dict(out=0), EINVAL, "null"),
        (dict(yt=5), EINVAL, "type"), (dict(ot=-2), EINVAL, "type"),
        (dict(tokens=0), EINVAL, "n_tokens"), (dict(top_k=0), EINVAL, "top_k"), (dict(rows=0), EINVAL, "n_rows"),
        (dict(y=A + 2), EALIGN, "aligned"), (dict(w=A + 2), EALIGN, "aligned"), (dict(out=A + 1), EALIGN, "aligned"),
    ])


def test_lora_errors(qmv):
    need = qmv.lib().qmv_lora_workspace_bytes(5, 4, 3)
    good = dict(fmt=1, W=A, rows=8, cols=64, x=A, xt=0, ldx=64, tokens=5, A=A, B=A, at=2, adapters=3, rank=4, scales=A,
                ids=A, y=A, ldy=8, ws=A, bytes=need, stream=None)
    check(qmv, "qmv_lora", good, [
        (dict(fmt=-1), EUNSUPPORTED, "format"),
        *[({k: 0}, EINVAL, "null") for k in ("W", "x", "A", "B", "scales", "ids", "y", "ws")],
        (dict(xt=3), EINVAL, "type"), (dict(at=3), EINVAL, "type"),
        (dict(rows=0), EINVAL, "n_rows"), (dict(cols=40), EINVAL, "multiple of 32"), (dict(cols=35456), EINVAL, "n_cols"),
        (dict(fmt=4, cols=64), EINVAL, "multiple of 256"),
        (dict(tokens=0), EINVAL, "n_tokens"), (dict(tokens=(1 << 20) + 1), EINVAL, "n_tokens"),
        (dict(adapters=0), EINVAL, "n_adapters"), (dict(adapters=1025), EINVAL, "n_adapters"),
        (dict(rank=0), EINVAL, "rank"), (dict(rank=129), EINVAL, "rank"),
        (dict(ldx=63), EINVAL, "ldx"), (dict(ldy=7), EINVAL, "ldy"), (dict(bytes=need - 1), EINVAL, "workspace"),
        (dict(W=A + 2), EALIGN, "aligned"), (dict(x=A + 2), EALIGN, "aligned"), (dict(A=A + 1), EALIGN, "aligned"),
        (dict(B=A + 1), EALIGN, "aligned"), (dict(y=A + 2), EALIGN, "aligned"), (dict(ws=A + 4), EALIGN, "aligned"),
        (dict(ids=A + 2), EALIGN, "aligned"), (dict(scales=A + 2), EALIGN, "aligned"),
    ])


def test_spec_verify_errors(qmv):
    need = qmv.lib().qmv_spec_verify_workspace_bytes(3, 4, 100)
    good = dict(l=A, lt=0, lr=500, ll=100, q=A, qr=400, ql=100, x=A, n=A, u=A, ul=A, requests=3, drafts=4, vocab=100, tokens=A,
                kept=A, ws=A, bytes=need, stream=None)
    check(qmv, "qmv_spec_verify", good, [
        *[({k: 0}, EINVAL, "null") for k in ("l", "x", "n", "u", "ul", "tokens", "kept", "ws")],
        (dict(lt=3), EINVAL, "logits_type"),
        (dict(requests=0), EINVAL, "n_requests"), (dict(requests=65536), EINVAL, "n_requests"),
        (dict(drafts=0), EINVAL, "max_drafts"), (dict(drafts=65), EINVAL, "max_drafts"),
        (dict(vocab=0), EINVAL, "vocab"), (dict(vocab=(1 << 22) + 1), EINVAL, "vocab"),
        (dict(ll=99), EINVAL, "strides"), (dict(lr=99), EINVAL, "strides"),
        (dict(ql=99), EINVAL, "strides"), (dict(qr=99), EINVAL, "strides"),
        (dict(bytes=need - 1), EINVAL, "workspace"),
        (dict(l=A + 2), EALIGN, "aligned"), (dict(q=A + 2), EALIGN, "aligned"), (dict(ws=A + 8), EALIGN, "aligned"),
        (dict(tokens=A + 1), EALIGN, "aligned"), (dict(kept=A + 2), EALIGN, "aligned"),
    ])
