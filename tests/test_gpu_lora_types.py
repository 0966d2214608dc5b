"""Adapters: every pair of activation and adapter types, and the base up to 8 tokens at fp32's bound, on an MI355X."""
import numpy as np
import pytest

from tests import operator_values as ov
from tests.test_gpu_lora import Case, FORMATS, assert_close, env  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = ["f32", "f16", "bf16"]


@pytest.mark.parametrize("x_name", TYPES)
@pytest.mark.parametrize("a_name", TYPES)
@pytest.mark.parametrize("fmt", ["q4_0", "q6_k"])
@pytest.mark.parametrize("T,N,R", [(5, 90, 12), (40, 130, 12), (40, 70, 100), (8, 70, 128), (1, 300, 128)])
def test_every_pair_of_types(env, x_name, a_name, fmt, T, N, R):  # noqa: F811
    torch, qmv = env
    print("lora types", fmt, x_name, a_name, T, N, R, flush=True)
    c = Case(torch, fmt, T, N, 512, R, 3, x_name, a_name)
    y, e, d = c.expect()
    if T <= 8 and x_name == "f32":
        # the FMA kernels: fp32's own bound in place of the matrix cores'
        base, eb = ov.product(fmt, c.raw, N, 512, c.x)
        e = eb + ov.adapters(c.x, c.A, c.B, c.scales, c.ids)[1] + 2 * ov.U * (np.abs(base) + np.abs(d))
    assert_close(c.run(torch, qmv), y, e, (x_name, a_name))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8])
def test_fp32_base_of_few_tokens_is_the_fma_kernels(env, fmt, T):  # noqa: F811
    """1100 rows of 512 columns: a size at which the matvec by itself takes its matrix cores at some of these widths."""
    torch, qmv = env
    c = Case(torch, fmt, T, 1100, 512, 4, 2, "f32", "bf16", ids=np.full(T, -1))
    want = qmv.qmv_matvec_path(fmt, torch.from_numpy(c.raw.reshape(-1)).cuda(), 1100, 512, c.xt.cuda(), qmv.PATH_FMA)
    assert torch.equal(c.run(torch, qmv), want)
