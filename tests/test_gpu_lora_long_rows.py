"""Adapters beside rows longer than the matvec's (35424 columns): past 8 tokens the base is the tile product, which has no such
limit."""
import pytest

from tests.test_gpu_lora import Case, assert_close, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,K", [("q8_0", 35456), ("q4_0", 35424 + 64), ("q4_1", 40000), ("q4_k", 36096), ("q6_k", 51200)])
@pytest.mark.parametrize("T,N,x_name,a_name", [(9, 40, "bf16", "bf16"), (33, 150, "f32", "f16"), (140, 30, "f16", "f32")])
def test_rows_past_the_matvecs(env, fmt, K, T, N, x_name, a_name):
    torch, qmv = env
    print("lora long", fmt, K, T, N, x_name, a_name, flush=True)
    c = Case(torch, fmt, T, N, K, 8, 3, x_name, a_name)
    y, e, _ = c.expect()
    assert_close(c.run(torch, qmv), y, e)
    c = Case(torch, fmt, 8, N, K, 8, 3, x_name, a_name)
    with pytest.raises(qmv.QmvError, match="n_cols"):
        c.run(torch, qmv)
