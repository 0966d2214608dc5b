"""Sizes within the documented ranges whose launch would pass 2^32 threads: refused on the host, before anything is launched
(no GPU)."""
import pytest

EINVAL = 1
A = 0x10000          # a fake, aligned, never dereferenced device address


@pytest.mark.parametrize("name,rows", [("qmv_moe_grouped", 1 << 28), ("qmv_moe_grouped_swiglu", 1 << 27)])
@pytest.mark.parametrize("xt", [0, 1, 2])
def test_products_past_a_launch(name, rows, xt):
    import bandwidth_bound_block_amd as qmv
    stride = (1 << 28) * 18
    f = getattr(qmv.lib(), name)
    # 64 items in up to 10 tiles of 32, by 2^21 tiles of rows
    assert f(1, A, stride, 8, rows, 32, A, 64, 1, A, xt, 32, 0, A, 0, None) == EINVAL, qmv.last_error()
    assert "launch" in qmv.last_error() and "tiles" in qmv.last_error()


def test_lora_columns():
    """Up to 8 tokens rows are the matvec's; past that only 2^24 columns bound them, and a bad size is still refused."""
    import bandwidth_bound_block_amd as qmv
    f = qmv.lib().qmv_lora

    def call(tokens, cols):
        need = qmv.lib().qmv_lora_workspace_bytes(tokens, 4, 3)
        # a workspace a byte short: the check after the sizes, before any launch
        return f(1, A, 8, cols, A, 0, cols, tokens, A, A, 2, 3, 4, A, A, A, 8, A, need - 1, None), qmv.last_error()
    for tokens, cols, word in ((8, 35424, "workspace"), (8, 35456, "n_cols"), (9, 35456, "workspace"), (9, 1 << 24, "workspace"),
                               (9, (1 << 24) + 32, "n_cols"), (9, 35457, "n_cols")):
        code, error = call(tokens, cols)
        assert code == EINVAL and word in error, (tokens, cols, error)
