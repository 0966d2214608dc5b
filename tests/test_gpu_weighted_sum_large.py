"""A weighted sum of more outputs than one launch has threads for, on an MI355X."""
import pytest

pytestmark = pytest.mark.gpu


def test_outputs_past_a_launch():
    import torch
    import bandwidth_bound_block_amd as qmv
    # 2^34 outputs, four to a thread: 2^32 threads
    T, n = 1 << 20, (1 << 14) + 4
    if torch.cuda.mem_get_info()[0] < 5 * T * n:
        pytest.skip("needs 86 GB of GPU memory")
    y = torch.empty((T, 1, n), dtype=torch.bfloat16, device="cuda")
    bits = y.view(torch.int16).view(-1)
    # small whole numbers of 7 bits that differ by place and by token: exact in bf16, as their products by 2
    row = (torch.arange(n, device="cuda") * 37 % 101).to(torch.bfloat16)
    for t in range(0, T, 1 << 16):
        y[t:t + (1 << 16), 0] = row + (torch.arange(t, t + (1 << 16), device="cuda") % 19).to(torch.bfloat16)[:, None]
    w = torch.full((T, 1), 2.0, device="cuda")
    out = torch.empty((T, n), dtype=torch.bfloat16, device="cuda")
    qmv.qmv_moe_weighted_sum(y, w, out=out)
    bits += 128                     # the exponent one up: doubled (zeros become the smallest normal)
    assert torch.equal(out[:1 << 15], torch.where(y[:1 << 15, 0] < 1e-30, 0, y[:1 << 15, 0]))
    for t in range(0, T, 1 << 16):
        a, b = out[t:t + (1 << 16)], y[t:t + (1 << 16), 0]
        assert bool(((a == b) | ((a == 0) & (b < 1e-30))).all()), t
    del y, out
    torch.cuda.empty_cache()
