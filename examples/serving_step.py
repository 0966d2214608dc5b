"""One serving step of many requests on block-quantized weights.

Every request has drafted a few tokens.  Their hidden states (random here, as
are the weights: the shapes are a small MoE model's) go through a projection
that all requests share plus each request's own low-rank adapter, through a
mixture of experts grouped by expert, and through the lm_head; the drafts are
then kept or replaced by the target's probabilities.

    python examples/serving_step.py [--requests 12] [--drafts 4] [--seed 0]

Prints each request's kept tokens and the one drawn after them.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import bandwidth_bound_block_amd as qmv  # noqa: E402
import workloads as wl  # noqa: E402

HIDDEN, FFN, EXPERTS, TOP_K, VOCAB, RANK, ADAPTERS = 512, 256, 16, 2, 1000, 8, 5


class Model:
    """Weights on the GPU: an adapted projection (Q4_0), experts (Q4_K) and an lm_head (Q8_0)."""

    def __init__(self, seed=0):
        def put(a):
            return torch.from_numpy(a.reshape(-1)).cuda()
        self.proj = put(wl.quant_weights("q4_0", f"example/{seed}/proj", HIDDEN, HIDDEN))
        self.gate_up = put(wl.quant_weights("q4_k", f"example/{seed}/gu", EXPERTS * 2 * FFN, HIDDEN))
        self.down = put(wl.quant_weights("q4_k", f"example/{seed}/down", EXPERTS * HIDDEN, FFN))
        self.head = put(wl.quant_weights("q8_0", f"example/{seed}/head", VOCAB, HIDDEN, std=0.2))
        g = torch.Generator().manual_seed(seed)
        self.router = torch.randn(HIDDEN, EXPERTS, generator=g).cuda()
        self.A = (torch.randn(ADAPTERS, RANK, HIDDEN, generator=g) * HIDDEN ** -0.5).bfloat16().cuda()
        self.B = (0.05 * torch.randn(ADAPTERS, HIDDEN, RANK, generator=g)).bfloat16().cuda()
        self.scales = torch.ones(ADAPTERS).cuda()

    def logits(self, x, adapter_ids):
        """x bfloat16 [tokens, HIDDEN], adapter_ids int32 [tokens] (-1: none) -> float32 [tokens, VOCAB]."""
        h = qmv.qmv_lora("q4_0", self.proj, HIDDEN, HIDDEN, x, self.A, self.B, self.scales, adapter_ids).bfloat16()
        top = torch.topk(h.float() @ self.router, TOP_K, dim=1)
        plan = qmv.qmv_group_plan(top.indices.to(torch.int32), EXPERTS)
        e = qmv.qmv_moe_grouped_swiglu("q4_k", self.gate_up, 2 * FFN * qmv.row_bytes("q4_k", HIDDEN), EXPERTS, FFN,
                                       HIDDEN, plan, TOP_K, h, h_dtype=torch.bfloat16)
        y = qmv.qmv_moe_grouped("q4_k", self.down, HIDDEN * qmv.row_bytes("q4_k", FFN), EXPERTS, HIDDEN, FFN, plan,
                                TOP_K, e)
        out = h + qmv.qmv_moe_weighted_sum(y, torch.softmax(top.values, dim=1), out_dtype=torch.bfloat16)
        # the lm_head is a matvec of up to 8 columns: a request's drafts at a time
        return torch.cat([qmv.qmv_matvec_xt("q8_0", self.head, VOCAB, HIDDEN, c.contiguous()) for c in out.split(8)])


def step(model, requests, drafts, seed=0):
    """Random drafted tokens and hidden states -> (drafted, tokens, kept)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(requests * (drafts + 1), HIDDEN, generator=g).bfloat16().cuda()
    owner = torch.randint(-1, ADAPTERS, (requests,), generator=g).repeat_interleave(drafts + 1).to(torch.int32).cuda()
    logits = model.logits(x, owner).view(requests, drafts + 1, VOCAB)
    # a draft model near the target: its own probabilities, and the tokens it drew from them
    near = logits[:, :drafts] + 0.5 * torch.randn(requests, drafts, VOCAB, generator=g).cuda()
    q = torch.softmax(near, dim=-1)
    pick = torch.searchsorted(q.double().cumsum(-1), torch.rand(requests, drafts, 1, generator=g).double().cuda() * 0.999999)
    drafted = pick.squeeze(-1).clamp_(max=VOCAB - 1).to(torch.int32)
    n = torch.full((requests,), drafts, dtype=torch.int32).cuda()
    u, u_last = torch.rand(requests, drafts, generator=g).cuda(), torch.rand(requests, generator=g).cuda()
    tokens, kept = qmv.qmv_spec_verify(logits, q, drafted, n, u, u_last)
    return drafted, tokens, kept


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=12)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    drafted, tokens, kept = step(Model(a.seed), a.requests, a.drafts, a.seed)
    for r, (k, t) in enumerate(zip(kept.tolist(), tokens.tolist())):
        print(f"request {r}: kept {k} of {a.drafts}: {t[:k]}, then {t[k]}")


if __name__ == "__main__":
    main()
