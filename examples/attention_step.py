"""Serving steps of one softmax-attention layer over the paged 4-bit cache: a prompt, then speculative steps of 4 drafts.

    python examples/attention_step.py

Every step: page plan (pages, slots, positions), norm + rotation of the projected rows with the store of their keys and
values, attention over the pages; after a speculative step each lane's length moves on by what it accepted.  The last step
is checked against attention in plain torch over the rows that the cache gives back."""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_mtp_gb300 as gdn  # noqa: E402

B, HQ, HK, D, R, PAGE, PAGES, WIDTH = 3, 16, 2, 128, 64, 64, 64, 16


def main():
    torch.manual_seed(0)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = gdn.Kv4Cache(torch.zeros((PAGES, 2, HK, PAGE, D // 2), dtype=torch.uint8, device="cuda"),
                         torch.zeros((PAGES, 2, HK, PAGE, D // 16), dtype=torch.uint8, device="cuda"))
    qw, kw = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    inv_freq = 1e6 ** (-torch.arange(0, R, 2, device="cuda") / R)
    lens, held, taken = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros(1, **i32)
    tables = torch.full((B, WIDTH), -1, **i32)
    free = torch.randperm(PAGES, device="cuda").int()
    ticket, err = torch.zeros(1, **i32), torch.zeros(1, **i32)

    def step(new):
        n = int(new.sum())
        qkv = torch.randn((n, HQ + 2 * HK, D), device="cuda").bfloat16()  # the layer's projection would give these
        q, k, v = qkv.split((HQ, HK, HK), 1)
        plan = gdn.PagePlan(torch.empty(B + 1, **i32), torch.empty(n, **i32), torch.empty(n, **i32), torch.empty(B, **i32),
                            held, taken)
        gdn.gdn_page_plan(lens, new, PAGE, tables, held, free, taken, plan, ticket, err)
        qr = torch.empty((n, HQ, D), dtype=torch.bfloat16, device="cuda")
        gdn.gdn_qk_norm_rope(q, k, qw, kw, plan.positions, inv_freq, qr, v=v, cache=cache, slot_map=plan.slot_map,
                             err_word=err)
        o, most = torch.empty_like(qr), int(new.max())
        gdn.gdn_kv4_attention(qr, cache, tables, plan.total_lens, o, gdn.kv4_attention_workspace(B, most, HQ, HK, D),
                              cu_seqlens=plan.cu_seqlens, max_q=most, err_word=err)
        return plan, qr, o

    plan, _, _ = step(torch.tensor([100, 1, 333], **i32))
    lens.copy_(plan.total_lens)
    for accepted in ((4, 1, 2), (1, 3, 4)):
        plan, qr, o = step(torch.full((B,), 4, **i32))
        total = plan.total_lens.tolist()
        lens += torch.tensor(accepted, **i32)
    assert int(err) == 0
    for b in range(B):
        L = total[b]
        j = torch.arange(L, device="cuda")
        k, v = (torch.empty((L, HK, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        gdn.gdn_kv4_read(cache, (tables[b, j // PAGE] * PAGE + j % PAGE).int(), k, v)
        rows = slice(4 * b, 4 * b + 4)
        kk, vv = (x.float().repeat_interleave(HQ // HK, 1) for x in (k, v))
        s = torch.einsum("thd,lhd->htl", qr[rows].float(), kk) / math.sqrt(D)
        s.masked_fill_(j > L - 4 + torch.arange(4, device="cuda")[:, None], -math.inf)
        want = torch.einsum("htl,lhd->thd", torch.softmax(s, -1), vv)
        assert (o[rows].float() - want).abs().max() < 2e-2
    print(f"attention steps ok: lengths {lens.tolist()}, pages held {held.tolist()}, pages taken {int(taken)}")


if __name__ == "__main__":
    main()
