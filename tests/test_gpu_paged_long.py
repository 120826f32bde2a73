"""Attention over the most positions a table may have: one page, repeated, so that the result
is a weighted mean of its rows with counts for weights."""
import pytest
import torch

import sparse_kv_prefetch_gb300 as dd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# tokens, d, dtype, q4
CASES = [(40, 128, BF, False), (40, 64, BF, False), (40, 256, BF, False), (40, 128, BF, True),
         (1, 128, BF, False), (1, 64, BF, True), (1, 64, F32, False), (20, 64, F32, False)]


@pytest.mark.parametrize("tokens,d,dtype,q4", CASES)
def test_sums_of_a_thousand_million_terms(tokens, d, dtype, q4):
    """Queries of 0 give every key the weight 1, exact in every type, and values in [1, 2) make the
    sums grow.  bf16: a term is cut by at most 2^-24 of the sum it meets, half the last one in the
    mean over a split's 2^18, which is 2^-7 of the result, which is rounded by 2^-8.  fp32: a warp
    adds 2^11 partial sums of 16 terms, each addition rounded by 2^-24 of a sum that is half the
    last in the mean, 2^-14, and as much again for the sum of the splits."""
    heads = 2
    n, page = (1 << 30) - 117, 128
    g = torch.Generator("cuda").manual_seed(d + tokens)
    pages = -(-n // page)
    shape = dd.PagedShape(1, heads, heads, d, page, 1, pages,
                          dd.DD_BF16 if dtype == BF else dd.DD_F32,
                          dd.DD_PAGES_Q4 if q4 else dd.DD_PAGES_PLAIN)
    if q4:  # 1 + c / 16
        codes = torch.randint(0, 16, (1, heads, page, d), device="cuda", generator=g)
        pair = torch.tensor([1 / 16, 1.0], device="cuda").bfloat16().expand(
            1, heads, page, d // 32, 2).contiguous()
        pool = torch.cat([(codes[..., 0::2] + 16 * codes[..., 1::2]).to(torch.uint8).flatten(2),
                          pair.flatten(2).view(torch.uint8)], 2)
        v = 1 + codes.double() / 16
    else:
        pool = (1 + torch.rand(1, heads, page, d, device="cuda", generator=g)).to(dtype)
        v = pool.double()
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    seqs = dd.PagedSeqs(torch.tensor([0, tokens], dtype=torch.int32).cuda(),
                        torch.tensor([n], dtype=torch.int32).cuda(), table, pool, pool)
    q = torch.zeros(tokens, heads, d, device="cuda", dtype=dtype)
    out, lse = torch.empty_like(q), torch.empty(tokens, heads, device="cuda")
    ws = torch.empty(dd.paged_attn_workspace_size(shape, tokens, tokens, n), dtype=torch.uint8,
                     device="cuda")
    dd.paged_attn(shape, seqs, q, out, lse, ws, max_q_len=tokens, max_kv_len=n)
    dd.check_device()
    seen = torch.arange(n - tokens + 1, n + 1, device="cuda")  # keys that a token sees
    count = seen[:, None] // page + (torch.arange(page, device="cuda") < seen[:, None] % page)
    want = torch.einsum("tr,hrd->thd", count.double(), v[0]) / seen[:, None, None]
    err = ((out.double() - want) / want).abs().max().item()
    assert err <= (2.0 ** -7 + 2.0 ** -8 if dtype == BF else 2.0 ** -13)
    assert ((lse.double() - seen.double().log()[:, None]).abs() <= 2.0 ** -19).all()
