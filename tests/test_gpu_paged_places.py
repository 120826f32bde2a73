"""Attention of many tokens on grids with more places than multiprocessors, where a CTA goes
on with the work of places that have not started: barriers' phases, ring stages and tensor
memory are carried from one place to the next."""
import pytest
import torch

import sparse_kv_prefetch_gb300 as dd
from paged_util import Cache, check_attention

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_a_place_of_seconds_beside_short_ones():
    """Eight places of 200 million positions (one page, repeated) and 312 short ones.  The second
    row tile of every place is empty, so its warps wait for the work of the others, longer than
    any wait for a tile may last.

    The long sequence's queries are 0 and its values powers of two.  The weights are added up by
    tiles of 64, exact below 2^30, so lse is the logarithm of the number of positions, to the
    rounding of the last tile and of a number above 16 (2^-19 a step).  max_kv_len = 0 keeps the
    sums of 200 million values in one accumulator each.  Sums of up to 2^24 equal values are
    exact in fp32 however it adds them; beyond, terms may be lost (a tensor core cuts each term
    to its sum's last bits) but none is added twice, so a result lies between 2^24 / n of its
    value and the value, to the rounding to bf16."""
    heads, d, page, m, n_long = 8, 64, 128, 40, 200_000_011
    lens = [41 + 17 * b for b in range(39)]
    c = Cache([m] * 39, lens, heads, heads, d, page, BF, True, extra=1)
    spare = min(set(range(c.n_pages)) - set(c.table.flatten().tolist()))
    values = torch.tensor([(-1) ** h * 2.0 ** -h for h in range(heads)])
    pair = torch.zeros(heads, page, d // 32, 2)
    pair[..., 1] = values[:, None, None]
    for i in range(2):
        c.pools[i][spare] = 0
        c.pools[i][spare, :, page * d // 2:] = pair.bfloat16().flatten(1).view(torch.uint8).cuda()
    max_pages = -(-n_long // page)
    table = torch.full((40, max_pages), -1, dtype=torch.int32, device="cuda")
    table[0] = spare
    table[1:, :c.max_pages] = c.table.cuda()
    shape = dd.PagedShape(40, heads, heads, d, page, c.n_pages, max_pages, dd.DD_BF16,
                          dd.DD_PAGES_Q4)
    seqs = dd.PagedSeqs(torch.arange(0, 40 * m + 1, m, dtype=torch.int32).cuda(),
                        torch.tensor([n_long] + lens, dtype=torch.int32).cuda(), table, *c.pools)
    q = torch.cat([torch.zeros_like(c.q[:m]), c.q])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    assert dd.paged_attn_workspace_size(shape, 40 * m, m, 0) == 0  # not split
    dd.paged_attn(shape, seqs, q, out, lse, None, max_q_len=m, max_kv_len=0)
    dd.check_device()
    part = out[:m].cpu().double() / values.double()[None, :, None]
    assert (part >= 2.0 ** 24 / n_long * (1 - 2.0 ** -8)).all() and (part <= 1 + 2.0 ** -8).all()
    want = torch.arange(n_long - m + 1, n_long + 1, dtype=torch.double).log()
    assert ((lse[:m].cpu().double() - want[:, None]).abs() <= 2.0 ** -19 + 2.0 ** -22).all()
    check_attention(c, out[m:], lse[m:])


FORMS = [
    # heads, kv heads, d, page, q4
    (16, 8, 64, 32, False),
    (8, 8, 128, 16, False),
    (16, 8, 256, 64, False),
    (8, 8, 64, 128, True),
    (16, 8, 128, 64, True),
    (8, 8, 256, 16, True),
]


def mixed(n, seed):
    """n sequences of 0, 1, 33, 150 and 300 tokens, after odd numbers of others."""
    g = torch.Generator().manual_seed(seed)
    q_lens = [(0, 1, 33, 150, 300)[(b * 7 + seed) % 5] for b in range(n)]
    extra = (2 * torch.randint(0, 300, (n,), generator=g) + 1).tolist()
    return q_lens, [m + (0 if b % 4 == 0 else x) for b, (m, x) in enumerate(zip(q_lens, extra))]


def call(c, max_q, max_kv, window=0, sinks=0):
    """(out, lse, bytes of workspace); twice, the second time over the first one's results."""
    n = dd.paged_attn_workspace_size(c.shape, c.n_tokens, max_q, max_kv)
    ws = torch.empty(max(16, n), dtype=torch.uint8, device="cuda").fill_(255)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    seqs = c.seqs()
    first = None
    for _ in range(2):
        out.fill_(float("nan")), lse.fill_(float("nan"))
        dd.paged_attn(c.shape, seqs, c.q, out, lse, ws, max_q_len=max_q, max_kv_len=max_kv,
                      window=window, sinks=sinks)
        if first is None:
            first = out.clone()
    dd.check_device()
    assert torch.equal(out, first)
    return out, lse, n


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 0), (130, 70)])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_mixed_sequences_on_more_places_than_multiprocessors(form, window, sinks):
    heads, kv_heads, d, page, q4 = form
    q_lens, kv_lens = mixed(45, d + window)
    c = Cache(q_lens, kv_lens, heads, kv_heads, d, page, BF, q4, seed=d + sinks)
    c.poison(window, sinks)
    out, lse, _ = call(c, 300, max(kv_lens), window, sinks)
    check_attention(c, out, lse, window, sinks)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_split_prompts_on_more_places_than_multiprocessors(form):
    heads, kv_heads, d, page, q4 = form
    c = Cache([290, 300, 0, 300, 1, 300, 300, 33, 300, 300],
              [6001, 300, 0, 4999, 3001, 305, 700, 33, 911, 8999], heads, kv_heads, d, page, BF, q4)
    c.poison()
    out, lse, ws = call(c, 300, 20000)  # a hint at which every form is split
    assert ws > 2 * c.n_tokens * heads * d * 4  # at least two splits
    check_attention(c, out, lse)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_sequences_of_several_turns_of_the_grid(form):
    """More row tiles than the grid has places for: max_q_len is below the sequences' length."""
    heads, kv_heads, d, page, q4 = form
    lens = [300, 700, 1, 517, 0, 650] * 4
    c = Cache(lens, [n + 61 * (b % 3) for b, n in enumerate(lens)], heads, kv_heads, d, page, BF,
              q4)
    c.poison(250, 3)
    out, lse, _ = call(c, 40, 900, 250, 3)
    check_attention(c, out, lse, 250, 3)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_prompts_on_two_streams_at_once(form):
    """Two grids larger than the card beside each other, one of them split."""
    heads, kv_heads, d, page, q4 = form
    caches = [Cache(*mixed(45, 3), heads, kv_heads, d, page, BF, q4, seed=1),
              Cache([300] * 6, [300, 2000, 999, 5000, 301, 777], heads, kv_heads, d, page, BF, q4)]
    made = []
    for c, most in zip(caches, (900, 20000)):
        n = dd.paged_attn_workspace_size(c.shape, c.n_tokens, 300, most)
        made.append((c, c.seqs(), torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda"),
                     torch.empty(max(16, n), dtype=torch.uint8, device="cuda"), most))
    want = []
    for c, seqs, out, lse, ws, most in made:
        dd.paged_attn(c.shape, seqs, c.q, out, lse, ws, max_q_len=300, max_kv_len=most)
        check_attention(c, out, lse)
        want.append((out.clone(), lse.clone()))
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (c, seqs, out, lse, ws, most) in zip(streams, made):
            dd.paged_attn(c.shape, seqs, c.q, out, lse, ws, max_q_len=300, max_kv_len=most,
                          stream=st)
    torch.cuda.synchronize()
    for (o, l), (_, _, out, lse, _, _) in zip(want, made):
        assert torch.equal(o, out) and torch.equal(l, lse)
    dd.check_device()
