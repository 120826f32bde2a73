"""Calls of the paged cache that the documentation allows: hints far off, captures, strides,
infinities."""
import pytest
import torch

import sparse_kv_prefetch_gb300 as dd
from paged_util import Cache, check_attention, run_attention

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,q4", [(BF, False), (BF, True), (F32, False)])
def test_a_length_hint_beyond_the_call_costs_nothing(dtype, q4):
    """The grid follows the call's tokens where max_q_len is larger: with a place for each of 2^31
    rows the call below would have 33 million CTAs."""
    c = Cache([1, 0] * 32, [3 + b for b in range(64)], 8, 8, 64, 16, dtype, q4)
    out, lse = run_attention(c, max_q=2 ** 31 - 1)
    check_attention(c, out, lse)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    run_attention(c, max_q=2 ** 31 - 1)
    b.record()
    b.synchronize()
    assert a.elapsed_time(b) < 20
    dd.check_device()


def captured_split_call(heads, kv_heads, d, page, dtype, q4, tokens, most):
    """A call that is split and merged through the workspace, captured as the first of its kind
    and replayed over other lengths, tables and pools, the workspace full of NaN each time."""
    lens = [([tokens, tokens], [most, tokens + 1]), ([1, 2 * tokens - 1], [17, most - 40]),
            ([2 * tokens, 0], [most - 3, 9])]
    if tokens == 1:
        lens = [([1, 1], [most, 2]), ([1, 1], [17, most - 40]), ([0, 1], [9, most - 3])]
    caches = [Cache(q, n, heads, kv_heads, d, page, dtype, q4, seed=i, behind=2 * tokens - sum(q),
                    extra=2 * -(-most // page) - sum(-(-x // page) for x in n))
              for i, (q, n) in enumerate(lens)]
    rows = max(c.max_pages for c in caches)
    T, n_pages = 2 * tokens, caches[0].n_pages
    shape = dd.PagedShape(2, heads, kv_heads, d, page, n_pages, rows, caches[0].shape.dtype,
                          caches[0].shape.format)
    pools = [torch.zeros_like(p) for p in caches[0].pools]
    q_start, seq_len = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (3, 2))
    table = torch.full((2, rows), -1, dtype=torch.int32, device="cuda")
    q = torch.zeros(T, heads, d, dtype=dtype, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(T, heads, device="cuda")
    seqs = dd.PagedSeqs(q_start, seq_len, table, *pools)
    size = dd.paged_attn_workspace_size(shape, T, T if tokens > 1 else 1, 40000)
    splits = size // (T * heads * (4 * d + 8))
    assert splits > 8 if tokens == 1 else splits > 1
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dd.paged_attn(shape, seqs, q, out, lse, ws, max_q_len=T if tokens > 1 else 1,
                      max_kv_len=40000)
    for c in caches:
        assert c.n_pages == n_pages
        c.poison()
        for p, x in zip(pools, c.pools):
            p.copy_(x)
        q_start.copy_(torch.tensor(c.q_start, dtype=torch.int32))
        seq_len.copy_(torch.tensor(c.kv_lens, dtype=torch.int32))
        table.fill_(-1)
        table[:, :c.max_pages] = c.table.cuda()
        q.copy_(c.q)
        ws.fill_(255)
        out.fill_(3.0)
        graph.replay()
        check_attention(c, out, lse)
        assert (out[c.q_start[2]:] == 3).all()  # rows of no sequence
    dd.check_device()


MERGED = [(8, 2, 128, 64, BF, False), (4, 4, 64, 16, F32, False), (8, 1, 256, 32, BF, False),
          (2, 2, 64, 16, BF, True)]


# (fp32 calls of many rows are split into clusters, which need no workspace)
@pytest.mark.parametrize("form,tokens", [(f, t) for f in MERGED for t in (1, 40)
                                         if t == 1 or f[4] == BF])
def test_captured_split_calls(form, tokens):
    captured_split_call(*form, tokens, 9000)


def test_the_first_call_of_a_process_may_be_a_captured_split_one():
    """In a process of its own, where no kernel has been used before the capture."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import torch, test_gpu_paged_calls as t\n"
            "t.captured_split_call(8, 2, 128, 64, torch.bfloat16, False, 1, 9000)\n"
            "t.captured_split_call(8, 2, 128, 64, torch.bfloat16, True, 40, 3000)\n"
            % (os.path.dirname(here), here))
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


F32_FORMS = [(4, 4, 64, 16), (8, 1, 128, 16), (2, 2, 128, 64)]


@pytest.mark.parametrize("tokens,most", [(1, 0), (1, 20000), (3, 0), (50, 0)])
@pytest.mark.parametrize("form", F32_FORMS, ids=lambda f: "-".join(map(str, f)))
def test_fp32_keys_of_logit_minus_infinity_have_no_weight(form, tokens, most):
    """Pages whose every key has the logit -infinity for every query count as no page."""
    heads, kv_heads, d, page = form
    c = Cache([tokens, tokens], [900, tokens + 70], heads, kv_heads, d, page, F32)
    c.q[..., 5] = c.q[..., 5].abs() + 0.25
    for b, i in ((0, 3), (0, 7), (1, 0)):
        c.pools[0][int(c.table[b, i]), :, :, 5] = -torch.inf
    out, lse = run_attention(c, max_kv=max(most, 900))
    for b, i in ((0, 3), (0, 7), (1, 0)):
        c.table[b, i] = -1
    check_attention(c, out, lse)
    dd.check_device()


@pytest.mark.parametrize("tokens,most", [(1, 0), (1, 20000), (3, 0), (50, 0)])
@pytest.mark.parametrize("form", F32_FORMS, ids=lambda f: "-".join(map(str, f)))
def test_fp32_infinite_values_stay_in_their_elements_and_rows(form, tokens, most):
    """A token that sees an infinite value has it in that element and no other; a token that does
    not has none; of a key with logit +infinity nothing is known but that rows before it are
    untouched."""
    heads, kv_heads, d, page = form
    n, at = 900, 899 - tokens // 2
    c = Cache([tokens, 1], [n, 33], heads, kv_heads, d, page, F32)
    where = (int(c.table[0, at // page]), slice(None), at % page)
    c.pools[1][where + (9,)] = torch.inf
    out, lse = run_attention(c, max_kv=max(most, n))
    sees = slice(at - (n - tokens), tokens)
    assert (out[sees, :, 9] == torch.inf).all()
    c.pools[1][where + (9,)] = 0.5
    fixed, _ = run_attention(c)
    out[sees, :, 9] = fixed[sees, :, 9]
    check_attention(c, out, lse)
    c.pools[0][where + (5,)] = torch.inf
    out, lse = run_attention(c, max_kv=max(most, n))
    before = torch.ones(tokens + 1, dtype=torch.bool)
    before[sees] = False
    assert out[before].isfinite().all() and lse[before].isfinite().all()
    c.pools[0][where + (5,)] = 0.0
    fixed, fixed_lse = run_attention(c)
    out[sees], lse[sees] = fixed[sees], fixed_lse[sees]
    check_attention(c, out, lse)


def test_a_table_with_rows_of_another_length_is_refused():
    """The kernels step from row to row by max_pages; a flat table has no rows to compare."""
    c = Cache([1, 1], [40, 30])
    wide = torch.full((2, c.max_pages + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.max_pages] = c.table.cuda()
    q_start, seq_len = (torch.tensor(x, dtype=torch.int32).cuda() for x in (c.q_start, c.kv_lens))
    out = torch.empty_like(c.q)
    with pytest.raises(ValueError):
        dd.paged_attn(c.shape, dd.PagedSeqs(q_start, seq_len, wide, *c.pools), c.q, out,
                      max_q_len=1, max_kv_len=40)
    with pytest.raises(ValueError):
        dd.paged_read(c.shape, dd.PagedSeqs(None, seq_len, wide, *c.pools), 0, 1, out, out)
    flat = dd.PagedSeqs(q_start, seq_len, c.table.cuda().flatten(), *c.pools)
    out, lse = run_attention(c, seqs=flat)
    check_attention(c, out, lse)


def test_a_workspace_by_its_address():
    """Raw addresses with their size, as the other calls take them."""
    c = Cache([1], [9000])
    n = dd.paged_attn_workspace_size(c.shape, 1, 1, 9000)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(1, 8, device="cuda")
    kw = dict(max_q_len=1, max_kv_len=9000)
    dd.paged_attn(c.shape, c.seqs(), c.q, out, lse.data_ptr(), ws.data_ptr(), ws_bytes=n, **kw)
    check_attention(c, out, lse)
    with pytest.raises(dd.DDError):
        dd.paged_attn(c.shape, c.seqs(), c.q, out, lse, ws.data_ptr(), ws_bytes=n - 1, **kw)
    with pytest.raises(dd.DDError):
        dd.paged_attn(c.shape, c.seqs(), c.q, out, lse, ws, ws_bytes=n - 1, **kw)


@pytest.mark.parametrize("tokens,most", [(1, 0), (1, 20000), (3, 0), (50, 0), (50, 20000)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_bf16_keys_of_logit_minus_infinity_have_no_weight(d, tokens, most):
    """Pages whose every key has the logit -infinity for every query count as no page."""
    c = Cache([tokens, tokens], [900, tokens + 70], 8, 2, d, 32)
    c.q[..., 5] = c.q[..., 5].abs() + 0.25
    for b, i in ((0, 0), (0, 3), (0, 7), (1, 0)):
        c.pools[0][int(c.table[b, i]), :, :, 5] = -torch.inf
    out, lse = run_attention(c, max_kv=max(most, 900))
    for b, i in ((0, 0), (0, 3), (0, 7), (1, 0)):
        c.table[b, i] = -1
    check_attention(c, out, lse)
    dd.check_device()


@pytest.mark.parametrize("dtype,q4", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("tokens", [1, 5, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_the_same_bits_beside_other_kernels(d, tokens, dtype, q4):
    """Attention, reading and appending beside kernels that keep the load/store units busy."""
    c = Cache([tokens] * 12, [tokens + 700 * b for b in range(12)], 16, 4, d, 64, dtype, q4)
    count, T = 4000, c.n_tokens
    seqs = c.seqs()
    ws = torch.empty(max(16, dd.paged_attn_workspace_size(c.shape, T, tokens, 8000)),
                     dtype=torch.uint8, device="cuda")
    out, lse, q_out = torch.empty_like(c.q), torch.empty(T, 16, device="cuda"), torch.empty_like(c.q)
    dense = [torch.empty(12, 4, count, d, dtype=dtype, device="cuda") for _ in range(2)]
    k, v = (c.q[:, i:i + 4].contiguous() for i in (0, 4))
    cs = torch.randn(8100, 2, d // 2, device="cuda")
    results = [out, lse, q_out, *dense, *c.pools]
    start = [p.clone() for p in c.pools]

    def calls(stream=None):
        dd.paged_append(c.shape, seqs, c.q, k, v, q_out, rope=cs, stream=stream)
        dd.paged_attn(c.shape, seqs, q_out, out, lse, ws, max_q_len=tokens, max_kv_len=8000,
                      stream=stream)
        dd.paged_read(c.shape, seqs, 17, count, *dense, stream=stream)

    calls()
    torch.cuda.synchronize()
    want = [x.view(torch.uint8).clone() for x in results]
    a = torch.randn(1 << 22, device="cuda")
    b = torch.empty_like(a)
    main, side = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    for _ in range(6):
        for p, x in zip(c.pools, start):
            p.copy_(x)
        for x in results[:5]:
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(10):
                torch.mul(a, 2.0, out=b)
        calls(main)
        with torch.cuda.stream(side):
            for _ in range(10):
                torch.mul(a, 2.0, out=b)
        torch.cuda.synchronize()
        for got, x in zip(results, want):
            assert torch.equal(got.view(torch.uint8), x)
    dd.check_device()


@pytest.mark.parametrize("tokens", [1, 40])
def test_the_widest_window_takes_no_more_workspace(tokens):
    """The size asked for without a window serves any, at the largest values of everything."""
    c = Cache([tokens, 1], [500, 77])
    most = 2 ** 31 - 1
    check_attention(c, *run_attention(c, most, most, max_kv=most), most, most)
    check_attention(c, *run_attention(c, 2 ** 30, 2 ** 30, max_kv=most), 2 ** 30, 2 ** 30)
