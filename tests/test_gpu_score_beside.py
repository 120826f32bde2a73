"""The scoring step beside other kernels: its logits, and with them the selection and
every later step, are the same bits whatever else runs on the GPU meanwhile.

The keys stream through a ring in shared memory.  A stage must not be refilled before
the loads from it have been served, however long another kernel on the same
multiprocessor keeps them queued: a stage refilled too early gives the logits of four
stages later."""
import pytest
import torch

import sparse_kv_prefetch_gb300 as dd
import synth
from gpu_util import Outputs, Slot, dd_shape, run_layer

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# heads, KV heads, d, dtype: the per-lane form of each row width, and the tensor-core form
FORMS = [(32, 32, 128, BF), (32, 32, 64, BF), (16, 16, 256, BF), (32, 32, 64, F32),
         (16, 16, 128, F32), (16, 4, 128, F32), (32, 8, 128, BF), (32, 8, 64, BF)]


@pytest.mark.parametrize("heads,kv_heads,d,dtype", FORMS)
def test_logits_beside_elementwise_kernels(heads, kv_heads, d, dtype):
    B, n, k, W = 4, 65536, 512, 64
    shape = dd.Shape(B, heads, kv_heads, d, n, k, W, dd.DD_BF16 if dtype == BF else dd.DD_F32)
    g = torch.Generator("cuda").manual_seed(heads + d)
    q = torch.randn(B, heads, d, device="cuda", generator=g).to(dtype)
    K = torch.randn(B, kv_heads, n, d, device="cuda", generator=g, dtype=BF).to(dtype)
    U = B * kv_heads
    idx = torch.empty(U, k, dtype=torch.int32, device="cuda")
    sel = torch.empty(U, k, device="cuda")
    lse = torch.empty(B, heads, device="cuda")
    ws = torch.empty(dd.workspace_size(shape), dtype=torch.uint8, device="cuda")
    logits = ws[:B * heads * n * 4].view(torch.int32)  # the workspace starts with them
    dd.score_topk(shape, q, K, idx, sel, lse, ws)
    torch.cuda.synchronize()
    want, want_idx = logits.clone(), idx.clone()
    a = torch.randn(1 << 22, device="cuda", generator=g)
    b = torch.empty_like(a)
    main, side = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    for _ in range(6):
        ws.fill_(255)
        idx.fill_(-1)
        torch.cuda.synchronize()
        dd.score_topk(shape, q, K, idx, sel, lse, ws, stream=main)
        with torch.cuda.stream(side):
            for _ in range(20):
                torch.mul(a, 2.0, out=b)
        torch.cuda.synchronize()
        bad = int((logits != want).sum())
        assert bad == 0, f"{bad} logits differ"
        assert torch.equal(idx, want_idx)
    dd.check_device()


@pytest.mark.parametrize("fused", [False, True])
def test_pipeline_layers_beside_the_attention_of_the_last(fused):
    """In the pipeline schedule the attention of a layer runs beside the scoring of the
    next: eight layers over one layer slot, bit for bit the standalone calls."""
    w = synth.C4.scaled(batch=4)
    s = Slot(w, 0)
    o = Outputs(w)
    run_layer(w, s, o)
    torch.cuda.synchronize()
    kv = dd.host_empty(s.K_h.shape[:3] + (2,) + s.K_h.shape[3:], s.K_h.dtype, kind="pinned")
    kv[:, :, :, 0, :] = s.K_h
    kv[:, :, :, 1, :] = s.V_h
    ctx = dd.Ctx(dd_shape(w))
    main, side = torch.cuda.Stream(), torch.cuda.Stream(priority=-1)
    for _ in range(4):
        outs = [torch.full_like(o.out, float("nan")) for _ in range(8)]
        main.wait_stream(torch.cuda.current_stream())
        ctx.decode_step([dd.LayerIO(s.q_spec, s.q, s.K, None, None, s.v_win, x, kv_host=kv)
                         for x in outs], compute=main, copy=side, pipeline=True, fused_topk=fused)
        torch.cuda.synchronize()
        for l, x in enumerate(outs):
            assert torch.equal(x, o.out), f"layer {l}"
    dd.check_device()
    ctx.close()
