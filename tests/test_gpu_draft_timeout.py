"""kvq_tree_attn when a wait runs out: a producer that stops copying leaves every role of the kernel
waiting, the kernel reports KVQ_ERR_TIMEOUT and returns, and context and workspace stay usable."""
import pytest
import torch

import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import TreeWorkspace
from _draft import make_cfg, make_layer

TIMEOUT = -8


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dh,T,q_dtype,num_ctas,n_segments", [
    ("k8v8", 128, 16, torch.float16, 1, 0), ("k8v8", 128, 16, torch.float16, 1, 1), ("k4v4g32", 64, 64, torch.float32, 1, 4),
    ("e4m3", 128, 33, torch.bfloat16, 3, 0), ("k16v16", 128, 5, torch.float16, 3, 1), ("k8v8", 64, 16, torch.float16, 0, 0)])
def test_tree_kernel_waits_run_out_and_report_timeout(cuda_device, fmt, dh, T, q_dtype, num_ctas, n_segments):
    B, hkv, G, cap, lens = 3, 2, 4, 512, [300, 440, 1]     # six segments or more, sixteen tiles or more
    gen = torch.Generator().manual_seed(51)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, dh)
    layer = make_layer(cfg, gen)
    k, v = (torch.randn(B, cap, hkv, dh, generator=gen).cuda() for _ in range(2))
    kvq.kvq_append(cfg, layer, k, v, i32([0] * B), 0, cap)
    q = torch.randn(B, T, hkv * G, dh, generator=gen).to(q_dtype).cuda()
    d_len, ws = i32(lens), TreeWorkspace(cfg, T, num_ctas)
    want, got = (torch.zeros(q.shape, device="cuda") for _ in range(2))
    kvq.kvq_tree_attn(cfg, layer, q, d_len, max(lens), None, want, ws, num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert kvq.kvq_workspace_status(ws) == 0
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    kvq.kvq_selftest_tree_timeout(cfg, layer, q, d_len, max(lens), torch.empty_like(got), ws, n_segments, 20_000_000,
                                  num_ctas=num_ctas)
    b.record()
    torch.cuda.synchronize()
    assert 18.0 <= a.elapsed_time(b) < 1000.0, a.elapsed_time(b)
    print("gave up after %.1f ms" % a.elapsed_time(b))
    assert kvq.kvq_workspace_status(ws) == TIMEOUT
    assert kvq.kvq_workspace_status(ws) == 0                 # read clears it
    kvq.kvq_tree_attn(cfg, layer, q, d_len, max(lens), None, got, ws, num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert kvq.kvq_workspace_status(ws) == 0
    assert torch.equal(got, want)
