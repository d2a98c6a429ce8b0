"""kvq_rope_append, kvq_rope_table and kvq_tree_commit at the edges of what their arguments may hold."""
import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import LayerCache, RopeConfig
from _draft import FORMATS, logical, make_cfg, make_layer, rotated
from _helpers import to_np32
from test_gpu_draft_rope import expect_append

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- numbers that are none

@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype,rot,layout", [(torch.float32, 64, kvq.KVQ_ROPE_HALF), (torch.float16, 64, kvq.KVQ_ROPE_INTERLEAVED),
                                              (torch.bfloat16, 24, kvq.KVQ_ROPE_HALF)])
def test_nan_and_infinities_are_stored_as_kvq_append_stores_them(cuda_device, fmt, dtype, rot, layout):
    B, n, hkv, dh, cap = 2, 9, 2, 64, 32
    gen = torch.Generator().manual_seed(41)
    cfg = make_cfg(fmt, B, cap, hkv, hkv, dh)
    a, b = make_layer(cfg, gen), make_layer(cfg, gen)
    k, v = (torch.randn(B, n, hkv, dh, generator=gen) * 2 for _ in range(2))
    inf, nan = float("inf"), float("nan")
    for x in (k, v):
        x[0, 0, 0, 5] = nan
        x[0, 1, :, 3], x[0, 1, 1, 40] = inf, nan
        x[0, 2, 0, 60] = -inf
        x[0, 3] = nan                                   # a row of nothing else
        x[0, 4, 0, :32] = nan                           # a group of nothing else
        x[0, 5, 1, 32:40], x[0, 5, 1, 7] = nan, -inf
        x[0, 6, 0] = 0.0
        x[0, 6, 0, 63] = nan                            # zeros beside it
        x[1, 0, :, ::2] = nan
    k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
    r = RopeConfig(rot, layout, base=500.0)
    table = kvq.kvq_rope_table(r, cap)
    pos = [0, 17]
    kvq.kvq_rope_append(cfg, a, r, table, None, k, v, None, i32(pos), max(pos))
    t = table.cpu().numpy()
    with np.errstate(invalid="ignore"):
        turned = np.stack([np.stack([rotated(to_np32(k[s, j]), t[pos[s] + j], rot, layout) for j in range(n)]) for s in range(B)])
    kvq.kvq_append(cfg, b, torch.from_numpy(turned).cuda(), v.float(), i32(pos), max(pos), n)
    for got, want, name in zip(logical(a, cfg), logical(b, cfg), ("k codes", "k scales", "v codes", "v scales")):
        assert (got is None) == (want is None)
        assert got is None or np.array_equal(got, want), (name, np.argwhere(got != want)[:8].tolist())


# ----------------------------------------------------------------------------- ring

@pytest.mark.parametrize("n", [30, 56])
def test_a_skipped_token_overwrites_nothing_in_the_ring(cuda_device, n):
    """A token whose rope position is outside the table is skipped: the earlier token of the call that
    shares its slot stays."""
    gen = torch.Generator().manual_seed(42)
    B, window, anchor = 3, 24, 8
    cfg = make_cfg("k8v4g32", B, 32, 2, 1, 128, window=window, n_anchor=anchor)
    layer = make_layer(cfg, gen)
    r = RopeConfig(64)
    table = kvq.kvq_rope_table(r, 200)
    k, v = (torch.randn(B, n, 1, 128, generator=gen).half().cuda() for _ in range(2))
    pos = [4, 77, 0]
    rope_pos = [[p + j for j in range(n)] for p in pos]
    for j in (24, 27, 28, n - 1):
        rope_pos[0][j] = 200
    for j in range(26, n, 3):
        rope_pos[1][j] = -1
    for j in range(24, n):
        rope_pos[2][j] = 2**31 - 1
    count = [n, n, n - 2]
    before = logical(layer, cfg)
    kvq.kvq_rope_append(cfg, layer, r, table, None, k, v, None, i32(pos), 100, d_count=i32(count), d_rope_pos=i32(rope_pos))
    torch.cuda.synchronize()
    _, want = expect_append(cfg, before, None, k, v, table.cpu().numpy(), 64, kvq.KVQ_ROPE_HALF, pos, count, rope_pos)
    for g, w in zip(logical(layer, cfg), want):
        assert np.array_equal(g, w)


# ----------------------------------------------------------------------------- table

@pytest.mark.parametrize("orig_len,low,high", [(4, 1.0, 32.0), (1, 1.0, 2.0), (2048, 1000.0, 2000.0)])
def test_yarn_where_every_pair_turns_less_than_low(cuda_device, orig_len, low, high):
    r = RopeConfig(64, scaling=kvq.KVQ_ROPE_YARN, factor=8.0, orig_len=orig_len, low=low, high=high, gain=1.0)
    assert orig_len / (2 * math.pi) < low                     # pair 0 turns the most
    angle = np.arange(40, dtype=np.float64)[:, None] * (10000.0 ** (-2 * np.arange(32) / 64) / 8)
    want = np.stack([np.cos(angle), np.sin(angle)], -1)
    got = kvq.kvq_rope_table(r, 40).cpu().numpy()
    # half an fp32 step, and the roundings of the angle in 64 bits
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + (angle[..., None] + 1) * 2.0 ** -50)


# ----------------------------------------------------------------------------- commit

@pytest.mark.parametrize("fmt,dh", [("k8v8", 128), ("k4v4g32", 64), ("tensor", 128)])
def test_commit_in_layers_that_share_a_page_pool(cuda_device, fmt, dh):
    """One pool of pages for all layers, a block table each."""
    B, hkv, cap, T, n_layers = 2, 2, 256, 9, 3
    gen = torch.Generator().manual_seed(43)
    cfg = make_cfg(fmt, B, cap, hkv, hkv, dh, n_pages=2 * B * n_layers + 1)
    pool = make_layer(cfg, gen)
    for x in (pool.k_codes, pool.v_codes):
        x.random_(0, 256)
    if fmt != "tensor":
        pool.k_scales.uniform_(0, 1)
        pool.v_scales.uniform_(0, 1)
    pages = torch.randperm(cfg.n_pages, generator=gen)[: 2 * B * n_layers].view(n_layers, B, 2).to(torch.int32).cuda()
    layers = [LayerCache.from_buffers(cfg, pool.k_codes, pool.k_scales, pool.v_codes, pool.v_scales, block_table=pages[i])
              for i in range(n_layers)]
    before = [logical(x, cfg) for x in layers]
    lens, path = [120, 200], [1, 4, 8]
    new = i32([0, 0])
    kvq.kvq_tree_commit(cfg, layers, i32(lens), 200, i32([path] * B), i32([3, 2]), T, d_len_out=new)
    assert new.tolist() == [123, 202]
    for layer, was in zip(layers, before):
        for g, w in zip(logical(layer, cfg), was):
            if w is None:
                continue
            want = w.copy()
            for b, m in enumerate((3, 2)):
                for i in range(m):
                    want[b, :, lens[b] + i] = w[b, :, lens[b] + path[i]]
            assert np.array_equal(g, want)
