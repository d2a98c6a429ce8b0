"""kvq_tree_attn against a plain fp64 implementation, at the sizes, formats, masks and lengths
where it can go wrong.  The bound of every comparison is derived in _draft.tree_bound."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import TreeWorkspace
from _draft import (logical, make_cfg, make_layer, mask_tensor, random_masks, tree_bound, tree_reference, values)

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(cfg, gen, spread=1.0):
    layer = make_layer(cfg, gen)
    B, cap, hkv, dh = cfg.batch, cfg.capacity, cfg.n_kv_heads, cfg.head_dim
    k, v = (torch.randn(B, cap, hkv, dh, generator=gen) * spread for _ in range(2))
    kvq.kvq_append(cfg, layer, k.cuda(), v.cuda(), i32([0] * B), 0, cap)
    return layer


def run_tree(cfg, layer, q, lens, n_tree, masks, out_dtype, max_len=None, num_ctas=0, scale=0.0, ws=None):
    T = q.shape[1]
    out = torch.full(q.shape, 5.0, dtype=out_dtype, device="cuda")
    ws = ws or TreeWorkspace(cfg, T, num_ctas)
    kvq.kvq_tree_attn(cfg, layer, q, i32(lens), max(lens) if max_len is None else max_len,
                      None if masks is None else mask_tensor(masks), out, ws,
                      d_n_tree=None if n_tree is None else i32(n_tree), softmax_scale=scale, num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert kvq.kvq_workspace_status(ws) == 0
    return out


def check(cfg, layer, q, lens, n_tree, masks, out, scale=0.0):
    lo = logical(layer, cfg)
    k, v = values(lo[0], lo[1], cfg, 0), values(lo[2], lo[3], cfg, 1)
    T = q.shape[1]
    n = [T] * len(lens) if n_tree is None else [max(0, min(x, T)) for x in n_tree]
    want, vmax, qk = tree_reference(q.double().cpu().numpy(), k, v, lens, n, masks, cfg.capacity, scale)
    got = out.double().cpu().numpy()
    tokens = max(min(max(a, 0) + T, cfg.capacity) for a in lens)
    for b in range(len(lens)):
        assert np.all(got[b, n[b]:] == 5.0), "rows behind a sequence's tree were written"
    live = ~np.isnan(want)
    bound = tree_bound(np.where(live, want, 0), vmax, qk, tokens, cfg.head_dim, out.dtype, q.dtype == F32)
    err = np.abs(got - want)
    assert np.all(np.isfinite(got))
    assert np.all(err[live] <= np.broadcast_to(bound, err.shape)[live]), \
        float((err / bound)[live].max())
    return float((err / bound)[live].max()) if live.any() else 0.0


CASES = [  # format, dh, G, hkv, T, lengths, q dtype, out dtype, paged
    ("k8v8", 128, 4, 2, 16, [300, 1], F16, F16, False),
    ("k8v8", 128, 8, 1, 64, [500], BF16, BF16, False),
    ("k8v8", 64, 1, 3, 6, [250, 0, 127], F16, F32, False),
    ("k8v8", 128, 1, 1, 1, [128, 127, 129, 0], F32, F32, False),
    ("k8v8g32", 128, 2, 2, 33, [400, 95], F16, F32, True),
    ("k8v4g32", 128, 3, 2, 24, [401, 30], F16, F16, False),
    ("k4g32v8", 128, 3, 1, 9, [600, 255], BF16, F32, True),
    ("k4v4", 128, 4, 2, 8, [383, 120], BF16, BF16, True),
    ("k4v4", 64, 5, 1, 13, [100, 259], F16, F16, False),
    ("k4v4g32", 64, 4, 2, 64, [129, 64], F32, F32, False),
    ("k4v4g32", 128, 8, 1, 17, [700], F16, F32, False),
    ("k16v16", 128, 4, 1, 32, [310, 2], F16, F32, False),
    ("k16v16", 64, 8, 1, 64, [111], BF16, F32, True),
    ("k16v4g64", 128, 2, 1, 5, [140, 384], F16, F16, False),
    ("k4v16", 64, 2, 2, 7, [97], F16, F32, False),
    ("e4m3", 128, 4, 1, 12, [222, 640], F16, F32, False),
    ("e4m3g32", 64, 3, 1, 40, [333], BF16, F32, True),
    ("asym", 128, 6, 1, 20, [200, 511], F16, F32, False),
    ("asymg32", 128, 2, 2, 64, [260], F32, F16, False),
    ("tensor", 128, 4, 1, 11, [250, 77], F16, F32, False),
]


@pytest.mark.parametrize("fmt,dh,G,hkv,T,lens,q_dtype,out_dtype,paged", CASES)
def test_tree_attention_matches_64_bits(cuda_device, fmt, dh, G, hkv, T, lens, q_dtype, out_dtype, paged):
    B, cap = len(lens), -(-(max(lens) + T) // 128) * 128
    gen = torch.Generator().manual_seed(T * 100 + G)
    rng = np.random.default_rng(T * 100 + G)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, dh, n_pages=B * cap // 128 + 2 if paged else 0)
    layer = filled(cfg, gen)
    q = torch.randn(B, T, hkv * G, dh, generator=gen).to(q_dtype).cuda()
    masks = random_masks(rng, B, T)
    out = run_tree(cfg, layer, q, lens, None, masks, out_dtype)
    check(cfg, layer, q, lens, None, masks, out)


@pytest.mark.parametrize("num_ctas", [0, 1, 2, 7, 300])
def test_ragged_trees_and_lengths(cuda_device, num_ctas):
    """Tree sizes 0 .. T, lengths 0, 1, at and around tile borders, a length beyond the capacity
    (clamped), drafted tokens that the capacity cuts off; any number of CTAs."""
    lens = [0, 1, 127, 128, 129, 505, 512, 700, 300, 0]
    n_tree = [9, 0, 4, 9, 1, 9, 9, 9, 12, 0]
    B, T, G, hkv, cap = len(lens), 9, 4, 2, 512
    gen = torch.Generator().manual_seed(8)
    cfg = make_cfg("k8v8", B, cap, hkv * G, hkv, 128)
    layer = filled(cfg, gen)
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    masks = random_masks(np.random.default_rng(8), B, T)
    out = run_tree(cfg, layer, q, lens, n_tree, masks, F32, max_len=cap - T, num_ctas=num_ctas)
    check(cfg, layer, q, lens, n_tree, masks, out)


@pytest.mark.parametrize("fmt,dh,G,T,num_ctas,q_dtype", [
    ("k8v8", 128, 1, 1, 4, F16), ("k8v8", 64, 3, 3, 5, BF16), ("k4v4g32", 128, 5, 7, 3, F16), ("k16v16", 128, 3, 23, 4, F32),
    ("k8v8g32", 128, 1, 33, 2, BF16), ("asym", 64, 8, 9, 3, F32), ("tensor", 128, 5, 13, 1, F16), ("e4m3", 128, 2, 64, 6, F32)])
def test_segments_of_many_tiles_shared_by_ctas(cuda_device, fmt, dh, G, T, num_ctas, q_dtype):
    """Row tiles of several token tiles, some whole, some cut between CTAs (first and last partial of
    a CTA among them); odd numbers of rows; scores that grow along the sequence, so that the running
    maximum moves more than once."""
    B, hkv, lens, cap = 3, 2, [700, 850, 333], 1024
    gen = torch.Generator().manual_seed(13)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, dh)
    layer = make_layer(cfg, gen)
    k, v = (torch.randn(B, cap, hkv, dh, generator=gen) for _ in range(2))
    k *= torch.linspace(0.1, 8.0, cap)[None, :, None, None]
    kvq.kvq_append(cfg, layer, k.cuda(), v.cuda(), i32([0] * B), 0, cap)
    q = torch.randn(B, T, hkv * G, dh, generator=gen).to(q_dtype).cuda()
    n_tree = [T, max(T - 1, 1), T]
    masks = random_masks(np.random.default_rng(13), B, T)
    out = run_tree(cfg, layer, q, lens, n_tree, masks, F32, num_ctas=num_ctas)
    check(cfg, layer, q, lens, n_tree, masks, out)


def test_masks_causal_empty_dense_and_stray_bits(cuda_device):
    B, T, G, hkv, cap = 3, 64, 2, 1, 256
    lens = [0, 130, 64]
    gen = torch.Generator().manual_seed(9)
    cfg = make_cfg("k4v4", B, cap, hkv * G, hkv, 128)
    layer = filled(cfg, gen)
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    out = run_tree(cfg, layer, q, lens, None, None, F32)                     # causal
    check(cfg, layer, q, lens, None, None, out)
    causal = np.array([[(2 << i) - 1 for i in range(T)]] * B, dtype=object)
    causal = np.array([[np.uint64(x & (2**64 - 1)) for x in row] for row in causal], np.uint64)
    assert torch.equal(out, run_tree(cfg, layer, q, lens, None, causal, F32))
    masks = random_masks(np.random.default_rng(1), B, T)
    masks[:, ::3] = 0                                                       # rows that see the prefix only
    masks[:, 1::3] = np.uint64(2**64 - 1)                                   # rows that see every drafted token
    out = run_tree(cfg, layer, q, lens, [64, 10, 33], masks, F32)
    check(cfg, layer, q, lens, [64, 10, 33], masks, out)
    assert torch.all(out[0, ::3] == 0), "a row that attends nothing gets zeros"


@pytest.mark.parametrize("fmt", ["k16v16", "k8v8", "e4m3"])
def test_garbage_in_places_that_no_row_attends(cuda_device, fmt):
    """NaN, infinities and NaN scales behind the tree and in masked drafted tokens reach no row."""
    B, T, G, hkv, cap, L = 1, 8, 4, 1, 256, 100
    gen = torch.Generator().manual_seed(10)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, 128)
    layer = filled(cfg, gen)
    masks = random_masks(np.random.default_rng(5), B, T, forest=0.6)
    bad = T - 2                                        # only row `bad` attends drafted token `bad`
    keep = np.uint64(2**64 - 1) ^ np.uint64(1 << bad)
    masks[0, [i for i in range(T) if i != bad]] &= keep
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    clean = run_tree(cfg, layer, q, [L], None, masks, F32)
    for codes, scales in ((layer.k_codes, layer.k_scales), (layer.v_codes, layer.v_scales)):
        row = 256 if fmt == "k16v16" else 128
        rows = codes.view(-1)[: cap * row].view(cap, row)
        for at in [L + bad] + list(range(L + T, cap)):
            if fmt == "k16v16":
                rows[at].view(F16)[:] = float("nan") if at % 2 else float("inf")
            else:
                rows[at] = 0x7F                        # e4m3: NaN codes
                scales[at] = float("nan")
    out = run_tree(cfg, layer, q, [L], None, masks, F32)
    others = [i for i in range(T) if i != bad]
    assert torch.equal(out[:, others], clean[:, others])


@pytest.mark.parametrize("scale,spread", [(3.0, 4.0), (1e-4, 1.0), (0.0, 1e-3), (0.0, 3000.0), (-0.2, 1.0)])
def test_extreme_scores_and_value_scales(cuda_device, scale, spread):
    """One-hot and flat softmax, tiny and huge values, a negative softmax scale."""
    B, T, G, hkv, cap, L = 1, 10, 4, 1, 512, 490
    gen = torch.Generator().manual_seed(11)
    cfg = make_cfg("k8v8", B, cap, hkv * G, hkv, 128)
    layer = filled(cfg, gen, spread)
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    masks = random_masks(np.random.default_rng(6), B, T)
    out = run_tree(cfg, layer, q, [L], None, masks, F32, scale=scale)
    check(cfg, layer, q, [L], None, masks, out, scale)


@pytest.mark.parametrize("q_dtype,size", [(BF16, 1e30), (BF16, 1e-30), (F32, 1e20), (F32, 1e-6), (F16, 6e4)])
def test_queries_of_any_magnitude(cuda_device, q_dtype, size):
    """Rows of very large and very small queries (the softmax scale brings them back), a zero row."""
    B, T, G, hkv, cap, L = 1, 5, 2, 1, 256, 200
    gen = torch.Generator().manual_seed(12)
    cfg = make_cfg("k8v8", B, cap, hkv * G, hkv, 64)
    layer = filled(cfg, gen)
    q = (torch.randn(B, T, hkv * G, 64, generator=gen).clamp(-1, 1) * size).to(q_dtype).cuda()
    q[0, 2] = 0
    masks = random_masks(np.random.default_rng(7), B, T)
    out = run_tree(cfg, layer, q, [L], None, masks, F32, scale=0.3 / size)
    check(cfg, layer, q, [L], None, masks, out, 0.3 / size)


def test_values_of_very_different_scales(cuda_device):
    """Tokens whose value scales differ by 2^20: each row's error stays relative to the largest."""
    B, T, G, hkv, cap, L = 1, 12, 4, 1, 384, 350
    gen = torch.Generator().manual_seed(13)
    cfg = make_cfg("k8v4g32", B, cap, hkv * G, hkv, 128)
    layer = make_layer(cfg, gen)
    k, v = (torch.randn(B, cap, hkv, 128, generator=gen) for _ in range(2))
    v *= torch.exp2(torch.randint(-14, 7, (B, cap, 1, 1), generator=gen).float())
    v[0, 5] = 0
    v[0, 6, :, :32] = 0                               # one zero group
    kvq.kvq_append(cfg, layer, k.cuda(), v.cuda(), i32([0]), 0, cap)
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    masks = random_masks(np.random.default_rng(7), B, T)
    out = run_tree(cfg, layer, q, [L], None, masks, F32)
    check(cfg, layer, q, [L], None, masks, out)


def test_offsets_beyond_32_bits(cuda_device):
    """A cache of more than 2^31 bytes a tensor: the last sequence is read where it lies."""
    B, hkv, cap, T, L = 66, 8, 16384, 4, 16300
    cfg = make_cfg("k16v16", B, cap, hkv, hkv, 128)
    assert B * hkv * cap * 256 > 2**31
    gen = torch.Generator().manual_seed(14)
    layer = make_layer(cfg, gen)
    one = make_cfg("k16v16", 1, cap, hkv, hkv, 128)
    small = filled(one, gen)
    n = hkv * cap * 256
    for a, b in ((layer.k_codes, small.k_codes), (layer.v_codes, small.v_codes)):
        a[(B - 1) * n: B * n] = b[:n]
    q = torch.randn(1, T, hkv, 128, generator=gen).half().cuda()
    ref = run_tree(one, small, q, [L], None, None, F32)
    out = run_tree(cfg, layer, q.expand(B, -1, -1, -1).contiguous(), [3] * (B - 1) + [L], None, None, F32)
    bound = 4 * 2.0 ** -11 * float(small.v_codes[:n].view(F16).abs().max())   # two splits, each as in tree_bound
    assert (out[-1] - ref[0]).abs().max() <= bound
    assert torch.all(out[0] == 0)


def test_stream_graphs_and_repeats(cuda_device):
    """On a side stream and in two captured graphs that share a workspace: the same bits."""
    B, T, G, hkv, cap = 3, 16, 4, 2, 1024
    lens = [900, 17, 512]
    gen = torch.Generator().manual_seed(15)
    cfg = make_cfg("k8v8", B, cap, hkv * G, hkv, 128)
    layer = filled(cfg, gen)
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    masks = random_masks(np.random.default_rng(3), B, T)
    ws = TreeWorkspace(cfg, T)
    want = run_tree(cfg, layer, q, lens, None, masks, F16, ws=ws)
    for _ in range(3):
        assert torch.equal(want, run_tree(cfg, layer, q, lens, None, masks, F16, ws=ws))
    d_len, d_mask = i32(lens), mask_tensor(masks)
    outs, graphs = [torch.zeros_like(want) for _ in range(2)], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kvq.kvq_tree_attn(cfg, layer, q, d_len, 1000, d_mask, outs[0], ws)
        for o in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                kvq.kvq_tree_attn(cfg, layer, q, d_len, 1000, d_mask, o, ws)
            graphs.append(g)
    side.synchronize()
    assert torch.equal(outs[0], want)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # the lengths are read on the device at each replay
    d_len.copy_(i32([5, 1000, 0]))
    graphs[0].replay()
    torch.cuda.synchronize()
    check(cfg, layer, q, [5, 1000, 0], None, masks, outs[0])


def test_two_streams_with_a_workspace_each(cuda_device):
    B, T, G, hkv, cap = 4, 13, 4, 2, 1024
    gen = torch.Generator().manual_seed(16)
    cfg = make_cfg("k8v4g32", B, cap, hkv * G, hkv, 128)
    layers = [filled(cfg, gen) for _ in range(2)]
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    d_len = i32([1000, 3, 640, 511])
    want = [run_tree(cfg, x, q, [1000, 3, 640, 511], None, None, F16) for x in layers]
    outs, wss = [torch.zeros_like(q) for _ in layers], [TreeWorkspace(cfg, T) for _ in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, o, ws, st in zip(layers, outs, wss, streams):
            kvq.kvq_tree_attn(cfg, x, q, d_len, 1000, None, o, ws, stream=st)
    torch.cuda.synchronize()
    for o, w, ws in zip(outs, want, wss):
        assert torch.equal(o, w) and kvq.kvq_workspace_status(ws) == 0


@pytest.mark.parametrize("paged", [False, True])
def test_a_captured_step_equals_the_eager_one(cuda_device, paged):
    """Rotation and append, tree attention, commit and reading back in one graph, replayed on other
    inputs in the same buffers."""
    B, T, G, hkv, dh, cap = 3, 11, 3, 2, 128, 384
    gen = torch.Generator().manual_seed(17)
    cfg = make_cfg("k8v8", B, cap, hkv * G, hkv, dh, n_pages=B * cap // 128 + 2 if paged else 0)
    rope = kvq.RopeConfig(dh)
    table = kvq.kvq_rope_table(rope, cap)
    layers = [make_layer(cfg, gen) for _ in range(2)]
    for x in layers[1:]:                                        # both start with the same cache
        for name in ("k_codes", "k_scales", "v_codes", "v_scales", "block_table"):
            if getattr(x, name) is not None:
                getattr(x, name).copy_(getattr(layers[0], name))

    def buffers():
        return dict(qkv=torch.zeros(B, T, hkv * (G + 2), dh, dtype=F16, device="cuda"), d_len=i32([0] * B), n=i32([0] * B),
                    path=i32([[0, 2, 5]] * B), m=i32([0] * B), q=torch.zeros(B, T, hkv * G, dh, dtype=F16, device="cuda"),
                    out=torch.zeros(B, T, hkv * G, dh, dtype=F16, device="cuda"), new=i32([0] * B),
                    k=torch.zeros(B, 3, hkv, dh, device="cuda"), ws=TreeWorkspace(cfg, T))

    def step(layer, s):
        q, k, v = s["qkv"].split([hkv * G, hkv, hkv], dim=2)
        kvq.kvq_rope_append(cfg, layer, rope, table, q, k, v, s["q"], s["d_len"], cap - T, d_count=s["n"])
        kvq.kvq_tree_attn(cfg, layer, s["q"], s["d_len"], cap - T, None, s["out"], s["ws"], d_n_tree=s["n"])
        kvq.kvq_tree_commit(cfg, [layer], s["d_len"], cap - T, s["path"], s["m"], T, d_len_out=s["new"])
        kvq.kvq_read(cfg, layer, s["k"], None, s["d_len"], cap - T, d_count=s["m"])

    a, b = buffers(), buffers()
    step(layers[1], b)                                          # no tokens: loads the kernels, changes nothing
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        step(layers[1], b)
    for lens, n, m in (([0, 130, 1], [11, 7, 0], [3, 2, 0]), ([3, 132, 1], [11, 11, 9], [0, 3, 1])):
        qkv = torch.randn(B, T, hkv * (G + 2), dh, generator=gen).half()
        for s in (a, b):
            s["qkv"].copy_(qkv)
            for name, x in (("d_len", lens), ("n", n), ("m", m)):
                s[name].copy_(i32(x))
        step(layers[0], a)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for name in ("q", "out", "new", "k"):
            assert torch.equal(a[name], b[name]), name
        assert a["new"].tolist() == [x + y for x, y in zip(lens, m)]
        for x, y in zip(logical(layers[0], cfg), logical(layers[1], cfg)):
            assert np.array_equal(x, y)


def test_guard_bytes_around_out_and_workspace(cuda_device):
    B, T, G, hkv, cap = 2, 23, 3, 2, 640
    gen = torch.Generator().manual_seed(16)
    cfg = make_cfg("k4v4g32", B, cap, hkv * G, hkv, 128)
    layer = filled(cfg, gen)
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    ws = TreeWorkspace(cfg, T)
    n = ws.nbytes // 4
    big = torch.full((n + 2048,), 3.25, device="cuda")
    big[1024: 1024 + n] = 0
    ws.buf = big[1024: 1024 + n]
    out = torch.full((q.numel() + 2048,), 7.0, dtype=F16, device="cuda")
    view = out[1024: 1024 + q.numel()].view(q.shape)
    masks = random_masks(np.random.default_rng(2), B, T)
    kvq.kvq_tree_attn(cfg, layer, q, i32([600, 333]), 610, mask_tensor(masks), view, ws)
    torch.cuda.synchronize()
    assert torch.all(big[:1024] == 3.25) and torch.all(big[1024 + n:] == 3.25)
    assert torch.all(out[:1024] == 7) and torch.all(out[1024 + q.numel():] == 7)


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("fmt,paged", [("k8v8", False), ("k4g32v8", True)])
def test_a_speculative_step_as_a_program_runs_it(cuda_device, fmt, paged):
    """Prompt, drafted tree, verification, commit, the next single-token step: the cache after
    the commit holds what appending the accepted tokens one by one would have put there, and the
    tree's rows equal the single-token decode of each accepted token."""
    B, T, G, hkv, dh, cap = 2, 12, 4, 2, 128, 384
    lens = [200, 119]
    gen = torch.Generator().manual_seed(17)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, dh, n_pages=9 if paged else 0)
    layer, ref = make_layer(cfg, gen), make_layer(cfg, gen)
    rope = kvq.RopeConfig(dh, base=1e4)
    table = kvq.kvq_rope_table(rope, cap)
    P = max(lens)
    q, k, v = (torch.randn(B, P, h, dh, generator=gen).half().cuda() for h in (hkv * G, hkv, hkv))
    for x in (layer, ref):
        kvq.kvq_rope_append(cfg, x, rope, table, None, k, v, None, i32([0, 0]), 0, d_count=i32(lens))
    # a drafted tree: depth gives the rope position, order the slot
    parents = [-1, 0, 0, 1, 1, 2, 3, 5, 6, 6, 8, -1]
    depth = [0]
    masks = np.zeros((B, T), np.uint64)
    depths = []
    for j, p in enumerate(parents):
        depths.append(0 if p < 0 else depths[p] + 1)
        masks[:, j] = (1 << j) | (0 if p < 0 else int(masks[0, p]))
    path = [0, 1, 3, 6, 8]
    tq, tk, tv = (torch.randn(B, T, h, dh, generator=gen).half().cuda() for h in (hkv * G, hkv, hkv))
    q_rot = torch.empty_like(tq)
    d_len = i32(lens)
    kvq.kvq_rope_append(cfg, layer, rope, table, tq, tk, tv, q_rot, d_len, P,
                        d_rope_pos=i32([[n + d for d in depths] for n in lens]))
    out = run_tree(cfg, layer, q_rot, lens, None, masks, F32)
    check(cfg, layer, q_rot, lens, None, masks, out)
    new = torch.empty_like(d_len)
    kvq.kvq_tree_commit(cfg, [layer], d_len, P, i32([path] * B), i32([len(path), 3]), T, d_len_out=new)
    assert new.tolist() == [lens[0] + 5, lens[1] + 3]
    # the same tokens one at a time
    ws = kvq.Workspace(cfg)
    for i, node in enumerate(path):
        one_q = torch.empty(B, 1, hkv * G, dh, dtype=F16, device="cuda")
        kvq.kvq_rope_append(cfg, ref, rope, table, tq[:, node:node + 1], tk[:, node:node + 1], tv[:, node:node + 1],
                            one_q, d_len + i, P + i, d_count=i32([1, int(i < 3)]))
        single = torch.empty(B, hkv * G, dh, device="cuda")
        kvq.kvq_decode_attn(cfg, ref, one_q[:, 0], d_len + i + 1, P + i + 1, single, ws)
        assert torch.equal(one_q[0, 0], q_rot[0, node])
        # 2e-3 max |v| is the decode kernel's bound, 2^-10 the tree's own (both P roundings)
        assert (out[0, node] - single[0]).abs().max() <= (2e-3 + 2.0 ** -10) * 4.5
    got, want = logical(layer, cfg), logical(ref, cfg)
    for b in range(B):
        n = int(new[b])
        for g, w in zip(got, want):
            assert g is None or np.array_equal(g[b, :, :n], w[b, :, :n])
