"""kvq_rope_table, kvq_rope_append, kvq_read and kvq_tree_commit against plain references:
codes, scales, rotated queries, values read back and moved rows have to match bit for bit."""
import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import LayerCache, RopeConfig
from _draft import (FORMATS, logical, make_cfg, make_layer, plain_cfg, quantised, rotated, values)
from _helpers import to_np32

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- table

def frequencies(r: RopeConfig):
    i = np.arange(r.rot_dim // 2, dtype=np.float64)
    base, gain = r.base, 1.0
    if r.scaling == kvq.KVQ_ROPE_NTK:
        base *= r.factor ** (r.rot_dim / (r.rot_dim - 2))
    f = base ** (-2 * i / r.rot_dim)
    if r.scaling == kvq.KVQ_ROPE_LINEAR:
        f = f / r.factor
    if r.scaling == kvq.KVQ_ROPE_YARN:
        pair = lambda turns: r.rot_dim * math.log(r.orig_len / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), r.rot_dim - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        f = f / r.factor * ramp + f * (1 - ramp)
        gain = 0.1 * math.log(r.factor) + 1
    if r.scaling == kvq.KVQ_ROPE_BANDS:
        keep = np.clip((r.orig_len * f / (2 * math.pi) - 1) / 3, 0, 1)
        f = f / r.factor * (1 - keep) + f * keep
    return f, gain


@pytest.mark.parametrize("rot,first,scaling", [
    (128, 0, kvq.KVQ_ROPE_PLAIN), (64, 5, kvq.KVQ_ROPE_LINEAR), (24, 0, kvq.KVQ_ROPE_NTK),
    (128, 120_000, kvq.KVQ_ROPE_YARN), (64, 1_000_000, kvq.KVQ_ROPE_BANDS),
    (8, 2**31 - 1 - 37, kvq.KVQ_ROPE_PLAIN)])
def test_table_is_the_rounded_64_bit_value(cuda_device, rot, first, scaling):
    r = RopeConfig(rot, scaling=scaling, factor=8.0, orig_len=8192)
    n = 37
    got = kvq.kvq_rope_table(r, n, first).cpu().numpy().astype(np.float64)
    f, gain = frequencies(r)
    angle = np.arange(first, first + n, dtype=np.float64)[:, None] * f
    want = np.stack([np.cos(angle), np.sin(angle)], -1) * gain
    # half an fp32 step, and two pow / product roundings of the angle in 64 bits
    bound = 2.0 ** -24 * np.abs(want) + gain * (angle[..., None] * 2.0 ** -50 + 2.0 ** -50)
    assert np.all(np.abs(got - want) <= bound)


def test_table_position_zero_and_no_positions(cuda_device):
    t = kvq.kvq_rope_table(RopeConfig(16), 1)
    assert torch.equal(t[..., 0].cpu(), torch.ones(1, 8)) and torch.equal(t[..., 1].cpu(), torch.zeros(1, 8))
    assert kvq.kvq_rope_table(RopeConfig(16), 0).shape == (0, 8, 2)


# ----------------------------------------------------------------------------- append

def expect_append(cfg, layer0, q, k, v, table, rot, layout, pos, count, rope_pos):
    """(rotated queries, logical cache) after the call, from the cache before it."""
    B, n = k.shape[:2]
    want = [None if a is None else a.copy() for a in layer0]
    qo = None if q is None else to_np32(q)
    kk, vv = to_np32(k), to_np32(v)
    for b in range(B):
        for j in range(min(count[b], n)):
            at = rope_pos[b][j] if rope_pos is not None else pos[b] + j
            if not 0 <= at < len(table):
                continue
            if q is not None:
                qo[b, j] = rotated(qo[b, j], table[at], rot, layout)
            p = pos[b] + j
            if p < 0:
                continue
            slot = p if not cfg.window or p < cfg.n_anchor else cfg.n_anchor + (p - cfg.n_anchor) % cfg.window
            if slot >= cfg.capacity:
                continue
            for w, x in ((0, rotated(kk[b, j], table[at], rot, layout)), (1, vv[b, j])):
                c, s = quantised(x, cfg, w)
                want[2 * w][b, :, slot] = c
                if want[2 * w + 1] is not None:
                    want[2 * w + 1][b, :, slot] = s
    return (None if q is None else torch.from_numpy(qo).to(q.dtype)), want


CASES = [  # format, dh, hq, hkv, rot, layout, dtype, paged
    ("k8v8", 128, 8, 2, 128, kvq.KVQ_ROPE_HALF, torch.float16, False),
    ("k8v8g32", 128, 6, 3, 64, kvq.KVQ_ROPE_INTERLEAVED, torch.bfloat16, True),
    ("k8v4g32", 64, 5, 5, 64, kvq.KVQ_ROPE_HALF, torch.float32, False),
    ("k4g32v8", 128, 3, 1, 24, kvq.KVQ_ROPE_HALF, torch.float16, True),
    ("k4v4", 64, 3, 1, 8, kvq.KVQ_ROPE_INTERLEAVED, torch.float16, False),
    ("k4v4g32", 64, 4, 2, 40, kvq.KVQ_ROPE_HALF, torch.bfloat16, False),
    ("k16v16", 128, 2, 2, 120, kvq.KVQ_ROPE_INTERLEAVED, torch.float32, True),
    ("e4m3", 128, 8, 1, 128, kvq.KVQ_ROPE_INTERLEAVED, torch.float16, False),
    ("asym", 64, 2, 1, 64, kvq.KVQ_ROPE_HALF, torch.bfloat16, True),
    ("asymg32", 128, 4, 4, 32, kvq.KVQ_ROPE_HALF, torch.float16, False),
    ("tensor", 128, 2, 2, 128, kvq.KVQ_ROPE_HALF, torch.float16, False),
]


@pytest.mark.parametrize("fmt,dh,hq,hkv,rot,layout,dtype,paged", CASES)
@pytest.mark.parametrize("n,fused", [(1, True), (13, False)])
def test_rope_append_matches_bit_for_bit(cuda_device, fmt, dh, hq, hkv, rot, layout, dtype, paged, n, fused):
    pos = [0, 126, 243, -1 if n == 1 else 250]
    B, cap = len(pos), 256
    gen = torch.Generator().manual_seed(n + rot)
    cfg = make_cfg(fmt, B, cap, hq, hkv, dh, n_pages=2 * B + 3 if paged else 0)
    layer = make_layer(cfg, gen)
    r = RopeConfig(rot, layout, base=500.0)
    # the last sequence's positions run out of the table (and of the cache)
    table = kvq.kvq_rope_table(r, 260)
    if fused:
        # parts of one projection's output, with room between the sequences' tokens
        qkv = torch.randn(B, n + 2, hq + 2 * hkv, dh, generator=gen).to(dtype).cuda()[:, 1: n + 1]
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        count, rope_pos = [1, 1, 1, 1], None
    else:
        q, k, v = (torch.randn(B, n, h, dh, generator=gen).to(dtype).cuda() for h in (hq, hkv, hkv))
        k[1, 2] = 0.0                                    # an all-zero row
        count = [n, 0, 5, n + 9]
        rope_pos = [[(p + j * 7) % 270 for j in range(n)] for p in (3, 0, 240, 255)]
    before = logical(layer, cfg)
    q_out = torch.full((B, n, hq, dh), 7.0, dtype=dtype, device="cuda")
    kvq.kvq_rope_append(cfg, layer, r, table, q, k, v, q_out, i32(pos), cap - n,
                        d_count=None if fused else i32(count), d_rope_pos=None if fused else i32(rope_pos))
    torch.cuda.synchronize()
    want_q, want = expect_append(cfg, before, q, k, v, table.cpu().numpy(), rot, layout, pos, count, rope_pos)
    got = logical(layer, cfg)
    for i, name in enumerate(("k codes", "k scales", "v codes", "v scales")):
        assert (got[i] is None) == (want[i] is None)
        assert got[i] is None or np.array_equal(got[i], want[i]), name
    for b in range(B):
        for j in range(n):
            at = rope_pos[b][j] if rope_pos else pos[b] + j
            done = j < min(count[b], n) and 0 <= at < 260
            ref = want_q[b, j] if done else torch.full_like(want_q[b, j], 7.0)
            assert torch.equal(q_out[b, j].cpu(), ref), (b, j)


def test_rope_append_in_place_keys_only_and_repeat(cuda_device):
    """q_out may be q itself; q may be left out; the same call twice gives the same cache."""
    gen = torch.Generator().manual_seed(2)
    cfg = make_cfg("k8v8", 2, 64, 4, 2, 128)
    r = RopeConfig(128)
    table = kvq.kvq_rope_table(r, 64)
    q, k, v = (torch.randn(2, 3, h, 128, generator=gen).half().cuda() for h in (4, 2, 2))
    a, b = make_layer(cfg, gen), make_layer(cfg, gen)
    out, same = torch.empty_like(q), q.clone()
    kvq.kvq_rope_append(cfg, a, r, table, q, k, v, out, i32([0, 9]), 9)
    kvq.kvq_rope_append(cfg, a, r, table, q, k, v, out, i32([0, 9]), 9)
    kvq.kvq_rope_append(cfg, b, r, table, same, k, v, same, i32([0, 9]), 9)
    assert torch.equal(out, same)
    c = make_layer(cfg, gen)
    kvq.kvq_rope_append(cfg, c, r, table, None, k, v, None, i32([0, 9]), 9)
    for x in (b, c):
        for m in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(a, m), getattr(x, m))
    kvq.kvq_rope_append(cfg, c, r, table, q[:, :0], k[:, :0], v[:, :0], out[:, :0], i32([0, 9]), 9)   # no tokens


@pytest.mark.parametrize("dh,hq,rot,layout,dtype", [
    (128, 5, 24, kvq.KVQ_ROPE_HALF, torch.float16), (128, 9, 96, kvq.KVQ_ROPE_HALF, torch.float32),
    (64, 17, 8, kvq.KVQ_ROPE_HALF, torch.bfloat16), (64, 3, 40, kvq.KVQ_ROPE_INTERLEAVED, torch.float32),
    (128, 6, 128, kvq.KVQ_ROPE_HALF, torch.bfloat16)])
def test_rope_append_in_place_equals_apart(cuda_device, dh, hq, rot, layout, dtype):
    gen = torch.Generator().manual_seed(rot)
    cfg = make_cfg("k8v8", 3, 256, hq, 1, dh)
    r = RopeConfig(rot, layout=layout)
    table = kvq.kvq_rope_table(r, 300)
    q, k, v = (torch.randn(3, 70, h, dh, generator=gen).to(dtype).cuda() for h in (hq, 1, 1))
    a, b, out, same = make_layer(cfg, gen), make_layer(cfg, gen), torch.empty_like(q), q.clone()
    kvq.kvq_rope_append(cfg, a, r, table, q, k, v, out, i32([0, 100, 9]), 100)
    kvq.kvq_rope_append(cfg, b, r, table, same, k, v, same, i32([0, 100, 9]), 100)
    assert torch.equal(out, same) and not torch.equal(out, q)


@pytest.mark.parametrize("n", [5, 40])
def test_rope_append_sliding_window(cuda_device, n):
    """Ring slots, with more tokens than the ring holds in one call (n = 40 > 24)."""
    gen = torch.Generator().manual_seed(n)
    cfg = make_cfg("k4g32v8", 2, 32, 3, 1, 128, window=24, n_anchor=8)
    layer = make_layer(cfg, gen)
    r = RopeConfig(64)
    table = kvq.kvq_rope_table(r, 200)
    k, v = (torch.randn(2, n, 1, 128, generator=gen).half().cuda() for _ in range(2))
    pos = [4, 77]
    before = logical(layer, cfg)
    kvq.kvq_rope_append(cfg, layer, r, table, None, k, v, None, i32(pos), 100)
    _, want = expect_append(cfg, before, None, k, v, table.cpu().numpy(), 64, kvq.KVQ_ROPE_HALF, pos, [n, n], None)
    for g, w in zip(logical(layer, cfg), want):
        assert np.array_equal(g, w)
    # the newest tokens are read back by their positions
    got = torch.zeros(2, 5, 1, 128, device="cuda")
    kvq.kvq_read(cfg, layer, got, None, i32([4 + n - 5, 77 + n - 5]), 200)
    for b, p in enumerate(pos):
        for j in range(5):
            x = rotated(to_np32(k[b, n - 5 + j]), table.cpu().numpy()[p + n - 5 + j], 64, kvq.KVQ_ROPE_HALF)
            c, s = quantised(x, cfg, 0)
            assert np.array_equal(got[b, j].cpu().numpy(), values(c, s, cfg, 0).astype(np.float32))


# ----------------------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dh,dtype,paged,n", [(128, torch.float16, False, 67), (64, torch.bfloat16, True, 130),
                                              (128, torch.float32, True, 1)])
def test_read_matches_bit_for_bit(cuda_device, fmt, dh, dtype, paged, n):
    pos, B, hkv, cap = [0, 126, 60, 125], 4, 3, 256
    count = [n, n - 1, 0, n + 3]
    gen = torch.Generator().manual_seed(dh + n)
    cfg = make_cfg(fmt, B, cap, hkv, hkv, dh, n_pages=11 if paged else 0)
    layer = make_layer(cfg, gen)
    k, v = (torch.randn(B, cap, hkv, dh, generator=gen) * 3 for _ in range(2))
    kvq.kvq_append(cfg, layer, k.cuda(), v.cuda(), i32([0] * B), 0, cap)
    lo = logical(layer, cfg)
    ref = [values(lo[0], lo[1], cfg, 0), values(lo[2], lo[3], cfg, 1)]
    # outputs inside larger tensors
    k_out = torch.full((B, n + 1, 2 * hkv, dh), 9.0, dtype=dtype, device="cuda")
    v_out = torch.full((B, n, hkv, dh), 9.0, dtype=dtype, device="cuda")
    kvq.kvq_read(cfg, layer, k_out[:, 1:, hkv:], v_out, i32(pos), max(pos), d_count=i32(count))
    assert torch.all(k_out[:, 0] == 9) and torch.all(k_out[:, :, :hkv] == 9)
    for got, want in ((k_out[:, 1:, hkv:], ref[0]), (v_out, ref[1])):
        for b in range(B):
            m = max(0, min(count[b], n, cap - pos[b]))
            rows = torch.from_numpy(want[b, :, pos[b]: pos[b] + m]).transpose(0, 1)
            # exact in fp32 (at most 9 + 11 significant bits), then rounded once
            assert torch.equal(got[b, :m].cpu(), rows.float().to(dtype))
            assert torch.all(got[b, m:] == 9)


def test_read_one_side_and_hidden_states(cuda_device):
    gen = torch.Generator().manual_seed(4)
    cfg = make_cfg("k8v4g32", 2, 64, 2, 2, 128)
    layer = make_layer(cfg, gen)
    x = torch.randn(2, 64, 2, 128, generator=gen).cuda()
    kvq.kvq_append(cfg, layer, x, x, i32([0, 0]), 0, 64)
    full = [torch.empty(2, 64, 2, 128, device="cuda") for _ in range(2)]
    kvq.kvq_read(cfg, layer, *full, i32([0, 0]), 0)
    for i in range(2):
        one = torch.empty(2, 7, 2, 128, device="cuda")
        kvq.kvq_read(cfg, layer, *((one, None) if i == 0 else (None, one)), i32([3, 50]), 50)
        assert torch.equal(one[0], full[i][0, 3:10]) and torch.equal(one[1], full[i][1, 50:57])
    for bits, d in ((4, 384), (8, 2048), (16, 128)):
        cfg = kvq.Config(batch=2, capacity=48, mode=kvq.KVQ_MODE_H, d_model=d, h_bits=bits, h_groups=d // 32,
                         n_q_heads=d // 128, n_kv_heads=d // 128, head_dim=128)
        layer = LayerCache(cfg, zero=True)
        h = torch.randn(2, 48, d, generator=gen).half()
        kvq.kvq_append(cfg, layer, h.cuda(), None, i32([0, 0]), 0, 48)
        got = torch.empty(2, 40, d, device="cuda")
        kvq.kvq_read(cfg, layer, got, None, i32([8, 1]), 8)
        codes = layer.k_codes.cpu().numpy()[: 2 * 48 * d * bits // 8].reshape(2, 48, -1)
        if bits == 16:
            want = codes.copy().view(np.float16).astype(np.float32)
        else:
            ref = make_cfg("k4v4g32" if bits == 4 else "k8v8g32", 2, 48, 1, 1, 128)
            ref.mode, ref.d_model, ref.k_bits, ref.k_group = kvq.KVQ_MODE_H, d, bits, 32
            s = layer.k_scales.cpu().numpy().view(np.uint16)[: 2 * 48 * d // 32].reshape(2, 48, -1)
            want = values(codes, s, ref, 0).astype(np.float32)
        assert np.array_equal(got[0].cpu().numpy(), want[0, 8:]) and np.array_equal(got[1].cpu().numpy(), want[1, 1:41])


# ----------------------------------------------------------------------------- commit

@pytest.mark.parametrize("fmt,dh,paged,n_layers", [
    ("k8v8", 128, False, 1), ("k4v4g32", 64, True, 3), ("k16v16", 128, True, 2), ("asymg32", 128, False, 2),
    ("k4v4", 64, False, 2), ("tensor", 64, False, 1), ("k8v4g32", 128, False, 70)])
def test_commit_moves_exactly_the_path(cuda_device, fmt, dh, paged, n_layers):
    rng = np.random.default_rng(n_layers + dh)
    lens = [0, 127, 100, 190, 64, 5, 30]
    T, B, hkv, cap = 64, 7, 2, 256
    paths = [list(range(64)), sorted(rng.choice(64, 40, replace=False)), [63], [], [0, 1, 5, 5, 9],
             [2, 40, 64, 65], sorted(rng.choice(64, 33, replace=False))]
    m = [64, 40, 1, 0, 3, 2, 33]                      # valid prefixes: index 5 repeats, 64 is no token
    gen = torch.Generator().manual_seed(3)
    cfg = make_cfg(fmt, B, cap, hkv, hkv, dh, n_pages=2 * B + 1 if paged else 0)
    layers = []
    for _ in range(n_layers):
        layer = make_layer(cfg, gen)
        for name in ("k_codes", "v_codes"):
            getattr(layer, name).random_(0, 256)
        if fmt not in ("k16v16", "tensor"):
            layer.k_scales.uniform_(0, 1)
            layer.v_scales.uniform_(0, 1)
        layers.append(layer)
    before = [logical(x, cfg) for x in layers]
    d_path = i32([[int(x) for x in p] + [-1] * (T - len(p)) for p in paths])
    d_len, new = i32(lens), i32([-5] * B)
    kvq.kvq_tree_commit(cfg, layers, d_len, max(lens), d_path, i32([70, 40, 1, -2, 5, 4, 33]), T, d_len_out=new)
    assert new.tolist() == [a + b for a, b in zip(lens, m)] and d_len.tolist() == lens
    for layer, was in zip(layers, before):
        for g, w in zip(logical(layer, cfg), was):
            if w is None:
                continue
            want = w.copy()
            for b in range(B):
                for i in range(m[b]):
                    want[b, :, lens[b] + i] = w[b, :, lens[b] + paths[b][i]]
            assert np.array_equal(g, want)
