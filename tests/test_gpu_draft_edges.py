"""kvq_tree_attn where single elements matter: every output element is held against the sum of
p |v| of its own column, for values, scales and scores that lie far apart."""
import math

import numpy as np
import pytest
import torch

import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import TreeWorkspace
from _draft import FORMATS, TENSOR_SCALES, logical, make_cfg, make_layer, mask_tensor, random_masks, values

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def append(cfg, layer, k, v):
    kvq.kvq_append(cfg, layer, k.cuda(), v.cuda(), i32([0] * cfg.batch), 0, k.shape[1])


def run_tree(cfg, layer, q, lens, masks, num_ctas=0, out_dtype=F32, ws=None):
    out = torch.full(q.shape, 5.0, dtype=out_dtype, device="cuda")
    ws = ws or TreeWorkspace(cfg, q.shape[1], num_ctas)
    kvq.kvq_tree_attn(cfg, layer, q, i32(lens), max(lens), None if masks is None else mask_tensor(masks), out, ws,
                      num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert kvq.kvq_workspace_status(ws) == 0
    return out


def row_scales(scales, cfg, which):
    """The largest scale of every row (1 for 16-bit rows), and whether a row has several."""
    bits, grp = (cfg.k_bits, cfg.k_group) if which == 0 else (cfg.v_bits, cfg.v_group)
    if bits == 16:
        return 1.0, False
    if cfg.kv_format == kvq.KVQ_FMT_TENSOR:
        return float(TENSOR_SCALES[which]), False
    s = np.ascontiguousarray(scales).view(np.float16).astype(np.float64)
    if cfg.kv_format == kvq.KVQ_FMT_ASYM:
        s = s[..., 0::2]
    return s.max(-1), (grp or cfg.head_dim) != cfg.head_dim


def check(cfg, layer, q, lens, masks, out):
    """Every element against fp64.  The bound, from the arithmetic, with A = sum p |v| of the element:
      * P = p * (value scale) is an f16 number: 2^-11 of each term; below f16's normal numbers 2^-25
        of a P whose largest is at least 2^6 (twice where P was scaled after the maximum moved): 2^-30
        of the largest p * scale, times the sum of |code|;
      * scores: dh/8 fp32 product steps and 8 more roundings of 2^-23 of sum |q||k|, twice (p and its
        sum); z = score + log2(scale) - m: three roundings of 2^-24 of numbers up to 3 sum |q||k| + 64,
        the logarithm 2^-22 of at most 24; fp32 queries as two f16 parts: 2^-21 of sum |q||k|;
      * exp2, the inverse scale and the last division 2^-21 each; fp32 sums over n tokens (n/8 product
        steps of 2^-23, n roundings of 2^-24);
      * a row of several groups: x = code * scale / 2^e in two f16 parts, off by at most 2^-25 of 2^e
        times 2^-6;
      * the output's own half step."""
    lo = logical(layer, cfg)
    k, v = values(lo[0], lo[1], cfg, 0), values(lo[2], lo[3], cfg, 1)
    s_all, grouped = row_scales(lo[3], cfg, 1)
    s_all = np.broadcast_to(s_all, v.shape[:-1])
    dh, G, T = cfg.head_dim, cfg.n_q_heads // cfg.n_kv_heads, q.shape[1]
    tau, qq, got = 1 / math.sqrt(dh), q.double().cpu().numpy(), out.double().cpu().numpy()
    eps = torch.finfo(out.dtype).eps
    worst = 0.0
    for b, L in enumerate(lens):
        total = min(L + T, cfg.capacity)
        for i in range(T):
            m = int(masks[b, i]) if masks is not None else (2 << i) - 1
            at = list(range(L)) + [L + j for j in range(total - L) if m >> j & 1]
            for h in range(cfg.n_q_heads):
                kk, vv, s = k[b, h // G, at], v[b, h // G, at], s_all[b, h // G, at]
                z = kk @ qq[b, i, h] * tau
                p = np.exp(z - z.max())
                p /= p.sum()
                want, A = p @ vv, p @ np.abs(vv)
                qk = (np.abs(kk) @ np.abs(qq[b, i, h])).max() * tau
                score = qk * ((dh / 8 + 8) * 2.0 ** -23 + (2.0 ** -21 if q.dtype == F32 else 0.0))
                zr = math.log(2) * ((3 * qk + 64) * 3 * 2.0 ** -24 + 24 * 2.0 ** -22)
                n = len(at)
                rel = 2.0 ** -11 + 2 * math.expm1(score + zr) + 3 * 2.0 ** -21 + (n / 8 + 8) * 2.0 ** -23 + n * 2.0 ** -24
                codes = np.abs(vv) / np.where(s == 0, 1.0, np.abs(s))[:, None]
                small = 2.0 ** -30 * (2 if grouped else 1) * (p * np.abs(s)).max() * codes.sum(0)
                bound = rel * A + small + (2.0 ** -31 * (p @ s) if grouped else 0.0) + eps / 2 * np.abs(want) + 2.0 ** -149
                if out.dtype == F16:
                    bound = bound + 2.0 ** -25
                err = np.abs(got[b, i, h] - want)
                assert np.all(err <= bound), (b, i, h, float((err / bound).max()))
                worst = max(worst, float((err / bound).max()))
    return worst


# ----------------------------------------------------------------------------- one column at a time

@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("size,dtype,out_dtype", [(1.0, F16, F32), (0.01, BF16, F32), (1.0, F32, F16)])
def test_each_element_on_flat_scores(cuda_device, fmt, size, dtype, out_dtype):
    """A softmax that spreads over all tokens: outputs far smaller than the values."""
    B, T, G, hkv, cap, lens = 2, 5, 3, 1, 640, [600, 129]
    gen = torch.Generator().manual_seed(31)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, 64 if size == 1.0 else 128)
    layer = make_layer(cfg, gen)
    k, v = (torch.randn(B, cap, hkv, cfg.head_dim, generator=gen) for _ in range(2))
    append(cfg, layer, k * 0.5, v * size)
    q = torch.randn(B, T, hkv * G, cfg.head_dim, generator=gen).to(dtype).cuda()
    masks = random_masks(np.random.default_rng(31), B, T)
    check(cfg, layer, q, lens, masks, run_tree(cfg, layer, q, lens, masks, out_dtype=out_dtype))


# ----------------------------------------------------------------------------- value rows of zeros

def sink(cfg, gen, size, log2_ratio, L, T, zero_at):
    """A cache whose token(s) `zero_at` take nearly all of the probability and have zero values; the
    others' probabilities lie about 2^-log2_ratio below, their values about `size`."""
    B, dh, hkv, cap = cfg.batch, cfg.head_dim, cfg.n_kv_heads, cfg.capacity
    u = torch.randn(dh, generator=gen).sign()
    k, v = (torch.randn(B, cap, hkv, dh, generator=gen) for _ in range(2))
    k -= (k @ u)[..., None] / dh * u                                        # others: across u
    k[:, zero_at] = u * (log2_ratio * math.log(2) / math.sqrt(dh))
    v *= size
    v[:, zero_at] = 0.0
    q = (u + 0.3 * torch.randn(B, T, cfg.n_q_heads, dh, generator=gen)).half().cuda()
    return k, v, q


@pytest.mark.parametrize("fmt,dh,size,ratio,T,G", [
    ("k8v8", 128, 0.1, 13, 8, 4), ("k8v8", 128, 0.01, 20, 40, 4), ("k8v8", 64, 1e-3, 25, 1, 1), ("k16v4g64", 64, 0.01, 20, 8, 4),
    ("k4v4", 128, 0.01, 20, 5, 3), ("e4m3", 128, 0.01, 20, 8, 4), ("asym", 128, 0.01, 20, 8, 8), ("asym", 64, 1e-3, 12, 3, 2),
    ("k8v4g32", 128, 1e-4, 30, 8, 4), ("e4m3g32", 64, 1e-4, 26, 7, 2)])
def test_zero_values_that_take_the_probability(cuda_device, fmt, dh, size, ratio, T, G):
    B, hkv, cap, L = 1, 1, 768, 700
    gen = torch.Generator().manual_seed(32)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, dh)
    layer = make_layer(cfg, gen)
    k, v, q = sink(cfg, gen, size, ratio, L, T, [5, 300, 301])
    append(cfg, layer, k, v)
    masks = random_masks(np.random.default_rng(32), B, T)
    for ctas in (0, 1, 3):
        check(cfg, layer, q, [L], masks, run_tree(cfg, layer, q, [L], masks, num_ctas=ctas))


@pytest.mark.parametrize("fmt", ["k8v8", "k4v4", "e4m3", "asym", "k8v4g32"])
def test_codes_under_a_zero_scale(cuda_device, fmt):
    """value = code * scale: what the codes of a row of scale zero hold does not matter among others;
    alone such rows give at most 2^-64 of a code (a group's codes exactly nothing)."""
    B, T, G, hkv, cap, L = 1, 6, 4, 1, 512, 450
    gen = torch.Generator().manual_seed(33)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, 128)
    layer = make_layer(cfg, gen)
    zero_at = [0, 7, 129, 130, 449, 452]
    k, v, q = sink(cfg, gen, 0.1, 4, L, T, zero_at)
    append(cfg, layer, k, v)
    masks = random_masks(np.random.default_rng(33), B, T)
    clean = run_tree(cfg, layer, q, [L], masks)
    row = 128 * cfg.v_bits // 8
    rows = layer.v_codes.view(-1)[: cap * row].view(cap, row)
    rows[zero_at] = 0x33                               # 51, or two 3, or 1.375
    assert torch.equal(run_tree(cfg, layer, q, [L], masks), clean)
    rows[:] = 0x33
    layer.v_scales.zero_()
    assert torch.all(run_tree(cfg, layer, q, [L], masks).abs() <= (0 if fmt == "k8v4g32" else 51.5 * 2.0 ** -64))
    layer.v_codes.zero_()
    assert torch.all(run_tree(cfg, layer, q, [L], masks) == 0)


def test_a_tensor_scale_of_zero(cuda_device):
    B, T, G, hkv, cap, L = 1, 6, 4, 1, 512, 450
    gen = torch.Generator().manual_seed(34)
    cfg = make_cfg("tensor", B, cap, hkv * G, hkv, 128)
    layer = make_layer(cfg, gen)
    k, v = (torch.randn(B, cap, hkv, 128, generator=gen) for _ in range(2))
    append(cfg, layer, k, v)
    layer.v_scales[0] = 0.0
    q = torch.randn(B, T, hkv * G, 128, generator=gen).half().cuda()
    for ctas in (1, 3):
        assert torch.all(run_tree(cfg, layer, q, [L], None, num_ctas=ctas) == 0)


# ----------------------------------------------------------------------------- a maximum that jumps

def test_a_tile_far_below_a_later_maximum_still_counts(cuda_device):
    """The tile after the one that raises the maximum by more than 2^24: its tokens are 2^-17.6 of the
    largest each, and the only ones with a value in most columns."""
    B, T, G, hkv, dh, cap, L = 1, 64, 2, 1, 64, 512, 384
    gen = torch.Generator().manual_seed(35)
    cfg = make_cfg("k8v8", B, cap, hkv * G, hkv, dh)
    layer = make_layer(cfg, gen)
    log2_score = torch.zeros(cap)
    log2_score[:128] = 6.0
    log2_score[128 + 40] = 31.5
    log2_score[256:384] = 13.9
    k, v = torch.zeros(B, cap, hkv, dh), torch.zeros(B, cap, hkv, dh)
    k[0, :, 0, 0] = log2_score
    v[0, :, 0, 0] = 1.0
    v[0, 256:384, 0] = torch.rand(128, dh, generator=gen) + 0.01
    v[0, 256:384, 0, 0] = 1.0
    append(cfg, layer, k, v)
    q = torch.zeros(B, T, hkv * G, dh)
    q[..., 0] = math.log(2) * math.sqrt(dh)
    q = q.half().cuda()
    for ctas in (1, 2):
        out = run_tree(cfg, layer, q, [L], None, num_ctas=ctas)
        check(cfg, layer, q, [L], None, out)


# ----------------------------------------------------------------------------- whatever the timing

@pytest.mark.parametrize("T,G,num_ctas", [(64, 2, 4), (12, 4, 4), (5, 3, 7), (64, 8, 0)])
def test_the_same_bits_whatever_the_timing(cuda_device, T, G, num_ctas):
    """Every second tile raises the maximum, by one group of softmax warps, while the other has the
    next tile in hand: a call's bits do not depend on which of them is ahead."""
    B, hkv, dh, cap, lens = 4, 2, 128, 4096, [4000, 3333, 4000, 2048]
    gen = torch.Generator().manual_seed(36)
    cfg = make_cfg("k8v8", B, cap, hkv * G, hkv, dh)
    layer = make_layer(cfg, gen)
    u = torch.randn(dh, generator=gen).sign()
    k, v = (torch.randn(B, cap, hkv, dh, generator=gen) for _ in range(2))
    tile = torch.arange(cap) // 128
    level = torch.where(tile % 2 == 1, (tile + 1) * 10.0, tile * 10.0 - 14.0)      # of the scores, log2
    k += (level * math.log(2) / math.sqrt(dh))[None, :, None, None] * u
    append(cfg, layer, k, v)
    q = (u + 0.2 * torch.randn(B, T, hkv * G, dh, generator=gen)).half().cuda()
    masks = random_masks(np.random.default_rng(36), B, T)
    ws = TreeWorkspace(cfg, T, num_ctas)
    first = run_tree(cfg, layer, q, lens, masks, num_ctas, ws=ws)
    # another stream's work moves the warps against one another
    other, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    d_len, d_mask, outs = i32(lens), mask_tensor(masks), [torch.empty_like(first) for _ in range(60)]
    torch.cuda.synchronize()
    for o in outs:
        with torch.cuda.stream(other):
            busy @ busy
        kvq.kvq_tree_attn(cfg, layer, q, d_len, 4000, d_mask, o, ws, num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    assert kvq.kvq_workspace_status(ws) == 0


# ----------------------------------------------------------------------------- groups that lie far apart

@pytest.mark.parametrize("which,fmt,dh", [
    (which, fmt, dh) for which in "kv" for fmt, dh in (
        ("k8v8g32", 128), ("k8v8g32", 64), ("k4v4g32", 64), ("e4m3g32", 128), ("asymg32", 128), ("asymg32", 64))]
    + [("k", "k4g32v8", 128), ("v", "k8v4g32", 128)])
def test_a_small_group_beside_a_large_one(cuda_device, which, fmt, dh):
    """One group's scale 2^18 times the others': their columns of the output, and scores that come from
    them alone, are as exact as any."""
    B, T, G, hkv, cap, L = 1, 9, 4, 1, 384, 333
    gen = torch.Generator().manual_seed(37)
    cfg = make_cfg(fmt, B, cap, hkv * G, hkv, dh)
    layer = make_layer(cfg, gen)
    k, v = (torch.randn(B, cap, hkv, dh, generator=gen) for _ in range(2))
    q = torch.randn(B, T, hkv * G, dh, generator=gen)
    if which == "k":
        k[..., :32] *= 2.0 ** 18
        q[..., :32] = 0.0
    else:
        v[..., :32] *= 2.0 ** 18
    append(cfg, layer, k, v)
    masks = random_masks(np.random.default_rng(37), B, T)
    q = q.half().cuda()
    check(cfg, layer, q, [L], masks, run_tree(cfg, layer, q, [L], masks))
