"""References of the drafted-token operators in plain numpy (fp64 where values are computed,
single-rounded fp32 where codes have to match bit for bit)."""
import math
from dataclasses import replace

import numpy as np
import torch

import oracle
import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import Config, LayerCache
from _helpers import obits, to_np32

PAGE = 128

# name -> (k_bits, v_bits, k_group, v_group, format)
FORMATS = {
    "k8v8": (8, 8, 0, 0, kvq.KVQ_FMT_INT),
    "k8v8g32": (8, 8, 32, 32, kvq.KVQ_FMT_INT),
    "k8v4g32": (8, 4, 0, 32, kvq.KVQ_FMT_INT),
    "k4g32v8": (4, 8, 32, 0, kvq.KVQ_FMT_INT),
    "k4v4": (4, 4, 0, 0, kvq.KVQ_FMT_INT),
    "k4v4g32": (4, 4, 32, 32, kvq.KVQ_FMT_INT),
    "k16v16": (16, 16, 0, 0, kvq.KVQ_FMT_INT),
    "k16v4g64": (16, 4, 0, 64, kvq.KVQ_FMT_INT),
    "k4v16": (4, 16, 0, 0, kvq.KVQ_FMT_INT),
    "e4m3": (8, 8, 0, 0, kvq.KVQ_FMT_E4M3),
    "e4m3g32": (8, 8, 32, 32, kvq.KVQ_FMT_E4M3),
    "asym": (8, 8, 0, 0, kvq.KVQ_FMT_ASYM),
    "asymg32": (8, 8, 32, 32, kvq.KVQ_FMT_ASYM),
    "tensor": (8, 8, 0, 0, kvq.KVQ_FMT_TENSOR),
}
TENSOR_SCALES = (np.float16(0.031), np.float16(0.027))


def make_cfg(fmt, batch, cap, hq, hkv, dh, n_pages=0, **more):
    kb, vb, kg, vg, f = FORMATS[fmt]
    paged = dict(page_tokens=PAGE, n_pages=n_pages) if n_pages else {}
    return Config(batch=batch, capacity=cap, n_q_heads=hq, n_kv_heads=hkv, head_dim=dh, k_bits=kb,
                  v_bits=vb, k_group=min(kg, dh) if kg else 0, v_group=min(vg, dh) if vg else 0,
                  kv_format=f, **paged, **more)


def make_layer(cfg, gen, zero=True):
    """A zeroed layer (a paged one behind a shuffled table) with the tensor scales set."""
    table = None
    if cfg.page_tokens:
        per = cfg.capacity // PAGE
        table = torch.randperm(cfg.n_pages, generator=gen)[: cfg.batch * per].view(cfg.batch, per)
        table = table.to(torch.int32).cuda()
    layer = LayerCache(cfg, zero=zero, block_table=table)
    if cfg.kv_format == kvq.KVQ_FMT_TENSOR:
        layer.k_scales[0], layer.v_scales[0] = float(TENSOR_SCALES[0]), float(TENSOR_SCALES[1])
    return layer


def plain_cfg(cfg):
    return replace(cfg, page_tokens=0, n_pages=0)


def logical(layer, cfg):
    """The layer's rows as [codes, scales] of K, then of V: bytes / fp16 bits [B][H][cap][...]."""
    B, H, cap, dh = cfg.batch, cfg.n_kv_heads, cfg.capacity, cfg.head_dim
    pair = 2 if cfg.kv_format == kvq.KVQ_FMT_ASYM else 1
    res = []
    for codes, scales, bits, grp in ((layer.k_codes, layer.k_scales, cfg.k_bits, cfg.k_group or dh),
                                     (layer.v_codes, layer.v_scales, cfg.v_bits, cfg.v_group or dh)):
        n = 0 if bits == 16 or cfg.kv_format == kvq.KVQ_FMT_TENSOR else dh // grp * pair
        for buf, width, dt in ((codes, dh * bits // 8, np.uint8), (scales, n, np.uint16)):
            if not width:
                res.append(None)
                continue
            a = buf.cpu().numpy().reshape(-1).view(dt)
            if cfg.page_tokens:
                a = a[: cfg.n_pages * H * PAGE * width].reshape(cfg.n_pages, H, PAGE, width)
                a = a[layer.block_table.cpu().numpy()]                 # [B][pages][H][128][..]
                a = a.transpose(0, 2, 1, 3, 4).reshape(B, H, cap, width)
            else:
                a = a[: B * H * cap * width].reshape(B, H, cap, width)
            res.append(a)
    return res


def values(codes, scales, cfg, which):
    """fp64 values of rows [..., row bytes] by the formats' definition."""
    bits, grp = (cfg.k_bits, cfg.k_group) if which == 0 else (cfg.v_bits, cfg.v_group)
    dh = cfg.head_dim if cfg.mode == kvq.KVQ_MODE_KV else cfg.d_model
    grp = grp or dh
    codes = np.ascontiguousarray(codes)
    if bits == 16:
        return codes.view(np.float16).astype(np.float64)
    if bits == 4:
        lo, hi = (codes & 15).astype(np.int64), (codes >> 4).astype(np.int64)
        c = np.stack([lo, hi], -1).reshape(*codes.shape[:-1], dh)
        c = np.where(c > 7, c - 16, c).astype(np.float64)
    elif cfg.kv_format == kvq.KVQ_FMT_E4M3:
        c = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    elif cfg.kv_format == kvq.KVQ_FMT_ASYM:
        c = codes.astype(np.float64)
    else:
        c = codes.view(np.int8).astype(np.float64)
    if cfg.kv_format == kvq.KVQ_FMT_TENSOR:
        return c * float(TENSOR_SCALES[which])
    s = np.ascontiguousarray(scales).view(np.float16).astype(np.float64)
    if cfg.kv_format == kvq.KVQ_FMT_ASYM:
        return (c - np.repeat(s[..., 1::2], grp, -1)) * np.repeat(s[..., 0::2], grp, -1)
    return c * np.repeat(s, grp, -1)


def quantised(x, cfg, which):
    """(codes, scales) of fp32 rows by the CPU oracle's quantiser."""
    bits, grp = (cfg.k_bits, cfg.k_group) if which == 0 else (cfg.v_bits, cfg.v_group)
    x = np.ascontiguousarray(x, dtype=np.float32)
    if bits == 16:
        return x.astype(np.float16).view(np.uint8).reshape(*x.shape[:-1], -1), None
    if cfg.kv_format == kvq.KVQ_FMT_TENSOR:
        return oracle.quantize_rows_tensor(x, int(TENSOR_SCALES[which].view(np.uint16))), None
    c, s = oracle.quantize_rows(x, grp or cfg.head_dim, obits(cfg, bits))
    return c, s.reshape(*x.shape[:-1], -1)


def rotated(x, table, rot, layout):
    """x [..., dh] fp32, table [..., rot/2, 2] fp32: every product and sum rounded once."""
    x = np.array(x, dtype=np.float32)
    c, s = table[..., 0], table[..., 1]
    if layout == kvq.KVQ_ROPE_HALF:
        a, b = x[..., : rot // 2].copy(), x[..., rot // 2: rot].copy()
        x[..., : rot // 2], x[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2].copy(), x[..., 1:rot:2].copy()
        x[..., 0:rot:2], x[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return x


def random_masks(rng, batch, n, forest=0.15):
    """Ancestor masks of random trees (each drafted token attends itself and its ancestors)."""
    out = np.zeros((batch, n), np.uint64)
    for b in range(batch):
        for j in range(n):
            m = 1 << j
            if j and rng.random() > forest:
                m |= int(out[b, rng.integers(max(0, j - 4), j)])
            out[b, j] = m
    return out


def mask_tensor(masks):
    return torch.from_numpy(masks.view(np.int64).copy()).cuda()


def tree_reference(q, k, v, lens, n_tree, masks, cap, scale=0.0):
    """fp64 outputs and, per row, the largest |v| and sum |q||k| among what it attends.
    q [B][T][Hq][dh], k, v [B][Hkv][cap][dh] fp64; rows >= n_tree[b] are nan."""
    B, T, Hq, dh = q.shape
    G = Hq // k.shape[1]
    tau = scale or 1 / math.sqrt(dh)
    out = np.full(q.shape, np.nan)
    vmax = np.zeros((B, T, Hq))
    qk = np.zeros((B, T, Hq))
    for b in range(B):
        L = min(max(lens[b], 0), cap)
        total = min(L + n_tree[b], cap)
        for i in range(n_tree[b]):
            m = int(masks[b, i]) if masks is not None else (2 << i) - 1
            at = list(range(L)) + [L + j for j in range(total - L) if m >> j & 1]
            for h in range(Hq):
                if not at:
                    out[b, i, h] = 0.0
                    continue
                kk, vv = k[b, h // G, at], v[b, h // G, at]
                s = kk @ q[b, i, h] * tau
                p = np.exp(s - s.max())
                out[b, i, h] = (p / p.sum()) @ vv
                vmax[b, i, h] = np.abs(vv).max()
                qk[b, i, h] = (np.abs(kk) @ np.abs(q[b, i, h])).max() * tau
    return out, vmax, qk


def tree_bound(want, vmax, qk, n_tokens, dh, out_dtype, q_f32=False):
    """How far an output element may be from fp64, from the arithmetic:
    P rounded to fp16: 2^-11 sum p|v|; scores: every fp32 step may truncate (2^-23 of
    sum |q||k|, dh/8 MMA steps and 8 more operations), twice as a relative error of p and of
    its sum; exp2 2^-21; P.V accumulated over n/16 MMA steps; the output's own half step.
    fp32 queries enter as two fp16 parts: 2^-21 of sum |q||k| more."""
    score = qk * ((dh / 8 + 8) * 2.0 ** -23 + (2.0 ** -21 if q_f32 else 0.0))
    rel = 2.0 ** -11 + 2 * np.expm1(score) + 2 * 2.0 ** -21 + (n_tokens / 16 + 8) * 2.0 ** -23
    return (rel * vmax)[..., None] + torch.finfo(out_dtype).eps / 2 * np.abs(want) + 2.0 ** -24
