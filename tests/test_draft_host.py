"""Refusals of the drafted-token calls that need no GPU: every argument is checked on the host
before anything is launched, and the binding checks what pointers cannot show."""
import ctypes

import pytest
import torch

import quantized_kv_cache_22_b200 as kvq
from quantized_kv_cache_22_b200 import Config, KvqLayer, KvqRopeConfig, KvqRows, RopeConfig

P = ctypes.c_void_p
INVALID, UNSUPPORTED, CAPACITY, ALIGN, WORKSPACE = -1, -2, -3, -4, -5


def ref(x):
    return None if x is None else ctypes.byref(x)


def config(**over):
    base = dict(batch=2, capacity=256, n_q_heads=8, n_kv_heads=2, head_dim=128)
    return Config(**{**base, **over}).c()


LAYER = KvqLayer(16, 16, 32, 48)
H = dict(mode=kvq.KVQ_MODE_H, d_model=256, h_bits=4, h_groups=2, n_q_heads=2, n_kv_heads=2)
WINDOW = dict(window=240, n_anchor=16)


def tree(cfg=None, layer=LAYER, q=P(16), qd=0, n=8, d_len=P(64), max_len=100, d_n=None, mask=P(64), scale=0.0,
         out=P(128), od=0, ws=P(256), wsb=1 << 30, ctas=4):
    return kvq.lib().kvq_tree_attn(ref(cfg or config()), ref(layer), q, qd, n, d_len, max_len, d_n, mask,
                                   ctypes.c_float(scale), out, od, ws, ctypes.c_uint64(wsb), ctas, None)


@pytest.mark.parametrize("want,over", [
    (INVALID, dict(q=None)), (INVALID, dict(d_len=None)), (INVALID, dict(out=None)), (INVALID, dict(ws=None)),
    (INVALID, dict(layer=None)), (INVALID, dict(qd=3)), (INVALID, dict(od=-1)), (INVALID, dict(n=0)),
    (INVALID, dict(n=65)), (INVALID, dict(max_len=-1)), (INVALID, dict(ctas=-1)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(cfg=config(**H))),
    (INVALID, dict(layer=KvqLayer(16, None, 32, 48))), (INVALID, dict(cfg=config(page_tokens=128, n_pages=4))),
    (UNSUPPORTED, dict(cfg=config(**WINDOW))), (UNSUPPORTED, dict(cfg=config(n_q_heads=18))),
    (CAPACITY, dict(max_len=249)), (CAPACITY, dict(max_len=2**31 - 1)),
    (ALIGN, dict(q=P(24))), (ALIGN, dict(out=P(130))), (ALIGN, dict(ws=P(260))), (ALIGN, dict(mask=P(68))),
    (ALIGN, dict(layer=KvqLayer(16, 16, 36, 48))), (WORKSPACE, dict(wsb=16))])
def test_tree_attn_refuses(want, over):
    assert tree(**over) == want


def test_tree_workspace_bytes():
    def need(n, ctas=148, **over):
        v = ctypes.c_uint64()
        rc = kvq.lib().kvq_tree_workspace_bytes(ref(config(**over)), n, ctas, ctypes.byref(v))
        return rc or v.value
    assert need(1) >= 256 and need(64) >= need(1)
    assert need(0) == INVALID and need(65) == INVALID and need(4, -1) == INVALID
    assert need(4, **H) == INVALID and need(4, **WINDOW) == UNSUPPORTED
    # partial results of a CTA (two slots each) start on 16 bytes, whatever the number of rows
    for n in (1, 3, 5, 8):
        for group in (1, 3, 4):
            for dh in (64, 128):
                over = dict(n_q_heads=2 * group, n_kv_heads=2, head_dim=dh)
                assert (need(n, 9, **over) - need(n, 8, **over)) % 32 == 0


def rope(cfg=None, layer=LAYER, r=None, table=P(32), table_len=256, q=KvqRows(16, 0, 0), k=KvqRows(16, 0, 0),
         v=KvqRows(32, 0, 0), q_out=KvqRows(48, 0, 0), dtype=0, d_pos=P(64), max_pos=100, n=4, count=None,
         rope_pos=None):
    r = r or RopeConfig(64).c()
    return kvq.lib().kvq_rope_append(ref(cfg or config()), ref(layer), ref(r), table, table_len, ref(q), ref(k),
                                     ref(v), ref(q_out), dtype, d_pos, max_pos, n, count, rope_pos, None)


@pytest.mark.parametrize("want,over", [
    (0, dict(n=0)), (0, dict(n=0, q=None, q_out=None)), (0, dict(n=0, cfg=config(**WINDOW), max_pos=252)),
    (INVALID, dict(q=None)), (INVALID, dict(q_out=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)),
    (INVALID, dict(table=None)), (INVALID, dict(table_len=0)), (INVALID, dict(d_pos=None)), (INVALID, dict(n=-1)),
    (INVALID, dict(max_pos=-1)), (INVALID, dict(dtype=5)), (INVALID, dict(cfg=config(**H))),
    (INVALID, dict(k=KvqRows(16, -8, 0))), (INVALID, dict(v=KvqRows(None, 0, 0))),
    (INVALID, dict(r=RopeConfig(64, layout=2).c())),
    (UNSUPPORTED, dict(r=RopeConfig(12).c())), (UNSUPPORTED, dict(r=RopeConfig(0).c())),
    (UNSUPPORTED, dict(r=RopeConfig(136).c())), (UNSUPPORTED, dict(r=RopeConfig(128).c(), cfg=config(head_dim=64))),
    (CAPACITY, dict(max_pos=253)), (CAPACITY, dict(table_len=103)), (CAPACITY, dict(n=2**31 - 1)),
    (ALIGN, dict(q=KvqRows(24, 0, 0))), (ALIGN, dict(k=KvqRows(16, 0, 260))), (ALIGN, dict(q_out=KvqRows(16, 4, 0))),
    (ALIGN, dict(table=P(40)))])
def test_rope_append_refuses(want, over):
    assert rope(**over) == want


@pytest.mark.parametrize("want,r,first,n,table", [
    (0, RopeConfig(64), 0, 0, None), (INVALID, RopeConfig(64), -1, 4, P(16)), (INVALID, RopeConfig(64), 0, -1, P(16)),
    (INVALID, RopeConfig(64), 2**31 - 4, 4, P(16)), (INVALID, RopeConfig(64), 0, 4, None),
    (ALIGN, RopeConfig(64), 0, 4, P(24)), (UNSUPPORTED, RopeConfig(130), 0, 4, P(16)),
    (INVALID, RopeConfig(64, scaling=5), 0, 4, P(16)), (INVALID, RopeConfig(64, base=1.0), 0, 4, P(16)),
    (INVALID, RopeConfig(64, scaling=1, factor=0.5), 0, 4, P(16)),
    (INVALID, RopeConfig(64, scaling=3, factor=2.0), 0, 4, P(16)),
    (INVALID, RopeConfig(64, scaling=4, factor=2.0, orig_len=64, low=4.0, high=4.0), 0, 4, P(16)),
    (INVALID, RopeConfig(64, gain=-1.0), 0, 4, P(16)), (INVALID, RopeConfig(64, base=float("inf")), 0, 4, P(16))])
def test_rope_table_refuses(want, r, first, n, table):
    assert kvq.lib().kvq_rope_table(ref(r.c()), first, n, table, None) == want


def read(cfg=None, layer=LAYER, k=KvqRows(16, 0, 0), v=KvqRows(32, 0, 0), dtype=0, d_pos=P(64), max_pos=100, n=4):
    return kvq.lib().kvq_read(ref(cfg or config()), ref(layer), ref(k), ref(v), dtype, d_pos, max_pos, n, None, None)


@pytest.mark.parametrize("want,over", [
    (0, dict(n=0)), (0, dict(n=0, v=None)), (0, dict(n=0, k=None)), (0, dict(n=0, cfg=config(**H), v=None)),
    (INVALID, dict(k=None, v=None)), (INVALID, dict(layer=None)), (INVALID, dict(d_pos=None)), (INVALID, dict(n=-1)),
    (INVALID, dict(max_pos=-1)), (INVALID, dict(dtype=7)), (INVALID, dict(cfg=config(**H))),
    (INVALID, dict(cfg=config(page_tokens=128, n_pages=4))), (INVALID, dict(k=KvqRows(None, 0, 0))),
    (CAPACITY, dict(max_pos=253)), (ALIGN, dict(k=KvqRows(18, 0, 0))), (ALIGN, dict(v=KvqRows(16, 0, 12))),
    (ALIGN, dict(dtype=1, v=KvqRows(16, 0, 258)))])
def test_read_refuses(want, over):
    assert read(**over) == want


def commit(cfg=None, layers=(LAYER,), d_len=P(64), max_len=100, n=8, path=P(80), stride=8, n_path=P(96), out=P(112)):
    arr = (KvqLayer * max(1, len(layers)))(*layers)
    return kvq.lib().kvq_tree_commit(ref(cfg or config()), arr, len(layers), d_len, max_len, n, path, stride, n_path,
                                     out, None)


@pytest.mark.parametrize("want,over", [
    (INVALID, dict(layers=())), (INVALID, dict(d_len=None)), (INVALID, dict(path=None)), (INVALID, dict(n_path=None)),
    (INVALID, dict(max_len=-1)), (INVALID, dict(n=0)), (INVALID, dict(n=65, stride=8)), (INVALID, dict(stride=0)),
    (INVALID, dict(stride=9)), (INVALID, dict(out=P(64))), (INVALID, dict(cfg=config(**H))),
    (INVALID, dict(layers=(LAYER, KvqLayer(160, 16, 64, 48), LAYER))), (INVALID, dict(layers=(LAYER, KvqLayer(160, 16, 32, 48)))),
    (INVALID, dict(layers=(LAYER, KvqLayer(16, 16, None, 48)))), (UNSUPPORTED, dict(cfg=config(**WINDOW))),
    (CAPACITY, dict(max_len=249)), (ALIGN, dict(layers=(KvqLayer(24, 16, 32, 48),)))])
def test_commit_refuses(want, over):
    assert commit(**over) == want


def test_binding_refuses_what_pointers_cannot_show():
    rows = kvq._rows
    x = torch.zeros(2, 3, 4, 128, dtype=torch.float16)
    assert rows(x, 3, 4, 128, 2, torch.float16, "x") == bytes(KvqRows(x.data_ptr(), 1536, 512))
    one = rows(x[:1, :1], 1, 4, 128, 1, torch.float16, "x")       # strides that no index uses
    assert one == bytes(KvqRows(x.data_ptr(), 0, 0))
    for bad in (x.float(), x[:, :2], x.transpose(2, 3), x[..., ::2], x[:, :, ::2], x[:, :1].expand(2, 3, 4, 128)):
        with pytest.raises(ValueError):
            rows(bad, 3, 4, 128, 2, torch.float16, "x")
    with pytest.raises(ValueError):
        kvq._ints(torch.zeros(2), (2,), "d_pos")
    with pytest.raises(ValueError):
        kvq._ints(torch.zeros(3, dtype=torch.int32), (2,), "d_pos")
    cfg = Config(batch=2, capacity=64, n_q_heads=2, n_kv_heads=2, head_dim=128)
    n = kvq.kvq_layer_buffer_bytes(cfg)
    bufs = [torch.zeros(b, dtype=torch.uint8) for b in n]
    assert kvq.LayerCache.from_buffers(cfg, *bufs).c().v_codes == bufs[2].data_ptr()
    with pytest.raises(ValueError):
        kvq.LayerCache.from_buffers(cfg, bufs[0][1:], *bufs[1:])
    with pytest.raises(ValueError):
        kvq.LayerCache.from_buffers(cfg, bufs[0], None, *bufs[2:])
