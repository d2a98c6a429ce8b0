"""Workloads of the operators around drafted tokens and rotated keys over a quantised cache.

Four operators, as a serving program calls them between two forward passes:

  rope    kvq_rope_append: rotates a step's queries and keys by their positions and quantises
          keys and values into the cache; kvq_read then gives the rows back as 16-bit values.
  read    kvq_read: dequantises a range of tokens of every sequence.
  tree    kvq_tree_attn: attention of a tree of drafted tokens over a cache.
  commit  kvq_tree_commit: moves the accepted path's rows to the front of the drafted region,
          for all layers at once.

`run` computes them in plain torch operations (own = False) or through the package's calls.
Cache layouts are the package's: codes [B][Hkv][capacity][row bytes] (paged: [pages][Hkv][128]
[row bytes] behind a block table), fp16 scales per group of a row.
"""
import math

import torch

own = False

PAGE = 128
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one small model's request with a short draft: latency is all that counts
        tree("tree-1x250-d64-t6", batch=1, hq=4, hkv=4, dh=64, length=250, t=6, kg=64, vg=64),
        # the 8K serving batch with an ordinary tree
        tree("tree-16x8k-t16", batch=16, hq=32, hkv=8, length=8175, t=16, dtype="bf16"),
        # the same with the widest tree, over every cached token
        tree("tree-16x8k-t64", batch=16, hq=32, hkv=8, length=8128, t=64),
        # three queries a KV head, values in 4-bit groups, ragged lengths and tree sizes
        tree("tree-8x2k-t24-k8v4g32", batch=8, hq=24, hkv=8, length=2011, t=24, vb=4, vg=32,
             ragged=True),
        # many requests over a shared pool of pages, 4-bit keys and values
        tree("tree-64x4k-t8-paged-k4v4", batch=64, hq=32, hkv=8, length=4000, t=8, kb=4, vb=4,
             paged=True, ragged=True, dtype="bf16"),
        # one decode step of a batch: keys in 4-bit groups, values in 8 bits
        rope("rope-64x1-k4g32v8", batch=64, hq=24, hkv=8, length=2000, n=1, kb=4, kg=32),
        # the drafted tokens of a batch, placed by their depth; interleaved pairs, half the head
        rope("rope-16x16-paged-interleaved", batch=16, hq=32, hkv=8, length=2001, n=16, rot=64,
             layout="interleaved", paged=True, ragged=True, depth=True),
        # a prompt beyond the trained length
        rope("rope-2x4096-yarn", batch=2, hq=32, hkv=8, length=24576, n=4096, dtype="bf16",
             scaling="yarn"),
        # a whole cache handed on in 16 bits
        read("read-16x8k-k8v8", batch=16, hkv=8, length=0, n=8192),
        # the tail of ragged sequences in a pool of pages, 4-bit groups
        read("read-16x515-paged-k4v4g32", batch=16, hkv=8, length=1533, n=515, kb=4, vb=4, kg=32,
             vg=32, paged=True, ragged=True, dtype="bf16"),
        # one layer's accepted path, single request
        commit("commit-1x1-t8", batch=1, hkv=8, layers=1, length=500, t=8),
        # a model's layers after a verified draft
        commit("commit-32x16-t16", batch=16, hkv=8, layers=32, length=1009, t=16),
    ]


def tree(name, batch, hq, hkv, length, t, dh=128, kb=8, vb=8, kg=128, vg=128, fmt="int",
         paged=False, ragged=False, dtype="f16"):
    return dict(name=name, op="tree", batch=batch, hq=hq, hkv=hkv, dh=dh, length=length, t=t,
                kb=kb, vb=vb, kg=kg, vg=vg, fmt=fmt, paged=paged, ragged=ragged, dtype=dtype)


def rope(name, batch, hq, hkv, length, n, dh=128, rot=None, layout="half", scaling="none", kb=8,
         vb=8, kg=128, vg=128, fmt="int", paged=False, ragged=False, depth=False, dtype="f16"):
    return dict(name=name, op="rope", batch=batch, hq=hq, hkv=hkv, dh=dh, length=length, n=n,
                rot=rot or dh, layout=layout, scaling=scaling, kb=kb, vb=vb, kg=kg, vg=vg,
                fmt=fmt, paged=paged, ragged=ragged, depth=depth, dtype=dtype)


def read(name, batch, hkv, length, n, dh=128, kb=8, vb=8, kg=128, vg=128, fmt="int", paged=False,
         ragged=False, dtype="f16"):
    return dict(name=name, op="read", batch=batch, hq=hkv, hkv=hkv, dh=dh, length=length, n=n,
                kb=kb, vb=vb, kg=kg, vg=vg, fmt=fmt, paged=paged, ragged=ragged, dtype=dtype)


def commit(name, batch, hkv, layers, length, t, dh=128):
    return dict(name=name, op="commit", batch=batch, hq=hkv, hkv=hkv, dh=dh, layers=layers,
                length=length, t=t, kb=16, vb=16, kg=dh, vg=dh, fmt="int", paged=False,
                ragged=True, dtype="f16")


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _format(rng, dh):
    fmt = rng.choice(["int", "int", "int", "int", "e4m3", "asym"])
    kb, vb = (8, 8) if fmt != "int" else rng.choice([(8, 8), (8, 8), (8, 4), (4, 8), (4, 4), (16, 16)])
    groups = [g for g in (32, 64, 128) if g <= dh] + [dh, dh]
    return dict(fmt=fmt, kb=kb, vb=vb, kg=rng.choice(groups), vg=rng.choice(groups))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "rope", "read", "commit"])
    dh = rng.choice([128, 128, 128, 64])
    hkv = rng.choice([1, 2, 4, 8, 8])
    g = rng.choice([1, 2, 3, 4, 4, 5, 8])
    dtype = rng.choice(["f16", "bf16"])
    if op == "commit":
        return _unnamed(commit("", _log(rng, 1, 32), hkv, _log(rng, 1, 32), _log(rng, 1, 1000),
                               _log(rng, 1, 32), dh))
    more = dict(dh=dh, paged=rng.random() < 0.3, ragged=rng.random() < 0.5, dtype=dtype,
                **_format(rng, dh))
    batch = _log(rng, 1, 48)
    if op == "tree":
        # tokens of all sequences and KV heads, and scores, within the largest listed case
        t = _log(rng, 1, 64)
        most = min(2 ** 20 // (batch * hkv), 2 ** 28 // (batch * hkv * t * g), 2 ** 15)
        return _unnamed(tree("", batch, hkv * g, hkv, _log(rng, 1, max(2, most)) - 1, t, **more))
    if op == "rope":
        n = _log(rng, 1, max(2, 2 ** 18 // (batch * hkv * (g + 2))))
        rot = rng.choice([dh, dh, dh // 2, dh // 4, 24])
        return _unnamed(rope("", batch, hkv * g, hkv, _log(rng, 1, 4000) - 1, n, rot=rot,
                             layout=rng.choice(["half", "interleaved"]),
                             scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                             depth=n <= 64 and rng.random() < 0.5, **more))
    n = _log(rng, 1, max(2, 2 ** 20 // (batch * hkv)))
    return _unnamed(read("", batch, hkv, _log(rng, 1, 2000) - 1, n, **more))


def _unnamed(case):
    del case["name"]
    return case


def _spread(most, batch, ragged, least, turn):
    """Per-sequence sizes from `least` to `most`: the same ones for every seed of a case."""
    if not ragged or batch == 1:
        return [most] * batch
    return [least + (most - least) * ((b * 37 + turn) % batch) // (batch - 1) for b in range(batch)]


def _sizes(case):
    """(cached tokens, new tokens) of every sequence."""
    lens = _spread(case["length"], case["batch"], case["ragged"], min(1, case["length"]), 0)
    new = _spread(case.get("t") or case["n"], case["batch"], case["ragged"], 1, 11)
    return lens, new


def _capacity(case):
    """Tokens a sequence has room for: a program's power-of-two steps, whole pages."""
    need = case["length"] + (case.get("t") or case["n"])
    step = 16 if need <= 256 else PAGE
    return -(-need // step) * step if not case["paged"] else -(-need // PAGE) * PAGE


def _row_bytes(case):
    """Bytes of one (token, KV head): (K codes, K scales, V codes, V scales)."""
    dh = case["dh"]
    pair = 2 if case["fmt"] == "asym" else 1
    k, v = ((dh * b // 8, 0 if b == 16 else dh // g * 2 * pair)
            for b, g in ((case["kb"], case["kg"]), (case["vb"], case["vg"])))
    return k + v


def work(case):
    lens, new = _sizes(case)
    hq, hkv, dh, row = case["hq"], case["hkv"], case["dh"], sum(_row_bytes(case))
    if case["op"] == "tree":
        # cache rows read once; queries, masks and outputs; two products of every score
        # (a drafted token sees the whole prefix and, at most, every drafted token)
        seen = sum(a + t for a, t in zip(lens, new))
        pairs = sum((a + (t + 1) / 2) * t for a, t in zip(lens, new))
        return {"bytes": seen * hkv * row + sum(new) * (hq * dh * 4 + 8),
                "flops": 4 * pairs * hq * dh}
    if case["op"] == "rope":
        # q, k, v read; q and codes written; codes read and values written by the read-back
        n = sum(new)
        angles = n * case["rot"] * 4
        return {"bytes": n * (hq * dh * 4 + hkv * dh * 4 + hkv * row * 2 + hkv * dh * 4) + angles,
                "flops": n * (hq + hkv) * case["rot"] * 3 + n * hkv * dh * 6}
    if case["op"] == "read":
        n = sum(new)
        return {"bytes": n * hkv * (row + dh * 4), "flops": n * hkv * dh * 2}
    moved = sum(_path_length(case, t) for t in new) * case["layers"]
    return {"bytes": moved * hkv * row * 2, "flops": 0}


def _path_length(case, t):
    """Accepted tokens of a tree of t drafted ones: about half of them in depth."""
    return (t + 1) // 2


# --------------------------------------------------------------------------- inputs

def _normal(shape, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _quantise(x, bits, group, fmt):
    """Rows of 32-bit values -> (codes as bytes, fp16 scales), by the cache formats' definition."""
    if bits == 16:
        return x.to(torch.float16).view(torch.uint8), None
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    if fmt == "asym":
        lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
        s16 = ((hi - lo) / 255).to(torch.float16).clamp(max=65504)
        s = s16.float()
        ok = s > 0
        one = torch.where(ok, s, torch.ones_like(s))
        z = torch.where(ok, torch.round(-lo / one).clamp(0, 255), torch.zeros_like(s))
        c = (torch.round(g / one[..., None]) + z[..., None]).clamp(0, 255)
        c = torch.where(ok[..., None], c, torch.zeros_like(c))
        scales = torch.stack([s16, z.to(torch.float16)], -1)
        return c.to(torch.uint8).reshape(x.shape), scales.reshape(*x.shape[:-1], -1)
    most = 448.0 if fmt == "e4m3" else 127.0 if bits == 8 else 7.0
    s16 = (g.abs().amax(-1) / most).to(torch.float16).clamp(max=65504)
    s = s16.float()[..., None]
    y = torch.where(s > 0, g / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    if fmt == "e4m3":
        c = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape)
    else:
        c = torch.round(y).clamp(-most, most).to(torch.int8).reshape(x.shape)
        c = c.view(torch.uint8) if bits == 8 else (c[..., 0::2] & 15 | c[..., 1::2] << 4).view(torch.uint8)
    return c, s16


def _values(codes, scales, bits, group, fmt):
    """Bytes and scales of rows -> 32-bit values."""
    if bits == 16:
        return codes.view(torch.float16).float()
    if bits == 4:
        c = torch.stack([(codes & 15 ^ 8).float() - 8, (codes >> 4 ^ 8).float() - 8], -1).flatten(-2)
    elif fmt == "e4m3":
        c = codes.view(torch.float8_e4m3fn).float()
    elif fmt == "asym":
        c = codes.float()
    else:
        c = codes.view(torch.int8).float()
    c = c.reshape(*c.shape[:-1], c.shape[-1] // group, group)
    if fmt == "asym":
        pair = scales.float().reshape(*c.shape[:-1], 2)
        return ((c - pair[..., 1:]) * pair[..., :1]).flatten(-2)
    return (c * scales.float()[..., None]).flatten(-2)


def _cache(case, gen, filled):
    """Buffers of one layer with `filled` tokens of every sequence quantised from N(0, 1)."""
    batch, hkv, dh, cap = case["batch"], case["hkv"], case["dh"], _capacity(case)
    s = {"cap": cap, "table": None}
    pages = cap // PAGE
    if case["paged"]:
        s["n_pages"] = batch * pages + 5
        order = torch.randperm(s["n_pages"], generator=gen, device="cuda")
        s["table"] = order[: batch * pages].reshape(batch, pages).to(torch.int32)
    kc, ks, vc, vs = _row_bytes(case)
    for name, nc, ns, bits, group in (("k", kc, ks, case["kb"], case["kg"]), ("v", vc, vs, case["vb"], case["vg"])):
        rows = (s["n_pages"], hkv, PAGE) if case["paged"] else (batch, hkv, cap)
        codes = torch.zeros(*rows, nc, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(*rows, ns // 2, dtype=torch.float16, device="cuda") if ns else None
        for b in range(batch if filled else 0):
            c, sc = _quantise(_normal((hkv, cap, dh), gen), bits, group, case["fmt"])
            for buf, x in ((codes, c), (scales, sc)):
                if x is None:
                    continue
                if case["paged"]:
                    buf[s["table"][b].long()] = x.reshape(hkv, pages, PAGE, -1).transpose(0, 1)
                else:
                    buf[b] = x
        s[name + "_codes"], s[name + "_scales"] = codes, scales
    return s


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _parents(case, new, seed):
    """A random tree for every sequence: the parent of each drafted token (-1: the prefix)."""
    import random
    rng = random.Random(seed)
    return [[-1 if j == 0 or rng.random() < 0.1 else rng.randrange(max(0, j - 4), j) for j in range(t)]
            for t in new]


def rotation_table(scaling, rot, n_pos, dh, base=10000.0, factor=8.0, trained=4096):
    """(cos, sin) of every position and pair, from angles in 64 bits: float32 [n_pos][rot/2][2]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    gain = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    freq = base ** (-2 * i / rot)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        # dimensions that turn less than once in the trained length are stretched, those that
        # turn more than 32 times are kept, with a ramp between
        lo = math.floor(rot * math.log(trained / (32 * 2 * math.pi)) / (2 * math.log(base)))
        hi = math.ceil(rot * math.log(trained / (1 * 2 * math.pi)) / (2 * math.log(base)))
        lo, hi = max(lo, 0), min(hi, rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        freq = freq / factor * ramp + freq * (1 - ramp)
        gain = 0.1 * math.log(factor) + 1
    elif scaling == "bands":
        # the same by wavelength: 1 and 4 turns in the trained length bound the ramp
        keep = ((trained * freq / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        freq = freq / factor * (1 - keep) + freq * keep
    angle = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([angle.cos() * gain, angle.sin() * gain], -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    lens, new = _sizes(case)
    op, batch, hq, hkv, dh = case["op"], case["batch"], case["hq"], case["hkv"], case["dh"]
    dt = DT[case["dtype"]]
    if op == "commit":
        t, cap = case["t"], _capacity(case)
        s = {"cap": cap, "table": None}
        for name in ("k", "v"):
            x = _normal((case["layers"], batch, hkv, cap, dh), gen, torch.float16)
            s[name + "_codes"], s[name + "_scales"] = x.view(torch.uint8), None
        import random
        rng = random.Random(seed)
        paths = [sorted(rng.sample(range(n), _path_length(case, n))) for n in new]
        most = max(len(p) for p in paths)
        s["path"] = _ints([p + [-1] * (most - len(p)) for p in paths])
        s["n_path"] = _ints([len(p) for p in paths])
        s["d_len"] = _ints(lens)
        s["new_len"] = torch.zeros(batch, dtype=torch.int32, device="cuda")
        return {"case": case, **s}
    s = _cache(case, gen, filled=op != "rope")
    s["d_len"], s["d_new"] = _ints(lens), _ints(new)
    n = case.get("t") or case["n"]
    if op == "tree":
        s["q"] = _normal((batch, n, hq, dh), gen, dt)
        masks = []
        for parents in _parents(case, new, seed):
            m = []
            for j, p in enumerate(parents):
                m.append((m[p] if p >= 0 else 0) | 1 << j)
            masks.append([x - (x >> 63 << 64) for x in m] + [0] * (n - len(m)))
        s["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
        s["out"] = torch.zeros(batch, n, hq, dh, dtype=dt, device="cuda")
    if op == "rope":
        # one projection's output: the rows of q, k and v side by side
        qkv = _normal((batch, n, hq + 2 * hkv, dh), gen, dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        s["rope_pos"] = None
        if case["depth"]:
            depths = []
            for b, parents in enumerate(_parents(case, new, seed)):
                d = []
                for p in parents:
                    d.append(d[p] + 1 if p >= 0 else 0)
                depths.append([lens[b] + x for x in d] + [0] * (n - len(d)))
            s["rope_pos"] = _ints(depths)
        s["table32"] = rotation_table(case["scaling"], case["rot"], s["cap"], dh).float()
        s["q_out"] = torch.zeros(batch, n, hq, dh, dtype=dt, device="cuda")
    if op in ("rope", "read"):
        s["k_out"] = torch.zeros(batch, n, hkv, dh, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros(batch, n, hkv, dh, dtype=dt, device="cuda")
    return {"case": case, **s}


# --------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return {"tree": _plain_tree, "rope": _plain_rope, "read": _plain_read, "commit": _plain_commit}[op](state)


def _all_rows(state, name):
    """Codes and scales of a tensor as [B][Hkv][capacity][...]."""
    got = []
    for x in (state[name + "_codes"], state[name + "_scales"]):
        if x is not None and state["table"] is not None:
            x = x[state["table"].long()].transpose(1, 2).flatten(2, 3)
        got.append(x)
    return got


def _plain_tree(state):
    case = state["case"]
    q, mask = state["q"].float(), state["mask"]
    batch, t, hq, dh = q.shape
    hkv = case["hkv"]
    k = _values(*_all_rows(state, "k"), case["kb"], case["kg"], case["fmt"])
    v = _values(*_all_rows(state, "v"), case["vb"], case["vg"], case["fmt"])
    q = q.reshape(batch, t, hkv, hq // hkv, dh).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(dh))
    at = torch.arange(state["cap"], device="cuda") - state["d_len"][:, None].long()
    drafted = (mask[:, :, None] >> at.clamp(0, 63)[:, None, :]) & 1
    seen = (at < 0)[:, None, :] | ((at >= 0) & (at < state["d_new"][:, None]))[:, None, :] & (drafted == 1)
    seen = seen[:, None, :, None, :].expand(-1, -1, -1, hq // hkv, -1).flatten(2, 3)
    scores = scores.masked_fill(~seen, float("-inf"))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    o = o.reshape(batch, hkv, t, hq // hkv, dh).permute(0, 2, 1, 3, 4).flatten(2, 3)
    live = torch.arange(t, device="cuda") < state["d_new"][:, None]
    return torch.where(live[:, :, None, None], o, torch.zeros_like(o)).to(state["out"].dtype)


def _rotate(x, table, rot, layout):
    """x [B][n][H][dh] in 32 bits, table [B][n][rot/2][2]."""
    c, s = table[..., None, :, 0], table[..., None, :, 1]
    head, tail = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        head = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([head, tail], -1)


def _places(state, n):
    """(live, sequence, position, page and slot or sequence and slot) of every new token."""
    j = torch.arange(n, device="cuda")
    live = j < state["d_new"][:, None]
    pos = (state["d_len"][:, None] + j).long().clamp(max=state["cap"] - 1)
    if state["table"] is None:
        first = torch.arange(len(live), device="cuda")[:, None].expand_as(pos)
        return live, pos, first, pos
    return live, pos, state["table"].long().gather(1, pos // PAGE), pos % PAGE


def _plain_rope(state):
    case, n = state["case"], state["q"].shape[1]
    live, pos, first, slot = _places(state, n)
    at = pos if state["rope_pos"] is None else state["rope_pos"].long()
    table = state["table32"][at]
    rows = live[:, :, None, None]
    q = _rotate(state["q"].float(), table, case["rot"], case["layout"])
    k = _rotate(state["k"].float(), table, case["rot"], case["layout"])
    got = {"q": torch.where(rows, q, torch.zeros_like(q)).to(state["q"].dtype)}
    for name, x, bits, group in (("k", k, case["kb"], case["kg"]), ("v", state["v"].float(), case["vb"], case["vg"])):
        codes, scales = _quantise(x, bits, group, case["fmt"])
        for buf, rows_new in ((state[name + "_codes"], codes), (state[name + "_scales"], scales)):
            if rows_new is not None:
                buf[first[live], :, slot[live]] = rows_new[live]
    return {**got, **_plain_read(state)}


def _plain_read(state):
    case, n = state["case"], state["k_out"].shape[1]
    live, _, first, slot = _places(state, n)
    got = {}
    for name, bits, group in (("k", case["kb"], case["kg"]), ("v", case["vb"], case["vg"])):
        codes, scales = (None if x is None else x[first, :, slot] for x in (state[name + "_codes"], state[name + "_scales"]))
        x = _values(codes, scales, bits, group, case["fmt"])
        got[name] = torch.where(live[:, :, None, None], x, torch.zeros_like(x)).to(state["k_out"].dtype)
    return got


def _plain_commit(state):
    path, n_path = state["path"].long(), state["n_path"]
    batch, most = path.shape
    live = torch.arange(most, device="cuda") < n_path[:, None]
    b = torch.arange(batch, device="cuda")[:, None].expand(batch, most)[live]
    to = (state["d_len"][:, None] + torch.arange(most, device="cuda"))[live].long()
    src = (state["d_len"][:, None] + path)[live].long()
    for name in ("k_codes", "v_codes"):
        x = state[name]
        x[:, b, :, to] = x[:, b, :, src]
    state["new_len"].copy_(state["d_len"] + n_path)
    return {"k": state["k_codes"].view(torch.float16), "v": state["v_codes"].view(torch.float16),
            "len": state["new_len"]}


# ---- the package's calls: the configuration, the cache handle and the workspace are made once

def _handles(state):
    import quantized_kv_cache_22_b200 as kvq
    if "cfg" not in state:
        case = state["case"]
        fmt = {"int": kvq.KVQ_FMT_INT, "e4m3": kvq.KVQ_FMT_E4M3, "asym": kvq.KVQ_FMT_ASYM}[case["fmt"]]
        paged = dict(page_tokens=PAGE, n_pages=state["n_pages"]) if case["paged"] else {}
        state["cfg"] = cfg = kvq.Config(
            batch=case["batch"], capacity=state["cap"], n_q_heads=case["hq"], n_kv_heads=case["hkv"],
            head_dim=case["dh"], k_bits=case["kb"], v_bits=case["vb"], k_group=case["kg"],
            v_group=case["vg"], kv_format=fmt, **paged)
        parts = [state[x] for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
        if case["op"] == "commit":
            state["layers"] = [kvq.LayerCache.from_buffers(cfg, k, None, v, None)
                               for k, v in zip(state["k_codes"], state["v_codes"])]
        else:
            state["layer"] = kvq.LayerCache.from_buffers(cfg, *parts, block_table=state["table"])
        if case["op"] == "tree":
            state["ws"] = kvq.TreeWorkspace(cfg, case["t"])
        if case["op"] == "rope":
            state["rope"] = kvq.RopeConfig(rot_dim=case["rot"], layout={
                "half": kvq.KVQ_ROPE_HALF, "interleaved": kvq.KVQ_ROPE_INTERLEAVED}[case["layout"]])
        state["most"] = max(_sizes(case)[0])
    return kvq


def _own_tree(s):
    kvq = _handles(s)
    kvq.kvq_tree_attn(s["cfg"], s["layer"], s["q"], s["d_len"], s["most"], s["mask"], s["out"], s["ws"],
                      d_n_tree=s["d_new"])
    return s["out"]


def _own_rope(s):
    kvq = _handles(s)
    kvq.kvq_rope_append(s["cfg"], s["layer"], s["rope"], s["table32"], s["q"], s["k"], s["v"], s["q_out"],
                        s["d_len"], s["most"], d_count=s["d_new"], d_rope_pos=s["rope_pos"])
    return {"q": s["q_out"], **_own_read(s)}


def _own_read(s):
    kvq = _handles(s)
    kvq.kvq_read(s["cfg"], s["layer"], s["k_out"], s["v_out"], s["d_len"], s["most"], d_count=s["d_new"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_commit(s):
    kvq = _handles(s)
    kvq.kvq_tree_commit(s["cfg"], s["layers"], s["d_len"], s["most"], s["path"], s["n_path"], s["case"]["t"],
                        d_len_out=s["new_len"])
    return {"k": s["k_codes"].view(torch.float16), "v": s["v_codes"].view(torch.float16), "len": s["new_len"]}


_OWN = {"tree": _own_tree, "rope": _own_rope, "read": _own_read, "commit": _own_commit}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _sizes(case)
    batch, hkv, dh = case["batch"], case["hkv"], case["dh"]
    if case["op"] == "commit":
        got = {"k": s["k_codes"].view(torch.float16).double(), "v": s["v_codes"].view(torch.float16).double(), "len": None}
        for b in range(batch):
            for i, j in enumerate(s["path"][b, : int(s["n_path"][b])].tolist()):
                for name in ("k", "v"):
                    got[name][:, b, :, lens[b] + i] = got[name][:, b, :, lens[b] + j]
        return got
    if case["op"] == "tree":
        hq, t = case["hq"], case["t"]
        out = torch.zeros(batch, t, hq, dh, dtype=torch.float64, device="cuda")
        for b in range(batch):
            k = _exact_rows(s, "k", b, lens[b] + new[b])
            v = _exact_rows(s, "v", b, lens[b] + new[b])
            kk = k.repeat_interleave(hq // hkv, 0)
            vv = v.repeat_interleave(hq // hkv, 0)
            for j in range(new[b]):
                bits = int(s["mask"][b, j])
                keep = list(range(lens[b])) + [lens[b] + i for i in range(new[b]) if bits >> i & 1]
                drop = torch.ones(lens[b] + new[b], dtype=torch.bool, device="cuda")
                drop[torch.tensor(keep, device="cuda", dtype=torch.long)] = False
                x = torch.einsum("hd,hnd->hn", s["q"][b, j].double(), kk) / math.sqrt(dh)
                out[b, j] = torch.einsum("hn,hnd->hd", torch.softmax(x.masked_fill(drop, -math.inf), -1), vv)
        return out
    n = case["n"]
    got = {"k": torch.zeros(batch, n, hkv, dh, dtype=torch.float64, device="cuda"),
           "v": torch.zeros(batch, n, hkv, dh, dtype=torch.float64, device="cuda")}
    if case["op"] == "read":
        for b in range(batch):
            for name in ("k", "v"):
                rows = _exact_rows(s, name, b, lens[b] + new[b])[:, lens[b]:]
                got[name][b, : new[b]] = rows.transpose(0, 1)
        return got
    got["q"] = torch.zeros(batch, n, case["hq"], dh, dtype=torch.float64, device="cuda")
    table = rotation_table(case["scaling"], case["rot"], s["cap"], dh)
    rot = case["rot"]
    first = torch.arange(rot // 2, device="cuda") * (1 if case["layout"] == "half" else 2)
    second = first + (rot // 2 if case["layout"] == "half" else 1)
    for b in range(batch):
        pos = torch.arange(lens[b], lens[b] + new[b], device="cuda")
        if s["rope_pos"] is not None:
            pos = s["rope_pos"][b, : new[b]].long()
        turn = torch.complex(table[pos, :, 0], table[pos, :, 1])[:, None]
        for name, x in (("q", s["q"]), ("k", s["k"]), ("v", s["v"])):
            x = x[b, : new[b]].double()
            if name != "v":
                z = torch.complex(x[..., first], x[..., second]) * turn
                x[..., first], x[..., second] = z.real, z.imag
            if name != "q":
                x = _exact_round(x, *((case["kb"], case["kg"]) if name == "k" else (case["vb"], case["vg"])), case["fmt"])
            got[name][b, : new[b]] = x
    return got


def _exact_rows(s, name, b, n):
    """The first n tokens of sequence b as [Hkv][n][dh] in 64 bits."""
    case = s["case"]
    bits, group, dh = (case["kb"], case["kg"], case["dh"]) if name == "k" else (case["vb"], case["vg"], case["dh"])
    at = torch.arange(n, device="cuda")
    if s["table"] is None:
        pick = lambda x: x[b, :, :n]  # noqa: E731
    else:
        page = s["table"][b].long()[at // PAGE]
        pick = lambda x: x[page, :, at % PAGE].transpose(0, 1)  # noqa: E731
    c = pick(s[name + "_codes"])
    if bits == 16:
        return c.contiguous().view(torch.float16).double()
    if bits == 4:
        signed = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device="cuda")
        x = torch.empty(*c.shape[:2], dh, dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = signed[(c % 16).long()], signed[(c // 16).long()]
    elif case["fmt"] == "e4m3":
        x = c.contiguous().view(torch.float8_e4m3fn).double()
    elif case["fmt"] == "asym":
        x = c.double()
    else:
        x = torch.where(c > 127, c.double() - 256, c.double())
    sc = pick(s[name + "_scales"]).double()
    if case["fmt"] == "asym":
        return (x - sc[..., 1::2].repeat_interleave(group, -1)) * sc[..., 0::2].repeat_interleave(group, -1)
    return x * sc.repeat_interleave(group, -1)


def _exact_round(x, bits, group, fmt):
    """x in 64 bits -> the values that its codes and fp16 scales stand for."""
    if bits == 16:
        return x.half().double()
    parts = []
    for y in x.split(group, -1):
        if fmt == "asym":
            lo = y.amin(-1, keepdim=True).clamp(max=0)
            s = ((y.amax(-1, keepdim=True).clamp(min=0) - lo) / 255).half().double()
            z = torch.round(-lo / s).clamp(0, 255)
            parts.append(((torch.round(y / s) + z).clamp(0, 255) - z) * s)
            continue
        most = 448 if fmt == "e4m3" else 2 ** (bits - 1) - 1
        s = (y.abs().amax(-1, keepdim=True) / most).half().double()
        c = (y / s).clamp(-most, most)
        parts.append((c.float().to(torch.float8_e4m3fn).double() if fmt == "e4m3" else torch.round(c)) * s)
    return torch.cat(parts, -1)
