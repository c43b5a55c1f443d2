"""Cases of the cache operators that work on whole blocks of rows, with their plain forms.

Three operators over the rotated INT2 cache (layout: include/oscar_kv.h):

* ``read``    kv_read: cached positions back as K and V rows in the model's basis;
* ``extend``  attn_extend: several new query tokens of each sequence attend its cache, causally;
* ``prefix``  attn_decode_prefix: one query token per sequence attends a prefix shared by the
  whole batch and then the sequence's own cache.

``own`` false computes them from the cache's bytes with elementary torch operations in 32 bits;
``own`` true calls the library.  ``exact`` computes them again in 64 bits.
"""
import math

import numpy as np
import torch

own = False

LM_RATIO = float(np.float32(1.16))  # gap ratio of the Lloyd-Max levels
MODES = {"int2": 0, "v_bf16": 16, "lloyd_max": 32}
HADAMARD, IN_FP32, OUT_FP32 = 8, 2, 4


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, q_heads=32, kv_heads=8, head_dim=128, sink=64, recent=256, length=1024, n=1,
             ragged=False, mode="int2", hadamard=False, fp32=False, prefix=0)
    c.update(kw)
    return c


def listed():
    return [
        # read: the last token of one sequence, as a check or a log takes it out (latency only)
        _case("read-token", "read", length=1000, n=1),
        # read: four prompts of 8192 tokens handed to another engine
        _case("read-prompt", "read", batch=4, q_heads=64, length=8192, n=8192),
        # read: ragged sequences at head_dim 512 with the windows inside the range, float32 rows
        _case("read-hd512", "read", batch=4, q_heads=16, head_dim=512, sink=512, recent=2048, length=4099, n=4099,
              ragged=True, fp32=True),
        # extend: five drafted tokens per sequence verified against 16K of context
        _case("extend-draft", "extend", batch=8, sink=512, recent=2048, length=16384, n=5, ragged=True),
        # extend: a 2048-token chunk of one long prompt, 64 query heads
        _case("extend-chunk", "extend", q_heads=64, length=16384, n=2048),
        # extend: the first chunk of three ragged prompts, odd sizes, Lloyd-Max levels
        _case("extend-first", "extend", batch=3, q_heads=24, length=777, n=777, ragged=True, mode="lloyd_max"),
        # extend: 32 tokens per sequence at head_dim 512
        _case("extend-hd512", "extend", batch=4, q_heads=16, head_dim=512, sink=512, recent=2048, length=16384, n=32),
        # prefix: two short conversations behind one system prompt (latency)
        _case("prefix-small", "prefix", batch=2, q_heads=8, kv_heads=2, prefix=700, length=40, ragged=True),
        # prefix: a serving batch of 32 over a 32K document, 1K of its own each
        _case("prefix-32", "prefix", batch=32, prefix=32768, length=1024, ragged=True),
        # prefix: 64 samples of one 128K context, 64 query heads
        _case("prefix-64", "prefix", batch=64, q_heads=64, prefix=131072, length=333, ragged=True),
        # prefix: values kept BF16
        _case("prefix-v-bf16", "prefix", batch=16, prefix=10001, length=513, ragged=True, mode="v_bf16"),
        # prefix: head_dim 256, data-free rotation
        _case("prefix-hd256", "prefix", batch=12, q_heads=16, kv_heads=4, head_dim=256, prefix=20000, length=200,
              ragged=True, hadamard=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["read", "extend", "prefix"])
    head_dim = rng.choice([128, 128, 128, 256, 512])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    kw = dict(head_dim=head_dim, kv_heads=kv_heads, q_heads=kv_heads * rng.randint(1, 8),
              sink=rng.choice([0, 7, 64, 512]), recent=rng.choice([0, 31, 256, 2048]), ragged=rng.random() < 0.5,
              mode=rng.choice(["int2", "int2", "v_bf16", "lloyd_max"]), hadamard=rng.random() < 0.2,
              fp32=rng.random() < 0.25)
    if op == "read":
        kw["batch"] = _log(rng, 1, 8)
        kw["n"] = _log(rng, 1, 8192 * 128 // head_dim // kw["batch"])
        kw["length"] = min(16384, kw["n"] + _log(rng, 1, 4096))
    elif op == "extend":
        kw["batch"] = _log(rng, 1, 8)
        kw["n"] = _log(rng, 1, 2048)
        most = int(2.0e9 // (kw["batch"] * kw["n"] * kw["q_heads"] * (head_dim // 128)))
        kw["n"] = min(kw["n"], max(1, most))
        kw["length"] = max(kw["n"], _log(rng, 16, max(17, min(16384, most))))
    else:
        kw["batch"] = _log(rng, 1, 64)
        kw["length"] = _log(rng, 1, 1024)
        kw["prefix"] = _log(rng, 100, min(65536, int(4.0e8 // (kw["batch"] * kw["q_heads"] * (head_dim // 128)))))
    c = _case("", op, **kw)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------
# inputs: a cache filled with quantised activations
# ------------------------------------------------------------------------------------------------
def _align(x):
    return (x + 255) // 256 * 256


def _layout(case, batch, capacity):
    """Sizes of a one-layer cache (kv_layout_query's formulas)."""
    h, d, s, w = case["kv_heads"], case["head_dim"], case["sink"], case["recent"]
    ncap = -(-max(capacity - s, 0) // 64) * 64
    sink, ring = _align(batch * h * s * d * 2), _align(batch * h * w * d * 2)
    codes, sz = _align(batch * h * ncap * (d // 4)), _align(batch * h * ncap * (d // 128) * 4)
    role = sink + ring + codes + sz
    v_role = _align(batch * h * capacity * d * 2) if case["mode"] == "v_bf16" else role
    return dict(ncap=ncap, batch=batch, capacity=capacity, at=(sink, sink + ring, sink + ring + codes), role=role,
                total=role + v_role)


def _view(lay, case, cache, role, region):
    """One region of a role as a typed tensor that shares the cache's memory."""
    b, h, d = lay["batch"], case["kv_heads"], case["head_dim"]
    base = lay["role"] if role else 0
    if region == "full":
        return cache[base:base + b * h * lay["capacity"] * d * 2].view(torch.bfloat16).view(b, h, lay["capacity"], d)
    if region == "sink":
        return cache[base:base + b * h * case["sink"] * d * 2].view(torch.bfloat16).view(b, h, case["sink"], d)
    if region == "ring":
        o = base + lay["at"][0]
        return cache[o:o + b * h * case["recent"] * d * 2].view(torch.bfloat16).view(b, h, case["recent"], d)
    if region == "codes":
        o = base + lay["at"][1]
        return cache[o:o + b * h * lay["ncap"] * d // 4].view(torch.int32).view(b, h, lay["ncap"], d // 16)
    o = base + lay["at"][2]
    return cache[o:o + b * h * lay["ncap"] * d // 32].view(torch.float16).view(b, h, lay["ncap"], d // 128, 2)


def _activations(shape, gen):
    """N(0, 1) rows with a few outlier channels (two per hundred, eight times larger with heavy tails), as bf16."""
    x = torch.randn(shape, generator=gen, device="cuda")
    ch = torch.arange(5, shape[-1], 47, device="cuda")
    z = torch.randn((4,) + tuple(shape[:-1]) + (len(ch),), generator=gen, device="cuda")
    x[..., ch] += 2.0 * z[0] / torch.sqrt(z[1:].square().mean(0) + 1e-3)
    return x.to(torch.bfloat16)


def _fill(case, lay, cache, lens, rots, gen):
    """Writes rows [0, lens[b]) of every sequence: the codec of kv_append, whole arrays at a time."""
    b, h, d, s, w = lay["batch"], case["kv_heads"], case["head_dim"], case["sink"], case["recent"]
    top = int(lens.max())
    if top == 0:
        return
    lm = case["mode"] == "lloyd_max"
    span = 2 * LM_RATIO + 1 if lm else 3.0
    at = torch.arange(top, device="cuda")
    for role in (0, 1):
        r = _activations((b, h, top, d), gen).float() @ rots[role]
        if s:
            _view(lay, case, cache, role, "sink" if not (role and case["mode"] == "v_bf16") else "full")[
                :, :, :min(s, top)] = r[:, :, :s].to(torch.bfloat16)
        if role and case["mode"] == "v_bf16":
            _view(lay, case, cache, 1, "full")[:, :, :top] = r.to(torch.bfloat16)
            continue
        if w:
            last = lens.view(b, 1) - w + torch.arange(w, device="cuda")
            ok = last >= 0
            rows = torch.gather(r, 2, last.clamp(min=0).view(b, 1, w, 1).expand(b, h, w, d)).to(torch.bfloat16)
            ring = _view(lay, case, cache, role, "ring")
            slot = (last % w).view(b, 1, w, 1).expand(b, h, w, d)
            ring.copy_(torch.zeros_like(ring).scatter_(2, slot, torch.where(ok.view(b, 1, w, 1), rows, 0)))
        if top <= s:
            continue
        r = r[:, :, s:]
        a = r.abs().amax(-1, keepdim=True) * (0.92 if role else 0.96)
        x = torch.maximum(torch.minimum(r, a), -a).view(b, h, top - s, d // 128, 128)
        lo, hi = x.amin(-1), x.amax(-1)
        sc, ze = ((hi - lo) / span).half(), lo.half()
        y = (x - ze.float()[..., None]) * torch.where(sc > 0, 1 / sc.float(), 0)[..., None]
        if lm:
            code = (y > LM_RATIO / 2).int() + (y > LM_RATIO + 0.5).int() + (y > span - LM_RATIO / 2).int()
        else:
            code = y.round().clamp(0, 3).int()
        if role == 0:  # channel = 64 i + 8 p + 2 c + hi of each group: word 2 c + i, bit 2 p + 16 hi
            code = code.view(b, h, top - s, d // 128, 2, 8, 4, 2).permute(0, 1, 2, 3, 6, 4, 7, 5)
        else:  # channel = 8 n + g: word g, bit 2 n
            code = code.view(b, h, top - s, d // 128, 2, 8, 8).permute(0, 1, 2, 3, 6, 4, 5)
        code = code.reshape(b, h, top - s, d // 16, 16).long()
        word = (code << (2 * torch.arange(16, device="cuda"))).sum(-1)
        word = torch.where(word >= 1 << 31, word - (1 << 32), word).int()
        written = (at[s:] < lens.view(b, 1)).view(b, 1, top - s, 1)
        _view(lay, case, cache, role, "codes")[:, :, :top - s] = torch.where(written, word, 0)
        _view(lay, case, cache, role, "sz")[:, :, :top - s] = torch.where(written[..., None], torch.stack((sc, ze), -1), 0)


def _rotations(case, seed):
    d = case["head_dim"]
    if case["hadamard"]:
        i = np.arange(128)
        par = np.array([[bin(x & y).count("1") & 1 for y in i] for x in i])
        r = np.kron(np.eye(d // 128), np.where(par, -1.0, 1.0) / math.sqrt(128.0))
        r = torch.from_numpy(r.astype(np.float32)).cuda()
        return r, r
    rng = np.random.default_rng(seed)
    return tuple(torch.from_numpy(np.linalg.qr(rng.standard_normal((d, d)))[0].astype(np.float32)).cuda() for _ in range(2))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng([seed, 1])
    b, hq, h, d, n, top = (case[k] for k in ("batch", "q_heads", "kv_heads", "head_dim", "n", "length"))
    lens = np.full(b, top)
    if case["ragged"] and b > 1:
        lens[1:] = np.maximum(1, (top * rng.uniform(0.25, 1.0, b - 1)).astype(int))
    st = dict(case=case, rots=_rotations(case, seed), scale=1.0 / math.sqrt(d))
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["lay"] = _layout(case, b, top + 16)
    st["cache"] = torch.zeros(st["lay"]["total"], dtype=torch.uint8, device="cuda")
    _fill(case, st["lay"], st["cache"], st["lens"].long(), st["rots"], gen)
    kind = torch.float32 if case["fp32"] else torch.bfloat16
    if case["op"] == "read":
        st["start"] = torch.tensor(np.maximum(0, lens - n), dtype=torch.int32, device="cuda")
        st["out"] = [torch.zeros(b, n, h, d, dtype=kind, device="cuda") for _ in range(2)]
    elif case["op"] == "extend":
        st["q"] = _activations((b, n, hq, d), gen).to(kind)
        st["q_lens"] = torch.tensor(np.minimum(lens, n), dtype=torch.int32, device="cuda")
        st["out"] = torch.zeros(b, n, hq, d, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros(b, n, hq, device="cuda")
    else:
        st["q"] = _activations((b, hq, d), gen).to(kind)
        st["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
        st["prefix_lay"] = _layout(case, 1, case["prefix"])
        st["prefix_cache"] = torch.zeros(st["prefix_lay"]["total"], dtype=torch.uint8, device="cuda")
        _fill(case, st["prefix_lay"], st["prefix_cache"], st["prefix_len"].long(), st["rots"], gen)
        st["out"] = torch.zeros(b, hq, d, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros(b, hq, device="cuda")
    return st


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _rows(case, lay, cache, role, lens, top):
    """Cached rows [batch][kv_heads][top][head_dim] in 32 bits, rotated basis, as attention sees them."""
    b, h, d, s, w = lay["batch"], case["kv_heads"], case["head_dim"], case["sink"], case["recent"]
    if role and case["mode"] == "v_bf16":
        return _view(lay, case, cache, 1, "full")[:, :, :top].float()
    at = torch.arange(top, device="cuda")
    body = min(s, top)
    word = _view(lay, case, cache, role, "codes")[:, :, :top - body]
    sz = _view(lay, case, cache, role, "sz")[:, :, :top - body].float()
    code = (word[..., None] >> (2 * torch.arange(16, device="cuda", dtype=torch.int32))) & 3
    if role == 0:
        code = code.view(b, h, top - body, d // 128, 4, 2, 2, 8).permute(0, 1, 2, 3, 5, 7, 4, 6)
    else:
        code = code.view(b, h, top - body, d // 128, 8, 16).permute(0, 1, 2, 3, 5, 4)
    level = code.reshape(b, h, top - body, d // 128, 128)
    if case["mode"] == "lloyd_max":
        level = torch.tensor([0.0, LM_RATIO, LM_RATIO + 1, 2 * LM_RATIO + 1], device="cuda")[level]
    x = (sz[..., 1:] + sz[..., :1] * level).view(b, h, top - body, d)
    if body:
        x = torch.cat((_view(lay, case, cache, role, "sink")[:, :, :body].float(), x), 2)
    if w:
        ring = _view(lay, case, cache, role, "ring")[:, :, at % w].float()
        recent = at >= torch.clamp(lens.view(b, 1) - w, min=s)
        x = torch.where(recent.view(b, 1, top, 1), ring, x)
    return x


def _plain_read(st):
    case, lens, n = st["case"], st["lens"].long(), st["case"]["n"]
    at = st["start"].long().view(-1, 1) + torch.arange(n, device="cuda")
    ok = (at < lens.view(-1, 1))[:, :, None, None]
    out = []
    for role in (0, 1):
        x = _rows(case, st["lay"], st["cache"], role, lens, case["length"])
        i = at.clamp(max=case["length"] - 1)[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3])
        x = (torch.gather(x, 2, i) @ st["rots"][role].T).transpose(1, 2)
        out.append(torch.where(ok, x.to(st["out"][role].dtype), st["out"][role]))
    return {"k": out[0], "v": out[1]}


def _softmax(s):
    """Row maxima, exponentials and their sums over the last dimension; empty rows give zeros."""
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - m)
    return m, p, p.sum(-1, keepdim=True)


def _plain_extend(st):
    case, lens, qlens = st["case"], st["lens"].long(), st["q_lens"].long()
    b, n, hq, d = st["q"].shape
    h, top = case["kv_heads"], case["length"]
    rk, rv = st["rots"]
    k, v = (_rows(case, st["lay"], st["cache"], role, lens, top) for role in (0, 1))
    q = (st["q"].float() @ rk).view(b, n, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    s = ((q @ k.transpose(2, 3)) * st["scale"]).view(b, h, hq // h, n, top)
    last = (lens - qlens).view(b, 1) + torch.arange(n, device="cuda")  # a query token's own position
    s = s.masked_fill_((torch.arange(top, device="cuda") > last[..., None])[:, None, None], -math.inf)
    m, p, l = _softmax(s)
    o = (p.view(b, h, -1, top) @ v).view(b, h, hq // h, n, d) / l
    o = (o @ rv.T).permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    lse = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2).reshape(b, n, hq)
    ok = (torch.arange(n, device="cuda") < qlens.view(b, 1))[..., None]
    return {"out": torch.where(ok[..., None], o.to(st["out"].dtype), st["out"]), "lse": torch.where(ok, lse, st["lse"])}


def _plain_prefix(st):
    case, lens = st["case"], st["lens"].long()
    b, hq, d = st["q"].shape
    h, top, pre = case["kv_heads"], case["length"], case["prefix"]
    g = hq // h
    rk, rv = st["rots"]
    k, v = (_rows(case, st["lay"], st["cache"], role, lens, top) for role in (0, 1))
    pk, pv = (_rows(case, st["prefix_lay"], st["prefix_cache"], role, st["prefix_len"].long(), pre) for role in (0, 1))
    q = (st["q"].float() @ rk).view(b, h, g, d)
    shared = q.transpose(0, 1).reshape(h, b * g, d) @ pk[0].transpose(1, 2)
    mine = (q @ k.transpose(2, 3)).masked_fill(torch.arange(top, device="cuda") >= lens.view(b, 1, 1, 1), -math.inf)
    m, p, l = _softmax(torch.cat((shared.view(h, b, g, pre).transpose(0, 1), mine), -1) * st["scale"])
    o = (p[..., :pre].transpose(0, 1).reshape(h, b * g, pre) @ pv[0]).view(h, b, g, d).transpose(0, 1)
    o = ((o + p[..., pre:] @ v) / l) @ rv.T
    return {"out": o.reshape(b, hq, d).to(st["out"].dtype), "lse": (m + torch.log(l)).view(b, hq)}


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------
def _config(case, batch, capacity):
    from int2_kv_cache_append_gb300 import oscar_kv as K

    flags = MODES[case["mode"]] | (HADAMARD if case["hadamard"] else 0)
    if case["fp32"]:
        flags |= OUT_FP32 if case["op"] == "read" else IN_FP32
    return K.KVConfig(1, batch, case["q_heads"], case["kv_heads"], case["head_dim"], case["sink"], case["recent"],
                      capacity, flags=flags)


def _own(st):
    from int2_kv_cache_append_gb300 import oscar_kv as K

    case = st["case"]
    if "cfg" not in st:  # what a program sets up once and keeps
        st["cfg"] = _config(case, case["batch"], st["lay"]["capacity"])
        if case["op"] == "extend":
            st["ws"] = torch.empty(K.attn_extend_workspace_bytes(st["cfg"], case["n"]), dtype=torch.uint8, device="cuda")
        elif case["op"] == "prefix":
            st["prefix_cfg"] = _config(case, 1, case["prefix"])
            st["ws"] = torch.empty(K.attn_decode_prefix_workspace_bytes(st["cfg"], st["prefix_cfg"]), dtype=torch.uint8,
                                   device="cuda")
    cfg, (rk, rv) = st["cfg"], (None, None) if case["hadamard"] else st["rots"]
    if case["op"] == "read":
        K.kv_read(cfg, st["cache"], 0, st["start"], st["lens"], rk, rv, st["out"][0], st["out"][1])
        return {"k": st["out"][0], "v": st["out"][1]}
    if case["op"] == "extend":
        K.attn_extend(cfg, st["cache"], 0, st["q"], st["lens"], rk, rv, st["out"], st["ws"], q_lens=st["q_lens"],
                      lse=st["lse"], seq_len_hint=case["length"])
    else:
        K.attn_decode_prefix(cfg, st["cache"], st["prefix_cfg"], st["prefix_cache"], 0, st["q"], st["lens"],
                             st["prefix_len"], rk, rv, st["out"], st["ws"], lse=st["lse"], seq_len_hint=case["length"],
                             prefix_len_hint=case["prefix"])
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"read": _plain_read, "extend": _plain_extend, "prefix": _plain_prefix}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def _token_bytes(case, tokens):
    """K and V bytes of `tokens` cached tokens of one (sequence, KV head)."""
    d = case["head_dim"]
    wide = min(tokens, case["sink"] + case["recent"])
    packed = d // 4 + d // 32
    body = (tokens - wide) * packed
    return wide * 4 * d + 2 * body if case["mode"] != "v_bf16" else wide * 2 * d + body + tokens * 2 * d


def work(case):
    b, hq, h, d, n, top = (case[k] for k in ("batch", "q_heads", "kv_heads", "head_dim", "n", "length"))
    fill = 0.625 if case["ragged"] else 1.0  # mean length of the ragged sequences behind the first
    mean = top * (1 + (b - 1) * fill) / b
    rots = 0 if case["hadamard"] else 8 * d * d
    turn = 14 * d if case["hadamard"] else 2 * d * d  # one row's rotation
    wide = 4 if case["fp32"] else 2
    if case["op"] == "read":
        rows = b * h * min(n, mean)
        share = min(n, mean) / mean
        return {"bytes": b * h * _token_bytes(case, int(mean)) * share + rows * 2 * d * wide + rots, "flops": 2 * rows * turn}
    if case["op"] == "extend":
        m = min(n, mean)
        pairs = b * m * (mean - (m - 1) / 2)
        return {"bytes": b * h * _token_bytes(case, int(mean)) + b * m * hq * (d * (wide + 2) + 4) + rots,
                "flops": 4 * hq * d * pairs + 2 * b * m * hq * turn}
    pairs = b * (case["prefix"] + mean)
    return {"bytes": h * _token_bytes(case, case["prefix"]) + b * h * _token_bytes(case, int(mean))
            + b * hq * (d * (wide + 2) + 4) + rots, "flops": 4 * hq * d * pairs + 2 * b * hq * turn}


# ------------------------------------------------------------------------------------------------
# 64 bits
# ------------------------------------------------------------------------------------------------
def _exact_rows(case, lay, cache, role, i, head, length):
    """Rows [0, length) of one (sequence, KV head) in 64 bits, in the model's basis times R: read byte by byte."""
    d, s, w, h = case["head_dim"], case["sink"], case["recent"], case["kv_heads"]
    unit = i * h + head
    base = lay["role"] * role

    def wide(offset, first, count):
        o = base + offset + first * d * 2
        return cache[o:o + count * d * 2].view(torch.bfloat16).view(count, d).double()

    if role and case["mode"] == "v_bf16":
        return wide(0, unit * lay["capacity"], length)
    x = torch.zeros(length, d, dtype=torch.float64, device="cuda")
    if length > s:
        rows = length - s
        o = base + lay["at"][1] + unit * lay["ncap"] * (d // 4)
        byte = cache[o:o + rows * (d // 4)].view(rows, d // 4).int()
        o = base + lay["at"][2] + unit * lay["ncap"] * (d // 32)
        sz = cache[o:o + rows * (d // 32)].view(torch.float16).view(rows, d // 128, 2).double()
        ch = np.arange(d)
        g, c = ch // 128, ch % 128
        if role == 0:
            word, bit = 8 * g + 2 * (c % 8 // 2) + c // 64, 2 * (c % 64 // 8) + 16 * (c % 2)
        else:
            word, bit = 8 * g + c % 8, 2 * (c // 8)
        where = torch.from_numpy(4 * word + bit // 8).cuda()
        shift = torch.from_numpy(bit % 8).int().cuda()
        level = (byte[:, where] >> shift) & 3
        if case["mode"] == "lloyd_max":
            level = torch.tensor([0.0, LM_RATIO, LM_RATIO + 1, 2 * LM_RATIO + 1], dtype=torch.float64, device="cuda")[level.long()]
        g = torch.from_numpy(g).cuda()
        x[s:] = sz[:, g, 1] + sz[:, g, 0] * level
    if s:
        x[:s] = wide(0, unit * s, min(s, length))
    first = max(s, length - w)
    if w and first < length:
        slots = torch.arange(first, length, device="cuda") % w
        x[first:] = wide(lay["at"][0], unit * w, w)[slots]
    return x


def exact(case, seed):
    st = prepare(case, seed)
    b, hq, h, d, n = (case[k] for k in ("batch", "q_heads", "kv_heads", "head_dim", "n"))
    g = hq // h
    rk, rv = (r.double() for r in st["rots"])
    lens = st["lens"].tolist()
    if case["op"] == "read":
        out = {k: torch.zeros(b, n, h, d, dtype=torch.float64, device="cuda") for k in "kv"}
        for i in range(b):
            first = int(st["start"][i])
            for j in range(h):
                for role, name in enumerate("kv"):
                    x = _exact_rows(case, st["lay"], st["cache"], role, i, j, lens[i])[first:first + n]
                    out[name][i, :len(x), j] = torch.einsum("tj,ij->ti", x, (rk, rv)[role])
        return out
    if case["op"] == "extend":
        out = torch.zeros(b, n, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(b, n, hq, dtype=torch.float64, device="cuda")
        for i in range(b):
            m = int(st["q_lens"][i])
            hidden = torch.ones(m, lens[i], dtype=torch.bool, device="cuda").triu(lens[i] - m + 1)
            for j in range(h):
                k = torch.einsum("tj,ij->ti", _exact_rows(case, st["lay"], st["cache"], 0, i, j, lens[i]), rk)
                v = torch.einsum("tj,ij->ti", _exact_rows(case, st["lay"], st["cache"], 1, i, j, lens[i]), rv)
                for e in range(j * g, j * g + g):
                    s = (st["q"][i, :m, e].double() @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                    lse[i, :m, e] = torch.logsumexp(s, -1)
                    out[i, :m, e] = torch.softmax(s, -1) @ v
        return {"out": out, "lse": lse}
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(b, hq, dtype=torch.float64, device="cuda")
    for j in range(h):
        pk = torch.einsum("tj,ij->ti", _exact_rows(case, st["prefix_lay"], st["prefix_cache"], 0, 0, j, case["prefix"]), rk)
        pv = torch.einsum("tj,ij->ti", _exact_rows(case, st["prefix_lay"], st["prefix_cache"], 1, 0, j, case["prefix"]), rv)
        for i in range(b):
            k = torch.einsum("tj,ij->ti", _exact_rows(case, st["lay"], st["cache"], 0, i, j, lens[i]), rk)
            v = torch.einsum("tj,ij->ti", _exact_rows(case, st["lay"], st["cache"], 1, i, j, lens[i]), rv)
            q = st["q"][i, j * g:j * g + g].double()
            s = torch.cat((q @ pk.T, q @ k.T), -1) / math.sqrt(d)
            p = torch.softmax(s, -1)
            out[i, j * g:j * g + g] = p[:, :case["prefix"]] @ pv + p[:, case["prefix"]:] @ v
            lse[i, j * g:j * g + g] = torch.logsumexp(s, -1)
    return {"out": out, "lse": lse}
