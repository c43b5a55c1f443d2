"""Cases of the operators that stand before and behind the INT2 cache, with their plain forms.

Five operators (layout and quantiser: include/oscar_kv.h):

* ``rope``    qk_norm_rope: root-mean-square norm of every query and key head, then the position rotation;
* ``prompt``  attn_prompt: causal attention of packed prompts over their own, unquantised K and V;
* ``append``  kv_append_packed: the rows of packed prompts into the cache;
* ``mass``    attn_mass: the attention weight that every cached position receives, added up;
* ``evict``   kv_evict: the positions of largest weight and the windows into another, shorter cache.

``own`` false computes them with elementary torch operations in 32 bits; ``own`` true calls the library.  ``exact``
computes them again in 64 bits.
"""
import math

import numpy as np
import torch

own = False

LM_RATIO = float(np.float32(1.16))  # gap ratio of the Lloyd-Max levels
V_BF16, LLOYD_MAX, HADAMARD, IN_FP32, OUT_FP32 = 16, 32, 8, 2, 4
MODES = {"int2": 0, "v_bf16": V_BF16, "lloyd_max": LLOYD_MAX}
K_CLIP, V_CLIP = 0.96, 0.92
EPS = 1e-6
SPARE = 3  # rows behind the last sequence of a packed batch


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, q_heads=32, kv_heads=8, head_dim=128, sink=64, recent=256, length=1024, n=1,
             ragged=False, mode="int2", hadamard=False, fp32=False, rot_dim=128, interleaved=False, far=0, keep=0)
    c.update(kw)
    return c


def listed():
    return [
        # rope: the tokens of one decode step behind 128K of context (latency only)
        _case("rope-step", "rope", length=8, far=131072),
        # rope: a chunk of 16384 prompt tokens out of the fused projection, 64 query heads
        _case("rope-prompt", "rope", q_heads=64, length=16384),
        # prompt: three short prompts of odd lengths in float32, as a check or a small model runs them (latency)
        _case("prompt-fp32", "prompt", batch=3, q_heads=24, length=333, ragged=True, fp32=True),
        # prompt: a serving batch of eight ragged prompts
        _case("prompt-batch", "prompt", batch=8, length=4096, ragged=True),
        # prompt: one long prompt
        _case("prompt-long", "prompt", length=16384),
        # prompt: head_dim 512
        _case("prompt-hd512", "prompt", batch=4, q_heads=16, head_dim=512, length=2048, ragged=True),
        # append: four ragged prompts of up to 8192 tokens into one cache
        _case("append-batch", "append", batch=4, length=8192, ragged=True, hadamard=True),
        # append: short prompts at head_dim 512, Lloyd-Max levels
        _case("append-hd512", "append", batch=5, q_heads=16, head_dim=512, length=700, ragged=True, hadamard=True,
              mode="lloyd_max"),
        # mass: one decode step of 32 sequences with 32K of context
        _case("mass-step", "mass", batch=32, length=32768, ragged=True),
        # mass: the last 32 tokens of a prompt choose what is kept of it, 64 query heads
        _case("mass-window", "mass", q_heads=64, length=16384, n=32),
        # evict: 32 sequences of 32K down to 4096 positions and the windows
        _case("evict-batch", "evict", batch=32, length=32768, ragged=True, keep=4096),
        # evict: one sequence at head_dim 512, values kept BF16
        _case("evict-hd512", "evict", q_heads=16, head_dim=512, sink=512, recent=2048, length=65536, keep=10001,
              mode="v_bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "append", "mass", "evict"])
    head_dim = rng.choice([128, 128, 128, 256, 512])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    kw = dict(head_dim=head_dim, kv_heads=kv_heads, q_heads=kv_heads * rng.randint(1, 8),
              sink=rng.choice([0, 7, 64, 512]), recent=rng.choice([0, 31, 256, 2048]), ragged=rng.random() < 0.6,
              mode=rng.choice(["int2", "int2", "v_bf16", "lloyd_max"]), hadamard=rng.random() < 0.2)
    if op == "rope":
        kw["length"] = _log(rng, 1, 16384 * 128 // head_dim)
        kw["rot_dim"] = rng.choice([head_dim, head_dim, 64, 16])
        kw["interleaved"] = rng.random() < 0.3
        kw["far"] = rng.choice([0, 1000, 1000003])
        kw["fp32"] = rng.random() < 0.25
    elif op == "prompt":
        kw["fp32"] = rng.random() < 0.15
        kw["batch"] = _log(rng, 1, 16)
        most = math.isqrt(int((1.5e8 if kw["fp32"] else 2.0e9) // (kw["batch"] * kw["q_heads"] * (head_dim // 128))))
        kw["length"] = _log(rng, 1, max(2, min(8192, most)))
    elif op == "append":
        kw["hadamard"] = True
        kw["batch"] = _log(rng, 1, 8)
        kw["length"] = _log(rng, 1, 8192 * 128 // head_dim // kw["batch"])
    elif op == "mass":
        kw["batch"] = _log(rng, 1, 16)
        kw["n"] = rng.choice([1, 1, 1, _log(rng, 2, 64)])
        most = int(1.0e9 // (kw["batch"] * kw["n"] * kw["q_heads"] * (head_dim // 128)))
        kw["length"] = max(kw["n"], _log(rng, 16, max(17, min(32768, most))))
    else:
        kw["batch"] = _log(rng, 1, 16)
        kw["length"] = _log(rng, 64, 32768 * 128 // head_dim)
        kw["keep"] = rng.choice([0, 1, _log(rng, 1, kw["length"]), kw["length"]])
    c = _case("", op, **kw)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------
# the cache
# ------------------------------------------------------------------------------------------------
def _align(x):
    return (x + 255) // 256 * 256


def _layout(case, capacity):
    """Sizes of a one-layer cache (kv_layout_query's formulas)."""
    b, h, d, s, w = case["batch"], case["kv_heads"], case["head_dim"], case["sink"], case["recent"]
    ncap = -(-max(capacity - s, 0) // 64) * 64
    sink, ring = _align(b * h * s * d * 2), _align(b * h * w * d * 2)
    codes, sz = _align(b * h * ncap * (d // 4)), _align(b * h * ncap * (d // 128) * 4)
    role = sink + ring + codes + sz
    v_role = _align(b * h * capacity * d * 2) if case["mode"] == "v_bf16" else role
    return dict(ncap=ncap, capacity=capacity, at=(sink, sink + ring, sink + ring + codes), role=role, total=role + v_role)


def _view(lay, case, cache, role, region):
    """One region of a role as a typed tensor that shares the cache's memory."""
    b, h, d = case["batch"], case["kv_heads"], case["head_dim"]
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


def _regions(case, role):
    return ("full",) if role and case["mode"] == "v_bf16" else ("sink", "ring", "codes", "sz")


def _whole(case, lay, cache):
    """The cache as a call's output: its BF16 rows, scales and zeros, and the code words (2-bit codes that the operators
    place or move: they have to be the same ones, so they are compared as the whole numbers that they are)."""
    return {"kv"[role] + "_" + region: _view(lay, case, cache, role, region)
            for role in (0, 1) for region in _regions(case, role)}


def _hadamard(d):
    """The in-quant Hadamard without its factor: block-diagonal, order 128, entries of +-1."""
    i = np.arange(128)
    par = np.array([[bin(x & y).count("1") & 1 for y in i] for x in i])
    return np.kron(np.eye(d // 128), np.where(par, -1.0, 1.0))


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _activations(shape, gen):
    """N(0, 1) rows with a few outlier channels (two per hundred, eight times larger with heavy tails), float32."""
    x = torch.randn(shape, generator=gen, device="cuda")
    ch = torch.arange(5, shape[-1], 47, device="cuda")
    z = torch.randn((4,) + tuple(shape[:-1]) + (len(ch),), generator=gen, device="cuda")
    x[..., ch] += 2.0 * z[0] / torch.sqrt(z[1:].square().mean(0) + 1e-3)
    return x


def _lengths(case, rng):
    top = case["length"]
    lens = np.full(case["batch"], top)
    if case["ragged"] and case["batch"] > 1:
        lens[1:] = np.maximum(1, (top * rng.uniform(0.25, 1.0, case["batch"] - 1)).astype(int))
    return lens


def _packed(case, rng):
    """Lengths of a packed batch: the seed gives their order, the case their sum."""
    lens = _lengths(case, np.random.default_rng(case["length"]))
    return rng.permutation(lens)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rotation(case, seed):
    d = case["head_dim"]
    if case["hadamard"]:
        return torch.from_numpy((_hadamard(d) / math.sqrt(128.0)).astype(np.float32)).cuda()
    return torch.from_numpy(np.linalg.qr(np.random.default_rng(seed).standard_normal((d, d)))[0].astype(np.float32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng([seed, 1])
    st = dict(case=case, scale=1.0 / math.sqrt(case["head_dim"]))
    {"rope": _prepare_rope, "prompt": _prepare_prompt, "append": _prepare_append, "mass": _prepare_mass,
     "evict": _prepare_evict}[case["op"]](case, st, seed, gen, rng)
    return st


def _prepare_rope(case, st, seed, gen, rng):
    n, hq, h, d = case["length"], case["q_heads"], case["kv_heads"], case["head_dim"]
    kind = torch.float32 if case["fp32"] else torch.bfloat16
    fused = torch.randn(n, (hq + 2 * h) * d, generator=gen, device="cuda").mul_(2.0).to(kind)  # the projection's output
    st["q"] = fused[:, :hq * d].view(n, hq, d)
    st["k"] = fused[:, hq * d:(hq + h) * d].view(n, h, d)
    st["qw"], st["kw"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
    st["inv_freq"] = 1e6 ** (-torch.arange(0, case["rot_dim"], 2, device="cuda", dtype=torch.float32) / case["rot_dim"])
    first = case["far"] + int(rng.integers(0, 100))
    st["positions"] = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
    st["q_out"], st["k_out"] = (torch.empty(n, x, d, dtype=kind, device="cuda") for x in (hq, h))


def _prepare_prompt(case, st, seed, gen, rng):
    lens = _packed(case, rng)
    n, hq, h, d = int(lens.sum()) + SPARE, case["q_heads"], case["kv_heads"], case["head_dim"]
    kind = torch.float32 if case["fp32"] else torch.bfloat16
    st["cu"] = _int32(np.concatenate(([0], np.cumsum(lens))))
    st["q"], st["k"], st["v"] = (_activations((n, x, d), gen).to(kind) for x in (hq, h, h))
    st["out"] = torch.zeros(n, hq, d, dtype=kind, device="cuda")
    st["lse"] = torch.zeros(n, hq, device="cuda")


def _prepare_append(case, st, seed, gen, rng):
    lens = _packed(case, rng)
    n, h, d = int(lens.sum()) + SPARE, case["kv_heads"], case["head_dim"]
    st["cu"] = _int32(np.concatenate(([0], np.cumsum(lens))))
    st["start"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
    # rows on a grid of 2^-10: the +-1 sums of the rotation are then exact in 32 bits in any order, and no code is a matter
    # of rounding (whole numbers have to be equal)
    st["k"], st["v"] = ((_activations((n, h, d), gen).clamp_(-60, 60) * 1024).round_().div_(1024).to(torch.bfloat16)
                        .float().mul_(1024).round_().div_(1024).to(torch.bfloat16) for _ in range(2))
    st["lay"] = _layout(case, case["length"] + 16)
    st["signs"] = torch.from_numpy(_hadamard(128).astype(np.float32)).cuda()
    st["cache"] = torch.zeros(st["lay"]["total"], dtype=torch.uint8, device="cuda")


def _random_cache(case, lay, gen):
    """A cache as appends leave it, drawn directly: codes, scales of about a third of a row's range, zeros at its low end."""
    cache = torch.zeros(lay["total"], dtype=torch.uint8, device="cuda")
    for role in (0, 1):
        for region in _regions(case, role):
            v = _view(lay, case, cache, role, region)
            if region == "codes":
                v.random_(-2**31, 2**31 - 1, generator=gen)
            elif region == "sz":
                s = 1.4 * torch.exp(0.25 * torch.randn(v.shape[:-1], generator=gen, device="cuda"))
                v[..., 0] = s
                v[..., 1] = -1.5 * s * (1 + 0.05 * torch.randn(s.shape, generator=gen, device="cuda"))
            else:
                v.normal_(generator=gen)
    return cache


def _prepare_mass(case, st, seed, gen, rng):
    b, hq, h, d, n, top = (case[k] for k in ("batch", "q_heads", "kv_heads", "head_dim", "n", "length"))
    lens = _lengths(case, rng)
    st["lens"], st["q_lens"] = _int32(lens), _int32(np.minimum(lens, n))
    st["lay"] = _layout(case, top + 16)
    st["cache"] = _random_cache(case, st["lay"], gen)
    st["rot"] = _rotation(case, seed)
    st["q"] = _activations((b, n, hq, d), gen).to(torch.bfloat16)
    st["mass"] = 0.01 * torch.rand(b, h, top + 16, generator=gen, device="cuda")
    st["out"] = torch.zeros_like(st["mass"])
    s, _ = _scores(st)
    st["lse"] = torch.logsumexp(s, -1).view(b, h, hq // h, n).permute(0, 3, 1, 2).reshape(b, n, hq).contiguous()


def _prepare_evict(case, st, seed, gen, rng):
    b, h, top, s, w = (case[k] for k in ("batch", "kv_heads", "length", "sink", "recent"))
    st["lens"] = _int32(_lengths(case, rng))
    st["lay"] = _layout(case, top + 16)
    st["out_lay"] = _layout(case, min(top, s + w + case["keep"]) + 16)
    st["cache"] = _random_cache(case, st["lay"], gen)
    # heavy-tailed weights on a grid: many small ones are equal
    x = torch.exp(2.0 * torch.randn(b, h, top + 16, generator=gen, device="cuda"))
    st["mass"] = (x * 256).round_().div_(256)
    st["out_cache"] = torch.zeros(st["out_lay"]["total"], dtype=torch.uint8, device="cuda")
    st["out_mass"] = torch.zeros(b, h, st["out_lay"]["capacity"], device="cuda")
    st["kept"] = torch.zeros(b, h, case["keep"], dtype=torch.int32, device="cuda")
    st["new_lens"] = torch.zeros(b, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _plain_rope(st):
    case = st["case"]
    r = case["rot_dim"]
    turn = st["positions"].double()[:, None] * st["inv_freq"].double()
    c, s = (f(turn).float()[:, None] for f in (torch.cos, torch.sin))

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if case["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
        a, b = a * c - b * s, b * c + a * s
        y = torch.cat((torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1), y[..., r:]), -1)
        return y.to(x.dtype)

    return {"q": one(st["q"], st["qw"]), "k": one(st["k"], st["kw"])}


def _places(cu, n):
    """Sequence and token of every packed row, and whether it belongs to one."""
    at = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu[1:].long(), at, right=True)
    ok = b < len(cu) - 1
    b = b.clamp(max=len(cu) - 2)
    return b, torch.where(ok, at - cu[b], 0), ok


def _plain_prompt(st):
    case, cu = st["case"], st["cu"].long()
    n, hq, d = st["q"].shape
    b, h, top = case["batch"], case["kv_heads"], case["length"]
    at = (cu[:-1, None] + torch.arange(top, device="cuda")).clamp(max=n - 1)  # [b][top]
    q, k, v = (st[x][at].float().transpose(1, 2) for x in "qkv")  # [b][heads][top][d]
    s = q.reshape(b, h, -1, d) @ k.transpose(2, 3)
    s = s.mul_(st["scale"]).view(b, h, hq // h, top, top)
    s.masked_fill_(torch.ones(top, top, dtype=torch.bool, device="cuda").triu_(1), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(b, h, -1, top) @ v).view(b, hq, top, d) / l.view(b, hq, top, 1)
    lse = (m + torch.log(l)).view(b, hq, top)
    i, t, ok = _places(cu, n)
    return {"out": torch.where(ok[:, None, None], o[i, :, t].to(st["out"].dtype), st["out"]),
            "lse": torch.where(ok[:, None], lse[i, :, t], st["lse"])}


def _plain_append(st):
    case, lay, cu = st["case"], st["lay"], st["cu"].long()
    n, top = st["k"].shape[0], case["length"]
    lens = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + torch.arange(top, device="cuda")).clamp(max=n - 1)
    live = (torch.arange(top, device="cuda") < lens[:, None])[:, None, :, None]
    out = torch.zeros_like(st["cache"])
    _append_role(case, lay, out, 0, st["k"][at].float().transpose(1, 2), st["signs"], lens, live, K_CLIP)
    _append_role(case, lay, out, 1, st["v"][at].float().transpose(1, 2), st["signs"], lens, live, V_CLIP)
    return _whole(case, lay, out)


def _append_role(case, lay, cache, role, x, signs, lens, live, clip):
    b, h, top, d = x.shape
    s, w = case["sink"], case["recent"]
    lm = case["mode"] == "lloyd_max"
    r = ((x.view(b, h, top, d // 128, 128) @ signs) * 0.08838834764831845).view(b, h, top, d)
    wide = r.to(torch.bfloat16)
    if role and case["mode"] == "v_bf16":
        _view(lay, case, cache, role, "full")[:, :, :top] = torch.where(live, wide, 0)
        return
    _view(lay, case, cache, role, "sink")[:, :, :min(s, top)] = torch.where(live, wide, 0)[:, :, :s]
    last = lens[:, None] - w + torch.arange(w, device="cuda")
    rows = torch.gather(wide, 2, last.clamp(min=0).view(b, 1, w, 1).expand(b, h, w, d))
    slot = (last % max(w, 1)).view(b, 1, w, 1).expand(b, h, w, d)
    ring = _view(lay, case, cache, role, "ring")
    ring.scatter_(2, slot, torch.where((last >= 0).view(b, 1, w, 1), rows, 0))
    r = r[:, :, s:]
    rest = r.shape[2]
    a = r.abs().amax(-1, keepdim=True) * clip
    x = torch.maximum(torch.minimum(r, a), -a).view(b, h, rest, d // 128, 128)
    lo, hi = x.amin(-1), x.amax(-1)
    span = torch.tensor(2 * LM_RATIO + 1 if lm else 3.0, device="cuda")
    sc, ze = ((hi - lo) / span).half(), lo.half()
    y = (x - ze.float()[..., None]) * torch.where(sc > 0, 1 / sc.float(), 0)[..., None]
    if lm:
        high = torch.tensor(2 * LM_RATIO + 1 - LM_RATIO / 2, dtype=torch.float32, device="cuda")
        code = (y > LM_RATIO / 2).int() + (y > LM_RATIO + 0.5).int() + (y > high).int()
    else:
        code = y.round().clamp(0, 3).int()
    code = code.masked_fill(sc[..., None] == 0, 0)
    if role == 0:  # channel = 64 i + 8 p + 2 c + hi of each group: word 2 c + i, bit 2 p + 16 hi
        code = code.view(b, h, rest, d // 128, 2, 8, 4, 2).permute(0, 1, 2, 3, 6, 4, 7, 5)
    else:  # channel = 8 n + g: word g, bit 2 n
        code = code.view(b, h, rest, d // 128, 2, 8, 8).permute(0, 1, 2, 3, 6, 4, 5)
    word = (code.reshape(b, h, rest, d // 16, 16) << (2 * torch.arange(16, device="cuda", dtype=torch.int32))).sum(-1, dtype=torch.int32)
    written = live[:, :, s:]
    _view(lay, case, cache, role, "codes")[:, :, :rest] = torch.where(written, word, 0)
    _view(lay, case, cache, role, "sz")[:, :, :rest] = torch.where(written[..., None], torch.stack((sc, ze), -1), 0)


def _keys(case, lay, cache, lens, top):
    """Cached K rows [batch][kv_heads][top][head_dim] in 32 bits, rotated basis, as attention sees them."""
    b, h, d, s, w = case["batch"], case["kv_heads"], case["head_dim"], case["sink"], case["recent"]
    at = torch.arange(top, device="cuda")
    body = min(s, top)
    word = _view(lay, case, cache, 0, "codes")[:, :, :top - body]
    sz = _view(lay, case, cache, 0, "sz")[:, :, :top - body].float()
    code = (word[..., None] >> (2 * torch.arange(16, device="cuda", dtype=torch.int32))) & 3
    code = code.view(b, h, top - body, d // 128, 4, 2, 2, 8).permute(0, 1, 2, 3, 5, 7, 4, 6)
    level = code.reshape(b, h, top - body, d // 128, 128)
    if case["mode"] == "lloyd_max":
        level = torch.tensor([0.0, LM_RATIO, LM_RATIO + 1, 2 * LM_RATIO + 1], device="cuda")[level]
    x = (sz[..., 1:] + sz[..., :1] * level).view(b, h, top - body, d)
    if body:
        x = torch.cat((_view(lay, case, cache, 0, "sink")[:, :, :body].float(), x), 2)
    if w:
        ring = _view(lay, case, cache, 0, "ring")[:, :, at % w].float()
        recent = at >= torch.clamp(lens.view(b, 1) - w, min=s)
        x = torch.where(recent.view(b, 1, top, 1), ring, x)
    return x


def _scores(st):
    """Scaled scores [batch][kv_heads][G * n][length], -inf where a token does not see a position, and the tokens' own."""
    case, lens, qlens = st["case"], st["lens"].long(), st["q_lens"].long()
    b, n, hq, d = st["q"].shape
    h, top = case["kv_heads"], case["length"]
    q = (st["q"].float() @ st["rot"]).view(b, n, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    s = (q @ _keys(case, st["lay"], st["cache"], lens, top).transpose(2, 3)).mul_(st["scale"]).view(b, h, hq // h, n, top)
    t = torch.arange(n, device="cuda")
    last = torch.where(t < qlens.view(b, 1), (lens - qlens).view(b, 1) + t, -1)  # a query token's own position
    s.masked_fill_((torch.arange(top, device="cuda") > last[..., None])[:, None, None], -math.inf)
    return s.view(b, h, -1, top), last


def _plain_mass(st):
    case = st["case"]
    b, n, hq, _ = st["q"].shape
    h, top = case["kv_heads"], case["length"]
    s, last = _scores(st)
    lse = st["lse"].view(b, n, h, hq // h).permute(0, 2, 3, 1)
    lse = torch.where((last >= 0)[:, None, None], lse, 0).reshape(b, h, -1, 1)
    got = s.sub_(lse).exp_().sum(2)
    out = st["out"].clone()
    live = (torch.arange(top, device="cuda") < st["lens"].view(b, 1))[:, None]
    out[:, :, :top] = torch.where(live, st["mass"][:, :, :top] + got, out[:, :, :top])
    return {"mass": out}


def _plain_evict(st):
    case, lay, new = st["case"], st["lay"], st["out_lay"]
    b, h, d, s, w, top, keep = (case[k] for k in ("batch", "kv_heads", "head_dim", "sink", "recent", "length", "keep"))
    lens = st["lens"].long().view(b, 1, 1)
    at = torch.arange(top, device="cuda")
    end = torch.clamp(lens - w, min=s)  # the window's first position
    body = (at >= s) & (at < end)
    count = torch.clamp(torch.minimum(end, lens) - s, min=0)
    held = torch.clamp(count, max=keep)
    order = torch.sort(torch.where(body, st["mass"][:, :, :top], -1.0), dim=-1, descending=True, stable=True).indices[..., :keep]
    rank = torch.arange(order.shape[-1], device="cuda")
    kept = torch.sort(torch.where(rank < held, order, top), -1).values
    kept = torch.where(rank < held, kept, -1)
    kept = torch.cat((kept, torch.full((b, h, keep - kept.shape[-1]), -1, device="cuda")), -1)
    gone = count - held
    length = lens - gone
    # every position of the new cache and the one that it was
    cap = new["capacity"]
    p = torch.arange(cap, device="cuda").expand(b, h, cap)
    inside = (p >= s) & (p < s + held)
    there = torch.gather(torch.cat((kept, torch.zeros(b, h, 1, dtype=torch.long, device="cuda")), -1), 2,
                         (p - s).clamp(0, keep))
    old = torch.where(p < s, p, torch.where(inside, there, p + gone)).clamp(0, top - 1)
    live = p < length
    out = torch.zeros_like(st["out_cache"])
    take = lambda x, i, ok: torch.where(ok.reshape(ok.shape + (1,) * (x.dim() - 3)), torch.gather(  # noqa: E731
        x, 2, i.reshape(i.shape + (1,) * (x.dim() - 3)).expand(i.shape + x.shape[3:])), 0)
    for role in (0, 1):
        src = {r: _view(lay, case, st["cache"], role, r) for r in _regions(case, role)}
        dst = {r: _view(new, case, out, role, r) for r in _regions(case, role)}
        if "full" in src:
            dst["full"].copy_(take(src["full"], old, live))
            continue
        if s:
            dst["sink"].copy_(take(src["sink"], torch.arange(s, device="cuda").expand(b, h, s), torch.arange(s, device="cuda") < lens.expand(b, h, 1)))
        if w:
            now = (length - w + torch.arange(w, device="cuda")).expand(b, h, w)  # the window's new positions
            ok = now >= s
            rows = take(src["ring"], (now + gone) % w, ok)
            slot = (now % w)[..., None].expand(rows.shape)
            dst["ring"].scatter_(2, slot, rows)
        body_old, body_live = old[:, :, s:], live[:, :, s:]
        for r in ("codes", "sz"):
            dst[r][:, :, :cap - s].copy_(take(src[r], (body_old - s).clamp(min=0), body_live)) if cap > s else None
    mass = torch.where(live, torch.gather(st["mass"], 2, old), 0)
    res = {"mass": mass, "kept": kept.int(), "lens": length.view(b).int()}
    res.update(_whole(case, new, out))
    return res


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------
def _config(case, capacity, flags=0):
    from int2_kv_cache_append_gb300 import oscar_kv as K

    return K.KVConfig(1, case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"], case["sink"], case["recent"],
                      capacity, K_CLIP, V_CLIP, flags=MODES[case["mode"]] | (HADAMARD if case["hadamard"] else 0) | flags)


def _own(st):
    from int2_kv_cache_append_gb300 import oscar_kv as K

    case, op = st["case"], st["case"]["op"]
    if "cfg" not in st:  # what a program sets up once and keeps
        wide = IN_FP32 | OUT_FP32 if case["fp32"] else 0
        st["cfg"] = _config(case, st["lay"]["capacity"] if "lay" in st else max(1, case["length"]), wide)
        size = 0
        if op == "mass":
            size = K.attn_mass_workspace_bytes(st["cfg"], case["n"])
        elif op == "evict":
            st["out_cfg"] = _config(case, st["out_lay"]["capacity"])
            size = K.kv_evict_workspace_bytes(st["cfg"], case["keep"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        if op == "append":
            st["whole"] = _whole(case, st["lay"], st["cache"])
        elif op == "evict":
            st["whole"] = _whole(case, st["out_lay"], st["out_cache"])
    cfg = st["cfg"]
    if op == "rope":
        K.qk_norm_rope(cfg, st["q"], st["k"], st["qw"], st["kw"], st["positions"], st["inv_freq"], st["q_out"], st["k_out"],
                       eps=EPS, interleaved=case["interleaved"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if op == "prompt":
        K.attn_prompt(cfg, st["q"], st["k"], st["v"], st["cu"], st["out"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "append":
        K.kv_append_packed(cfg, st["cache"], 0, st["k"], st["v"], st["cu"], st["start"], None, None)
        return st["whole"]
    if op == "mass":
        K.attn_mass(cfg, st["cache"], 0, st["q"], st["lens"], None if case["hadamard"] else st["rot"], st["lse"], st["out"],
                    st["ws"], mass_in=st["mass"], q_lens=st["q_lens"], seq_len_hint=case["length"])
        return {"mass": st["out"]}
    K.kv_evict(cfg, st["cache"], 0, st["mass"], st["lens"], case["keep"], st["out_cfg"], st["out_cache"], 0, st["new_lens"],
               st["ws"], out_mass=st["out_mass"], kept=st["kept"])
    return {"mass": st["out_mass"], "kept": st["kept"], "lens": st["new_lens"], **st["whole"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "prompt": _plain_prompt, "append": _plain_append, "mass": _plain_mass,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def _role_bytes(case, role, tokens):
    """Bytes of one role's `tokens` cached tokens of one (sequence, KV head), as a reader takes them."""
    d = case["head_dim"]
    if role and case["mode"] == "v_bf16":
        return tokens * 2 * d
    wide = min(tokens, case["sink"] + case["recent"])
    return wide * 2 * d + (tokens - wide) * (d // 4 + d // 32)


def work(case):
    b, hq, h, d, n, top = (case[k] for k in ("batch", "q_heads", "kv_heads", "head_dim", "n", "length"))
    fill = 0.625 if case["ragged"] else 1.0  # mean length of the ragged sequences behind the first
    mean = top * (1 + (b - 1) * fill) / b
    wide = 4 if case["fp32"] else 2
    if case["op"] == "rope":
        return {"bytes": n_rope(case) * 2 * wide, "flops": 10 * n_rope(case)}
    if case["op"] == "prompt":
        square = top * top * (1 + (b - 1) * (0.4375 if case["ragged"] else 1.0))  # mean of the squared lengths
        return {"bytes": b * mean * ((2 * hq + 2 * h) * d * wide + 4 * hq), "flops": 2 * hq * d * (square + b * mean)}
    if case["op"] == "append":
        rows = b * h * mean
        copies = min(mean, case["sink"]) + min(mean, case["recent"])
        out = b * h * copies * 2 * d + max(0.0, rows - b * h * case["sink"]) * (d // 4 + d // 32)
        v_out = rows * 2 * d if case["mode"] == "v_bf16" else out
        return {"bytes": 2 * rows * d * 2 + out + v_out, "flops": 2 * rows * 14 * d}
    if case["op"] == "mass":
        m = min(n, mean)
        return {"bytes": b * h * (_role_bytes(case, 0, int(mean)) + 8 * mean) + b * m * hq * (2 * d + 4),
                "flops": 2 * hq * d * b * m * (mean - (m - 1) / 2)}
    kept = min(max(0.0, mean - case["sink"] - case["recent"]), case["keep"])
    moved = min(mean, case["sink"] + case["recent"])
    packed = d // 4 + d // 32
    role = kept * packed + moved * 2 * d + min(moved, case["recent"]) * packed
    v_role = (kept + moved) * 2 * d if case["mode"] == "v_bf16" else role
    return {"bytes": b * h * (4 * mean + 2 * (role + v_role) + 4 * (2 * kept + moved)), "flops": b * h * mean}


def n_rope(case):
    return case["length"] * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]


# ------------------------------------------------------------------------------------------------
# 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "evict":
        return None  # selects and moves: no output is a computed number
    st = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "append": _exact_append, "mass": _exact_mass}[case["op"]](case, st)


def _exact_rope(case, st):
    r = case["rot_dim"]
    turn = torch.outer(st["positions"].double(), st["inv_freq"].double())
    z = torch.polar(torch.ones_like(turn), turn)[:, None]
    out = {}
    for name in "qk":
        x = st[name].double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["head_dim"] + EPS) * st[name + "w"].double()
        y = x.clone()
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
            w = torch.complex(x[..., a], x[..., b]) * z[..., i]
            y[..., a], y[..., b] = w.real, w.imag
        out[name] = y
    return out


def _exact_prompt(case, st):
    n, hq, d = st["q"].shape
    g = hq // case["kv_heads"]
    cu = st["cu"].tolist()
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, hq, dtype=torch.float64, device="cuda")
    for i in range(case["batch"]):
        at = slice(cu[i], cu[i + 1])
        hidden = torch.ones(cu[i + 1] - cu[i], cu[i + 1] - cu[i], dtype=torch.bool, device="cuda").triu(1)
        for e in range(hq):
            s = (st["q"][at, e].double() @ st["k"][at, e // g].double().T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
            lse[at, e] = torch.logsumexp(s, -1)
            out[at, e] = torch.softmax(s, -1) @ st["v"][at, e // g].double()
    return {"out": out, "lse": lse}


def _exact_append(case, st):
    """The BF16 rows, scales and zeros; the code words have no value in 64 bits."""
    b, h, d, s, w = (case[k] for k in ("batch", "kv_heads", "head_dim", "sink", "recent"))
    lay, cu = st["lay"], st["cu"].tolist()
    rot = torch.from_numpy(_hadamard(d)).cuda() / math.sqrt(128.0)
    span = 2 * LM_RATIO + 1 if case["mode"] == "lloyd_max" else 3.0
    out = {}
    for role, name in enumerate("kv"):
        shapes = {r: _view(lay, case, st["cache"], role, r) for r in _regions(case, role)}
        got = {r: torch.zeros(x.shape, dtype=torch.float64, device="cuda") for r, x in shapes.items()}
        for i in range(b):
            x = torch.einsum("thc,cd->htd", st[name][cu[i]:cu[i + 1]].double(), rot)
            t = x.shape[1]
            if "full" in got:
                got["full"][i, :, :t] = x
                continue
            got["sink"][i, :, :min(s, t)] = x[:, :s]
            for p in range(max(0, t - w), t):
                got["ring"][i, :, p % w] = x[:, p]
            if t > s:
                lim = x[:, s:].abs().amax(-1, keepdim=True) * float(np.float32(V_CLIP if role else K_CLIP))
                y = x[:, s:].clamp(-lim, lim).reshape(h, t - s, d // 128, 128)
                got["sz"][i, :, :t - s, :, 0] = (y.amax(-1) - y.amin(-1)) / span
                got["sz"][i, :, :t - s, :, 1] = y.amin(-1)
        for r, x in got.items():
            out[name + "_" + r] = None if r == "codes" else x
    return out


def _exact_keys(case, lay, cache, i, head, length):
    """K rows [0, length) of one (sequence, KV head) in 64 bits, rotated basis: read byte by byte."""
    d, s, w, h = case["head_dim"], case["sink"], case["recent"], case["kv_heads"]
    unit = i * h + head

    def wide(offset, first, count):
        o = offset + first * d * 2
        return cache[o:o + count * d * 2].view(torch.bfloat16).view(count, d).double()

    x = torch.zeros(length, d, dtype=torch.float64, device="cuda")
    if length > s:
        rows = length - s
        o = lay["at"][1] + unit * lay["ncap"] * (d // 4)
        byte = cache[o:o + rows * (d // 4)].view(rows, d // 4).int()
        o = lay["at"][2] + unit * lay["ncap"] * (d // 32)
        sz = cache[o:o + rows * (d // 32)].view(torch.float16).view(rows, d // 128, 2).double()
        ch = np.arange(d)
        g, c = ch // 128, ch % 128
        word, bit = 8 * g + 2 * (c % 8 // 2) + c // 64, 2 * (c % 64 // 8) + 16 * (c % 2)
        level = (byte[:, torch.from_numpy(4 * word + bit // 8).cuda()] >> torch.from_numpy(bit % 8).int().cuda()) & 3
        if case["mode"] == "lloyd_max":
            level = torch.tensor([0.0, LM_RATIO, LM_RATIO + 1, 2 * LM_RATIO + 1], dtype=torch.float64, device="cuda")[level.long()]
        g = torch.from_numpy(g).cuda()
        x[s:] = sz[:, g, 1] + sz[:, g, 0] * level
    if s:
        x[:s] = wide(0, unit * s, min(s, length))
    first = max(s, length - w)
    if w and first < length:
        x[first:] = wide(lay["at"][0], unit * w, w)[torch.arange(first, length, device="cuda") % w]
    return x


def _exact_mass(case, st):
    b, hq, h, n = (case[k] for k in ("batch", "q_heads", "kv_heads", "n"))
    g, rot = hq // h, st["rot"].double()
    lens, qlens = st["lens"].tolist(), st["q_lens"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for i in range(b):
        m = qlens[i]
        hidden = torch.ones(m, lens[i], dtype=torch.bool, device="cuda").triu(lens[i] - m + 1)
        for j in range(h):
            k = _exact_keys(case, st["lay"], st["cache"], i, j, lens[i])
            got = st["mass"][i, j, :lens[i]].double()
            for e in range(j * g, j * g + g):
                s = (st["q"][i, :m, e].double() @ rot @ k.T / math.sqrt(case["head_dim"])).masked_fill_(hidden, -math.inf)
                got = got + torch.exp(s - st["lse"][i, :m, e, None].double()).sum(0)
            out[i, j, :lens[i]] = got
    return {"mass": out}
