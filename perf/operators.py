"""Cases that time the operators around the attention kernels: the per-head
norm with rotation that makes queries and keys, the quantised K/V cache, and
decoding over it with and without a prefix that the whole batch shares.

`run` computes an operator in elementary torch operations, or, where `own` is
true, through the framework's entry points.
"""
import math

import torch

own = False

FP8_MAX, INT8_MAX = 448.0, 127.0
MIN_SCALE = 2.0 ** -120


def listed():
    return [
        # q and k of one Llama-2-7B layer, a training step: forward and backward, the projections' token-major layout
        dict(name="rope_train_7b", op="rope", B=8, N=2048, Hq=32, Hkv=32, D=128, rot=128, interleaved=False,
             train=True, wbf16=False, far=0),
        # grouped heads at an odd length, rotation of half the head in pairs (2i, 2i + 1), bf16 weights
        dict(name="rope_train_d64", op="rope", B=3, N=1237, Hq=12, Hkv=4, D=64, rot=32, interleaved=True, train=True,
             wbf16=True, far=0),
        # one new token of each of 8 sequences, far into a long context
        dict(name="rope_token", op="rope", B=8, N=1, Hq=64, Hkv=8, D=128, rot=128, interleaved=False, train=False,
             wbf16=True, far=1000000),
        # a prompt written into an 8-bit cache, and the history read back for the next chunk
        dict(name="cache_prompt_e4m3", op="cache", fmt="e4m3", B=8, Hkv=32, N=2048, capacity=4096, D=128, hist=1500),
        # a few tokens behind histories of other lengths
        dict(name="cache_chunk_int8", op="cache", fmt="int8", B=5, Hkv=8, N=37, capacity=1000, D=128, hist=700),
        # one token for each of 4 short sequences: the smallest call
        dict(name="cache_token_bf16", op="cache", fmt="bf16", B=4, Hkv=2, N=1, capacity=64, D=64, hist=60),
        # one new token of a short conversation: latency
        dict(name="decode_short_e4m3", op="decode", fmt="e4m3", B=1, Hq=32, Hkv=32, D=128, Nq=1, capacity=1024,
             len_min=513, len_max=513, prefix=0),
        # a 32K cache of a Llama-2-70B shaped layer at 8 bits
        dict(name="decode_70b_e4m3", op="decode", fmt="e4m3", B=8, Hq=64, Hkv=8, D=128, Nq=1, capacity=32768,
             len_min=32700, len_max=32768, prefix=0),
        # many sequences of very different lengths, three drafted tokens each
        dict(name="decode_ragged_int8", op="decode", fmt="int8", B=48, Hq=16, Hkv=4, D=128, Nq=3, capacity=8192,
             len_min=5, len_max=8100, prefix=0),
        # smaller heads, unquantised
        dict(name="decode_ragged_bf16", op="decode", fmt="bf16", B=13, Hq=12, Hkv=12, D=64, Nq=1, capacity=5000,
             len_min=1, len_max=4999, prefix=0),
        # 4 sequences behind one instruction text
        dict(name="prefix_small_bf16", op="decode", fmt="bf16", B=4, Hq=32, Hkv=8, D=128, Nq=1, capacity=256,
             len_min=1, len_max=130, prefix=1000),
        # 64 sequences behind one long document, 8-bit caches of their own
        dict(name="prefix_70b_e4m3", op="decode", fmt="e4m3", B=64, Hq=64, Hkv=8, D=128, Nq=1, capacity=1024,
             len_min=1, len_max=1000, prefix=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "decode", "prefix"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 32])
    fmt = rng.choice(["bf16", "e4m3", "int8"])
    if op == "rope":
        Hq = Hkv * rng.choice([1, 2, 4])
        train = rng.random() < 0.7
        rows = 1 << 20
        N = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, rows // (N * (Hq + Hkv)))))
        return dict(op="rope", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([16, 32, 48, 64, D]),
                    interleaved=rng.random() < 0.5, train=train, wbf16=rng.random() < 0.5,
                    far=rng.choice([0, 4096, 1000000]))
    if op == "cache":
        capacity = 4 * _log(rng, 4, 2048)
        N = _log(rng, 1, min(capacity, 2048))
        B = _log(rng, 1, max(1, min(64, (1 << 20) // (capacity * Hkv))))
        return dict(op="cache", fmt=fmt, B=B, Hkv=Hkv, N=N, capacity=capacity, D=D,
                    hist=rng.randint(0, capacity - N))
    G = rng.choice([1, 2, 4, 5, 8])
    Nq = rng.choice([1, 1, 1, 2, 4])
    if op == "decode":
        capacity = 4 * _log(rng, 8, 8192)
        B = _log(rng, 1, max(1, min(64, (1 << 21) // (capacity * Hkv))))
        hi = rng.randint(min(capacity, max(Nq, capacity // 2)), capacity)
        return dict(op="decode", fmt=fmt, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, Nq=Nq, capacity=capacity,
                    len_min=rng.choice([min(Nq, hi), hi]), len_max=hi, prefix=0)
    B = _log(rng, 2, 64)
    prefix = _log(rng, 64, max(65, min(32768, (1 << 27) // (B * G * Nq * Hkv))))
    capacity = 4 * _log(rng, 4, max(5, min(256, (1 << 19) // (4 * B * Hkv))))
    return dict(op="decode", fmt=fmt, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, Nq=Nq, capacity=capacity,
                len_min=min(Nq, capacity), len_max=rng.randint(min(Nq, capacity), capacity), prefix=prefix)


def _lens(case):
    """Lengths spread over [len_min, len_max], the longest among them."""
    lo, hi, B = case["len_min"], case["len_max"], case["B"]
    return [hi - int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(B)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _caches(g, case):
    """A cache as earlier writes left it, every slot of it: codes and their scales."""
    B, H, C, D, fmt = case["B"], case["Hkv"], case["capacity"], case["D"], case["fmt"]
    out = []
    for _ in range(2):
        x = _randn(g, B, H, C, D)
        if fmt == "bf16":
            out += [x.to(torch.bfloat16), None]
        elif fmt == "e4m3":
            out += [(x * 100).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn),
                    torch.exp2(torch.randint(-8, -5, (B, H, C), generator=g, device="cuda").float())]
        else:
            out += [(x * 40).round_().clamp_(-127, 127).to(torch.int8), 0.02 + 0.01 * _randn(g, B, H, C).abs()]
    return dict(zip(("kc", "ks", "vc", "vs"), out))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "rope":
        B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
        # the packed output of the projection, [B, N, Hq + 2 Hkv, D]; q and k are views of it
        qkv = _randn(g, B, N, Hq + 2 * Hkv, D).to(torch.bfloat16)
        s["q"], s["k"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        wt = torch.bfloat16 if case["wbf16"] else torch.float32
        s["qw"], s["kw"] = ((1 + 0.2 * _randn(g, D)).to(wt) for _ in range(2))
        i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2 * i / max(1, case["rot"]))).float()
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["pos"] = (first + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        if case["train"]:
            s["dq"] = _randn(g, B, Hq, N, D).to(torch.bfloat16)
            s["dk"] = _randn(g, B, Hkv, N, D).to(torch.bfloat16)
        return s
    s.update(_caches(g, case))
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    if case["op"] == "cache":
        N = case["N"]
        s["k"] = _randn(g, B, Hkv, N, D).to(torch.bfloat16)                       # as the rotation leaves it
        s["v"] = _randn(g, B, N, Hkv, D).to(torch.bfloat16).transpose(1, 2)       # as the projection leaves it
        start = [case["hist"] - (case["hist"] * b) // (2 * B) for b in range(B)]
        s["start"] = torch.tensor(start, device="cuda", dtype=torch.int32)
        s["lens"] = s["start"] + N
        s["n"] = case["hist"] + N
        return s
    s["q"] = _randn(g, B, case["Hq"], case["Nq"], D).to(torch.bfloat16)
    s["lens"] = torch.tensor(_lens(case), device="cuda", dtype=torch.int32)
    if case["prefix"]:
        s["pk"] = _randn(g, Hkv, case["prefix"], D).to(torch.bfloat16)
        s["pv"] = _randn(g, Hkv, case["prefix"], D).to(torch.bfloat16)
    return s


# ---- plain forms

def _turn(x, cos, sin, rot, interleaved):
    """x with its first `rot` values of each row turned in pairs by the angles' cos and sin."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _angles(s):
    a = s["pos"].double()[:, None, :, None] * s["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def _norm_turn(x, w, cos, sin, case):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return _turn(x * r * w.float(), cos, sin, case["rot"], case["interleaved"]).to(torch.bfloat16).contiguous()


def _norm_turn_bwd(dy, x, w, cos, sin, case):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    xh = x * r
    g = _turn(dy.float(), cos, -sin, case["rot"], case["interleaved"])
    dw = (g * xh).sum((0, 1, 2))
    h = g * w.float()
    return (r * (h - xh * (h * xh).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _quantise(x, fmt):
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "e4m3":
        m, e = torch.frexp(amax)                    # amax = m 2^e, m in [1/2, 1); 448 = (7/8) 2^9
        scale = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875).int()).clamp(min=-120))
        return (x / scale).to(torch.float8_e4m3fn), scale[..., 0]
    scale = (amax / INT8_MAX).clamp(min=MIN_SCALE)
    return (x / scale).round().to(torch.int8), scale[..., 0]


def _values(codes, scale):
    return codes.float() if scale is None else codes.float() * scale[..., None]


def _plain_cache(s):
    case = s["case"]
    B, H, N = case["B"], case["Hkv"], case["N"]
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(H, device="cuda")[None, :, None]
    slot = (s["start"].long()[:, None] + torch.arange(N, device="cuda"))[:, None, :]
    seen = (torch.arange(s["n"], device="cuda") < s["lens"][:, None])[:, None, :, None]

    def one(x, cache, scale):
        if scale is None:
            cache[b, h, slot] = x
        else:
            codes, new = _quantise(x, case["fmt"])
            cache.view(torch.uint8)[b, h, slot] = codes.view(torch.uint8)
            scale[b, h, slot] = new
        back = _values(cache[:, :, :s["n"]], None if scale is None else scale[:, :, :s["n"]])
        return torch.where(seen, back, torch.zeros_like(back)).to(torch.bfloat16)

    return one(s["k"], s["kc"], s["ks"]), one(s["v"], s["vc"], s["vs"])


def _plain_decode(s):
    case = s["case"]
    B, Hq, Hkv, D, Nq, C = (case[k] for k in ("B", "Hq", "Hkv", "D", "Nq", "capacity"))
    q = s["q"].float().view(B, Hkv, -1, D) * D ** -0.5                             # rows (head of the group, query)
    at = s["lens"][:, None] - Nq + torch.arange(Nq, device="cuda")                 # slot of each query
    hidden = torch.arange(C, device="cuda") > at.repeat(1, Hq // Hkv)[..., None]   # [B, rows, C]
    sc = (q @ _values(s["kc"], s["ks"]).transpose(-1, -2)).masked_fill(hidden[:, None], -math.inf)
    if case["prefix"]:
        sc = torch.cat([torch.einsum("bhrd,hnd->bhrn", q, s["pk"].float()), sc], -1)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    p = p / l
    o = p[..., case["prefix"]:] @ _values(s["vc"], s["vs"])
    if case["prefix"]:
        o = o + torch.einsum("bhrn,hnd->bhrd", p[..., :case["prefix"]], s["pv"].float())
    return o.view(B, Hq, Nq, D).to(torch.bfloat16), (m + l.log()).view(B, Hq, Nq)


def _plain(s):
    case = s["case"]
    if case["op"] == "rope":
        cos, sin = _angles(s)
        out = [_norm_turn(s["q"], s["qw"], cos, sin, case), _norm_turn(s["k"], s["kw"], cos, sin, case)]
        if case["train"]:
            dq, dqw = _norm_turn_bwd(s["dq"], s["q"], s["qw"], cos, sin, case)
            dk, dkw = _norm_turn_bwd(s["dk"], s["k"], s["kw"], cos, sin, case)
            out += [dq, dk, dqw, dkw]
        return out
    return _plain_cache(s) if case["op"] == "cache" else _plain_decode(s)


# ---- the framework's entry points

def _framework(s):
    from tiled_attention_16_b200 import cache, rope
    case = s["case"]
    if case["op"] == "rope":
        kw = dict(positions=s["pos"], interleaved=case["interleaved"])
        out = list(rope.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["inv_freq"], **kw))
        if case["train"]:
            out += rope.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["inv_freq"], **kw)
        return out
    if case["op"] == "cache":
        cache.cache_write(s["k"], s["v"], s["kc"], s["vc"], s["start"], k_scale=s["ks"], v_scale=s["vs"])
        return cache.cache_read(s["kc"], s["vc"], s["n"], lens=s["lens"], k_scale=s["ks"], v_scale=s["vs"])
    return cache.decode_cache(s["q"], s["kc"], s["vc"], s["lens"], k_scale=s["ks"], v_scale=s["vs"],
                              prefix_k=s.get("pk"), prefix_v=s.get("pv"))


def run(state):
    return _framework(state) if own else _plain(state)


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        n = case["B"] * case["N"] * (case["Hq"] + case["Hkv"]) * D
        return dict(bytes=(8 if case["train"] else 4) * n, flops=(24 if case["train"] else 9) * n)
    size = 2 if case["fmt"] == "bf16" else 1
    row = D * size + (0 if size == 2 else 4)                     # one cached row of K or of V
    if case["op"] == "cache":
        new = 2 * case["B"] * case["Hkv"] * case["N"]            # rows written
        starts = [case["hist"] - (case["hist"] * b) // (2 * case["B"]) for b in range(case["B"])]
        old = 2 * case["Hkv"] * sum(starts)                      # rows read that were there before
        out = 2 * case["B"] * case["Hkv"] * (case["hist"] + case["N"])
        return dict(bytes=new * (2 * D + row) + old * row + out * 2 * D, flops=3 * new * D)
    keys, heads = sum(_lens(case)), case["Hq"] * case["Nq"]
    byte = 2 * case["Hkv"] * (keys * row + case["prefix"] * 2 * D) + case["B"] * heads * (4 * D + 4)
    return dict(bytes=byte, flops=4 * D * heads * (keys + case["B"] * case["prefix"]))


# ---- 64 bits, from the definitions

def _exact_rope(s):
    case = s["case"]
    D, rot, half = case["D"], case["rot"], case["rot"] // 2
    # the turn as a matrix product: column j of a row gets x[j] cos + sign[j] x[partner[j]] sin
    j = torch.arange(D, device="cuda")
    if case["interleaved"]:
        pair, partner, first = j // 2, j ^ 1, j % 2 == 0
    else:
        pair, partner, first = j % max(1, half), (j + half) % max(1, rot), j < half
    moved = j < rot
    pair, partner = torch.where(moved, pair, 0), torch.where(moved, partner, j)
    ang = s["pos"].double()[..., None] * s["inv_freq"].double()[pair]              # [B, N, D]
    cos = torch.where(moved, ang.cos(), 1.0)[:, None]
    sin = torch.where(moved, ang.sin() * torch.where(first, -1.0, 1.0), 0.0)[:, None]
    out, grads, dws = [], [], []
    for x, w, dy in ((s["q"], s["qw"], s.get("dq")), (s["k"], s["kw"], s.get("dk"))):
        x, w = x.double(), w.double()
        size = (x.square().sum(-1, keepdim=True) / D + 1e-6).sqrt()
        u = w * x / size
        out.append(u * cos + u[..., partner] * sin)
        if dy is not None:
            g = dy.double()
            g = g * cos + (g * sin)[..., partner]                                  # the transposed turn
            dws.append((g * x / size).sum((0, 1, 2)))
            g = g * w
            grads.append(g / size - x * (g * x).sum(-1, keepdim=True) / (D * size ** 3))
    return out + grads + dws


def _exact_quantised(x, fmt):
    """The values that the codes of x stand for."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    if fmt == "bf16":
        return x
    if fmt == "int8":
        scale = (top.float() / 127).double().clamp(min=2.0 ** -120)
        return (x / scale).round() * scale
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-120))
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round() * step * scale


def _exact_cache(s):
    case, out = s["case"], []
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        full = cache.double() if scale is None else cache.double() * scale.double()[..., None]
        new = _exact_quantised(x, case["fmt"])
        for b, at in enumerate(s["start"].tolist()):
            full[b, :, at:at + case["N"]] = new[b]
            full[b, :, at + case["N"]:] = 0
        out.append(full[:, :, :s["n"]])
    return out


def _exact_decode(s):
    case = s["case"]
    B, Hq, Hkv, D, Nq = (case[k] for k in ("B", "Hq", "Hkv", "D", "Nq"))
    o = torch.zeros(B, Hq, Nq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    group = Hq // Hkv
    pk, pv = (s[k].double() if k in s else torch.zeros(Hkv, 0, D, dtype=torch.float64, device="cuda")
              for k in ("pk", "pv"))
    for b, n in enumerate(s["lens"].tolist()):
        own_k, own_v = s["kc"][b, :, :n].double(), s["vc"][b, :, :n].double()
        if s["ks"] is not None:
            own_k, own_v = own_k * s["ks"][b, :, :n, None].double(), own_v * s["vs"][b, :, :n, None].double()
        k, v = torch.cat([pk, own_k], 1), torch.cat([pv, own_v], 1)
        for i in range(Nq):
            end = case["prefix"] + n - Nq + i + 1
            if end <= 0:
                continue
            sc = s["q"][b, :, i].double().view(Hkv, group, D) @ k[:, :end].transpose(1, 2) / math.sqrt(D)
            total = torch.logsumexp(sc, -1, keepdim=True)
            o[b, :, i] = (torch.exp(sc - total) @ v[:, :end]).view(Hq, D)
            lse[b, :, i] = total.view(Hq)
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "cache": _exact_cache, "decode": _exact_decode}[case["op"]](s)
