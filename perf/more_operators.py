"""Cases that measure rotary positions and the 4-bit cache of a hybrid decode step's attention layers.

Four operators, each one pass as a serving loop makes it:

  rotary      rotary positions of a projection's query and key heads: half or interleaved pairs, all of a head
              or its first part, frequencies scaled for contexts longer than those that a model was trained on.
  place       the keys of new tokens rotated and stored with the values at their slots of a paged cache, and the
              queries beside them rotated: what comes between an attention layer's projection and its attention.
  cache4      new tokens' keys and values quantised to 4 bits as they are written to the cache, and read back
              from it, as for a prompt whose own attention is to see what later steps will see.
  attention4  the attention of new tokens (one a request, or T drafts) over a paged cache held in 4 bits,
              optionally in a sliding window.

The 4-bit format: for every token and cache head, blocks of 16 consecutive channels. With the head's scale s,
a block of largest magnitude m has the scale b = e4m3(m / (6 s)), and an element x the code e2m1(x / (b s)),
both rounded to nearest, ties to even; the code c stands for c b s.

The plain forms are elementary torch operations in 32 bits (angles in 64), rounded once at the end.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
_SIZE = {"f32": 4.0, "bf16": 2.0, "fp8": 1.0, "nvfp4": 0.5625}      # bytes an element, block scales included
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one token of one request between projection and cache, rotated alone: latency
        dict(name="rotary_b1", op="rotary", tokens=1, heads=40, wide=48, dim=128, rot=128, inter=False, scaling="none",
             base=10000.0, factor=1.0, pos=8191, io="bf16"),
        # prompt tokens far into a context stretched 16 times
        dict(name="rotary_rows16k_yarn", op="rotary", tokens=16384, heads=40, wide=48, dim=128, rot=128, inter=False,
             scaling="yarn", base=10000.0, factor=16.0, pos=131071, io="bf16"),
        # FP32, interleaved pairs in the first quarter of wide heads, an odd number of tokens
        dict(name="rotary_f32_quarter", op="rotary", tokens=5003, heads=18, wide=20, dim=256, rot=64, inter=True,
             scaling="linear", base=500000.0, factor=4.0, pos=40000, io="f32"),
        # a decode step of the serving batch: queries and keys rotated, keys and values stored
        dict(name="place_b256", op="place", batch=256, new=1, q_heads=32, kv_heads=8, dim=128, rot=128, inter=False,
             scaling="wavelength", base=500000.0, factor=8.0, page=16, pos=9000, kv="bf16", io="bf16"),
        # a chunk of three prompts into an FP8 cache
        dict(name="place_fp8_prompts", op="place", batch=3, new=4001, q_heads=32, kv_heads=8, dim=128, rot=64, inter=False,
             scaling="none", base=10000.0, factor=1.0, page=64, pos=60000, kv="fp8", io="bf16"),
        # a decode step's tokens into the 4-bit cache and back: latency
        dict(name="cache4_b64", op="cache4", batch=64, new=1, kv_heads=8, dim=128, page=16, pos=5000, io="bf16"),
        # long prompts written in 4 bits and read back for their own attention
        dict(name="cache4_prompts", op="cache4", batch=5, new=6550, kv_heads=8, dim=128, page=32, pos=30000, io="bf16"),
        # one request, one token, a short context: latency
        dict(name="attn4_b1_ctx777", op="attention4", batch=1, q_heads=32, kv_heads=8, dim=128, page=16, draft=1,
             window=0, lo=777, hi=777),
        # the serving batch at ordinary, ragged contexts, four query heads to a cache head
        dict(name="attn4_b256_ragged", op="attention4", batch=256, q_heads=32, kv_heads=8, dim=128, page=16, draft=1,
             window=0, lo=17, hi=9000),
        # few long requests: the split over the length carries it
        dict(name="attn4_b8_ctx128k", op="attention4", batch=8, q_heads=32, kv_heads=8, dim=128, page=64, draft=1,
             window=0, lo=100001, hi=131072),
        # a speculative round: 4 drafts of 16 query heads over 2 wide cache heads
        dict(name="attn4_draft4_b64_d256", op="attention4", batch=64, q_heads=16, kv_heads=2, dim=256, page=32, draft=4,
             window=0, lo=1000, hi=9999),
        # sliding-window layers: as many cache heads as query heads, most pages out of the window
        dict(name="attn4_window_b128_d64", op="attention4", batch=128, q_heads=16, kv_heads=16, dim=64, page=16, draft=1,
             window=1000, lo=5, hi=6000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_angles(rng, dim):
    rot = rng.choice([dim, dim, dim // 2, dim // 4, dim // 2 + 4, 24])
    return dict(rot=rot, inter=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]),
                base=rng.choice([10000.0, 500000.0]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]), pos=_log(rng, 10, 1000000))


def draw(rng):
    op = rng.choice(["rotary", "place", "cache4", "attention4", "attention4", "attention4"])
    dim = rng.choice([64, 128, 256])
    if op == "rotary":
        io = rng.choice(["bf16", "bf16", "f32"])
        dim = rng.choice([64, 80, 128, 256])
        heads = rng.choice([1, 5, 8, 16, 40, 72])
        tokens = _log(rng, 1, min(200000, int(160_000_000 / (heads * dim * _SIZE[io]))))
        return dict(op=op, tokens=tokens, heads=heads, wide=heads + rng.choice([0, 1, 8]), dim=dim, io=io,
                    **_draw_angles(rng, dim))
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "place":
        kv = rng.choice(["bf16", "bf16", "fp8", "f32"])
        io = "f32" if kv == "f32" else "bf16"
        q_heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        tokens = _log(rng, 1, max(1, int(100_000_000 / ((q_heads + 2 * kv_heads) * dim * _SIZE[io]))))
        batch = _log(rng, 1, min(tokens, 1000))
        return dict(op=op, batch=batch, new=max(1, tokens // batch), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    page=rng.choice([16, 32, 48, 64, 128]), kv=kv, io=io, **_draw_angles(rng, dim))
    if op == "cache4":
        tokens = _log(rng, 1, max(1, 34_000_000 // (kv_heads * dim)))
        batch = _log(rng, 1, min(tokens, 1000))
        return dict(op=op, batch=batch, new=max(1, tokens // batch), kv_heads=kv_heads, dim=dim,
                    page=rng.choice([16, 32, 48, 64, 128]), pos=_log(rng, 10, 200000), io="bf16")
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    batch = _log(rng, 1, 400)
    # at most 0.7 GB of cache, so that no case costs more than the largest listed one
    most = max(64, int(700_000_000 / (batch * kv_heads * dim * _SIZE["nvfp4"] * 2)))
    hi = _log(rng, 32, min(most, 150000))
    # at most 20 GFLOP: many drafts of many heads go with shorter contexts
    most = max(1, int(20e9 / (4 * batch * hi * kv_heads * group * dim)))
    draft = min(most, rng.choice([1, 1, 1, 2, 3, 4, 5, 8]))
    return dict(op=op, batch=batch, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                page=rng.choice([16, 32, 48, 64, 128]), draft=draft, window=rng.choice([0, 0, 0, _log(rng, 1, 5000)]),
                lo=rng.randint(max(1, hi // 20), hi), hi=hi)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _spread(n, lo, hi, seed):
    """n whole numbers spread evenly over lo..hi (a golden-ratio sequence), in an order that the seed turns."""
    v = [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(n)]
    k = seed % n
    return v[k:] + v[:k]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


_ORIGINAL = 4096                                              # positions that the scaled contexts were trained on


def _frequencies(case):
    """Angle per position of each rotated pair (64 bits), and the factor on the rotated values."""
    R, base, f = case["rot"], case["base"], case["factor"]
    i = torch.arange(R // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * f ** (R / (R - 2))
    w = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "yarn":                              # slow channels stretched, fast ones left, a ramp between
        at = [R * math.log(_ORIGINAL / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        w = w / f * ramp + w * (1 - ramp)
    if case["scaling"] == "wavelength":                        # the same, by each channel's wavelength
        s = ((_ORIGINAL * w / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        w = w / f * (1 - s) + w * s
    return w.cuda(), 0.1 * math.log(f) + 1.0 if case["scaling"] == "yarn" else 1.0


def _slots(case, seed, g):
    """Slots and positions of `new` consecutive tokens of each request, on shuffled pages."""
    B, n, ps = case["batch"], case["new"], case["page"]
    start = torch.tensor(_spread(B, 0, case["pos"], seed), device="cuda")
    pos = start[:, None] + torch.arange(n, device="cuda")[None, :]
    first = start // ps
    held = (start + n - 1) // ps - first + 1
    num = int(held.sum()) + 3
    order = torch.randperm(num, generator=g, device="cuda")
    page = order[(held.cumsum(0) - held - first)[:, None] + pos // ps]
    return (page * ps + pos % ps).reshape(-1).to(torch.int32), pos.reshape(-1).to(torch.int32), num


def _scales(n, kv):
    i = torch.arange(n, device="cuda")
    if kv == "fp8":
        return (0.010 + 0.0002 * i).float(), (0.006 + 0.0001 * i).float()
    return (0.0060 + 0.0001 * i).float(), (0.0030 + 0.0001 * i).float()


def _channels(dim):
    """Keys have a few large channels."""
    w = torch.ones(dim, device="cuda")
    w[dim // 8::dim // 4] = 3.0
    return w


def _rotary_inputs(case, seed):
    g = _gen(seed)
    x = _randn(g, case["tokens"], case["wide"], case["dim"]).to(_DT[case["io"]])     # a projection's first heads
    pos = torch.tensor(_spread(case["tokens"], 0, case["pos"], seed), dtype=torch.int32, device="cuda")
    return {"x": x[:, :case["heads"]], "positions": pos}


def _place_inputs(case, seed):
    g = _gen(seed)
    Hq, Hk, D = case.get("q_heads", 0), case["kv_heads"], case["dim"]
    slots, pos, num = _slots(case, seed, g)
    qkv = _randn(g, case["batch"] * case["new"], Hq + 2 * Hk, D)      # one projection's output: q, k and v are slices
    qkv[:, Hq:Hq + Hk] *= _channels(D)
    qkv[:, Hq + Hk:] *= 0.5
    qkv = qkv.to(_DT[case["io"]])
    ks, vs = _scales(Hk, case.get("kv"))
    return {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:], "slots": slots, "positions": pos,
            "k_scale": ks, "v_scale": vs, "num_pages": num}


def _attn_inputs(case, seed, store):
    """Requests on shuffled pages; store(first token slot, k, v) takes the pool's keys and values, a part at a time."""
    B, T, Hq, Hk, D, ps = (case[k] for k in ("batch", "draft", "q_heads", "kv_heads", "dim", "page"))
    g = _gen(seed)
    lens = _spread(B, case["lo"], case["hi"], seed)
    held = [-(-n // ps) for n in lens]
    max_pages = max(held) + 1
    num = sum(held) + 3
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    held_d = torch.tensor(held, dtype=torch.int64, device="cuda")
    j = torch.arange(max_pages, device="cuda")[None, :]
    at = (held_d.cumsum(0) - held_d)[:, None] + j
    table = torch.where(j < held_d[:, None], order[at.clamp(max=num - 1)], -1).to(torch.int32)
    q = _randn(g, B * T, Hq + 2 * Hk, D).to(torch.bfloat16)[:, :Hq]
    to = store(num)
    step = max(1, (1 << 26) // (Hk * ps * D))
    for i in range(0, num, step):
        n = min(step, num - i) * ps
        k = _randn(g, n, Hk, D) * _channels(D)
        v = _randn(g, n, Hk, D) * 0.5
        to(i * ps, k.to(torch.bfloat16), v.to(torch.bfloat16))
    return {"table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "q": q, "max_len": max(lens),
            "max_pages": max_pages, "num_pages": num}


def _plain_pool(case, s):
    """The pool as packed codes [pages][heads][page][dim / 2] and block scales [pages][heads][page][dim / 16]."""
    Hk, D, ps = case["kv_heads"], case["dim"], case["page"]

    def store(num):
        for x in "kv":
            s[x + "_codes"] = torch.empty((num, Hk, ps, D // 2), dtype=torch.uint8, device="cuda")
            s[x + "_blocks"] = torch.empty((num, Hk, ps, D // 16), dtype=torch.float8_e4m3fn, device="cuda")

        def to(slot, *kv):
            i, n = slot // ps, len(kv[0]) // ps
            for x, t in zip("kv", kv):
                codes, blocks = _quantise(t.float(), s[x + "_scale"])
                codes = codes[..., ::2] | codes[..., 1::2] << 4
                s[x + "_codes"][i:i + n] = codes.reshape(n, ps, Hk, D // 2).transpose(1, 2)
                s[x + "_blocks"][i:i + n] = blocks.reshape(n, ps, Hk, D // 16).transpose(1, 2).to(torch.float8_e4m3fn)
        return to
    return store


def prepare(case, seed):
    op = case["op"]
    if op == "attention4":
        return _prepare_attn(case, seed)
    s = _rotary_inputs(case, seed) if op == "rotary" else _place_inputs(case, seed)
    s["case"] = case
    if op != "cache4":
        x = s["x"] if op == "rotary" else s["q"]
        s["out"] = torch.empty(x.shape, dtype=x.dtype, device="cuda")
    if op == "place":
        shape = (s["num_pages"], case["kv_heads"], case["page"], case["dim"])
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, device="cuda").to(_DT[case["kv"]]) for _ in "kv")
    if op == "cache4":
        s["k_out"], s["v_out"] = torch.empty_like(s["k"].contiguous()), torch.empty_like(s["v"].contiguous())
    if not own:
        if op != "cache4":
            s["w"], s["gain"] = _frequencies(case)
        return s
    import hybrid_ssm_decode_gb300 as rssm
    if op != "cache4":
        s["rope"] = rssm.Rope(case["rot"], base=case["base"], interleaved=case["inter"], scaling=case["scaling"],
                              factor=case["factor"], original=_ORIGINAL)
    if op == "cache4":
        row = case["dim"] // 2 + case["dim"] // 16
        shape = (s["num_pages"], case["kv_heads"], case["page"], row)
        s["k_cache"], s["v_cache"] = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in "kv")
    if op != "rotary":
        scaled = op == "cache4" or case["kv"] == "fp8"
        s["attn"] = rssm.Attention(s["k_cache"], s["v_cache"], batch=case["batch"],
                                   q_heads=case.get("q_heads", case["kv_heads"]), max_pages=s["num_pages"],
                                   k_scale=s["k_scale"] if scaled else None, v_scale=s["v_scale"] if scaled else None)
    return s


def _prepare_attn(case, seed):
    B, T, Hq, Hk, D, ps = (case[k] for k in ("batch", "draft", "q_heads", "kv_heads", "dim", "page"))
    s = {"case": case}
    s["k_scale"], s["v_scale"] = _scales(Hk, "nvfp4")
    if own:
        import hybrid_ssm_decode_gb300 as rssm

        def store(num):
            for x in ("k_cache", "v_cache"):
                s[x] = torch.empty((num, Hk, ps, D // 2 + D // 16), dtype=torch.uint8, device="cuda")
            writer = rssm.Attention(s["k_cache"], s["v_cache"], batch=1, q_heads=Hq, max_pages=1, k_scale=s["k_scale"],
                                    v_scale=s["v_scale"])
            return lambda slot, k, v: writer.append(k, v, torch.arange(slot, slot + len(k), dtype=torch.int32, device="cuda"))
        s.update(_attn_inputs(case, seed, store))
        s["attn"] = rssm.Attention(s["k_cache"], s["v_cache"], batch=B, q_heads=Hq, max_pages=s["max_pages"], max_draft=T,
                                   window=case["window"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        s.update(_attn_inputs(case, seed, _plain_pool(case, s)))
        pairs = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device="cuda")
        byte = torch.arange(256, device="cuda")
        s["pairs"] = torch.stack([pairs[byte % 16], pairs[byte // 16]], 1)       # the two values of a byte
    s["out"] = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((B, T, Hq), dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return {"rotary": _run_rotary, "place": _run_place, "cache4": _run_cache,
            "attention4": _run_attn}[state["case"]["op"]](state)


def _rotate(s, x):
    """The first `rot` channels of every head turned by their position's angles; FP32."""
    c = s["case"]
    R = c["rot"]
    a = s["positions"].double()[:, None, None] * s["w"]
    cos, sin = (torch.cos(a) * s["gain"]).float(), (torch.sin(a) * s["gain"]).float()
    x = x.float()
    u, v = (x[..., 0:R:2], x[..., 1:R:2]) if c["inter"] else (x[..., :R // 2], x[..., R // 2:R])
    u, v = u * cos - v * sin, v * cos + u * sin
    turned = torch.stack([u, v], -1).flatten(-2) if c["inter"] else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _run_rotary(s):
    if own:
        import hybrid_ssm_decode_gb300 as rssm
        rssm.rotary(s["out"], s["x"], s["positions"], s["rope"])
        return s["out"]
    return _rotate(s, s["x"]).to(s["x"].dtype)


def _run_place(s):
    c = s["case"]
    if own:
        s["attn"].append(s["k"], s["v"], s["slots"], rope=s["rope"], positions=s["positions"], q=s["q"], q_out=s["out"])
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    slots, ps, fp8 = s["slots"].long(), c["page"], c["kv"] == "fp8"

    def store(cache, new, scale):
        if fp8:                                                # indexed writes move the codes as bytes
            new = (new / scale[:, None]).clamp(-448, 448).to(cache.dtype).view(torch.uint8)
            cache = cache.view(torch.uint8)
        cache[slots // ps, :, slots % ps] = new.to(cache.dtype)

    store(s["k_cache"], _rotate(s, s["k"]), s["k_scale"])
    store(s["v_cache"], s["v"].float(), s["v_scale"])
    return {"q": _rotate(s, s["q"]).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _quantise(x, scale):
    """x [tokens][heads][dim] in 32 bits -> codes (whole numbers, the sign in bit 3) and block scales, as floats."""
    x = x.reshape(*x.shape[:-1], -1, 16)
    b = (x.abs().amax(-1) * (1 / (6 * scale))[:, None]).clamp(max=448).to(torch.float8_e4m3fn).float()
    y = x * torch.where(b > 0, 1 / (b * scale[:, None]), 0.0)[..., None]
    a = y.abs()
    # the borders between neighbouring codes; on a border the even code
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())
    return (code + 8 * (y < 0).byte()).flatten(-2), b


def _run_cache(s):
    if own:
        s["attn"].append(s["k"], s["v"], s["slots"])
        s["attn"].read(s["k_out"], s["v_out"], s["slots"])
        return {"k": s["k_out"], "v": s["v_out"]}
    table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device="cuda")

    def there_and_back(x, scale):
        codes, blocks = _quantise(x.float(), scale)
        return (table[codes.int()].unflatten(-1, (-1, 16)) * (blocks * scale[:, None])[..., None]).flatten(-2).to(x.dtype)

    return {"k": there_and_back(s["k"], s["k_scale"]), "v": there_and_back(s["v"], s["v_scale"])}


def _run_attn(s):
    c = s["case"]
    B, T, Hq, Hk, D, ps = (c[k] for k in ("batch", "draft", "q_heads", "kv_heads", "dim", "page"))
    if own:
        s["attn"].decode(s["out"], s["q"], s["lens"], s["table"], T=T, lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    L = s["max_len"]
    pages = s["table"][:, :-(-L // ps)].clamp(min=0).long()
    pos = torch.arange(pages.shape[1] * ps, device="cuda")

    def rows(x):                                               # [B][Hk][tokens][D] in 32 bits
        v = s["pairs"][s[x + "_codes"][pages].int()].reshape(B, -1, Hk, ps, D // 16, 16)
        b = s[x + "_blocks"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * s[x + "_scale"][:, None, None]
        return (v * b[..., None]).permute(0, 2, 1, 3, 4, 5).reshape(B, Hk, -1, D)

    p = s["lens"].long()[:, None] - T + torch.arange(T, device="cuda")[None, :]        # [B][T]
    seen = pos[None, None, :] <= p[:, :, None]
    if c["window"]:
        seen = seen & (pos[None, None, :] > p[:, :, None] - c["window"])
    q = s["q"].float().reshape(B, T, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)
    score = torch.matmul(q, rows("k").transpose(-1, -2)) / math.sqrt(D)
    score = score.reshape(B, Hk, T, Hq // Hk, -1).masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    w = torch.where(total > 0, e / total, 0.0).reshape(B, Hk, T * (Hq // Hk), -1)
    v = torch.where(seen.any(1)[:, None, :, None], rows("v"), 0.0)
    o = torch.matmul(w, v).reshape(B, Hk, T, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = (torch.log(total) + top).reshape(B, Hk, T, Hq // Hk).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return {"out": o.to(torch.bfloat16), "lse": lse}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op, D = case["op"], case["dim"]
    if op == "rotary":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * D * _SIZE[case["io"]] + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    if op in ("place", "cache4"):
        tokens, io, Hk, Hq = case["batch"] * case["new"], _SIZE[case["io"]], case["kv_heads"], case.get("q_heads", 0)
        if op == "place":
            b = tokens * D * (2 * Hq * io + 2 * Hk * (io + _SIZE[case["kv"]])) + 8 * tokens
            return {"bytes": b, "flops": 3 * tokens * (Hq + Hk) * case["rot"]}
        # read, written in 4 bits, read in 4 bits, written
        return {"bytes": tokens * D * 4 * Hk * (io + _SIZE["nvfp4"]) + 8 * tokens, "flops": 6 * tokens * Hk * D}
    T, W, Hq, Hk = case["draft"], case["window"], case["q_heads"], case["kv_heads"]
    lens = _spread(case["batch"], case["lo"], case["hi"], 0)
    tokens = sum(min(n, W + T - 1) if W else n for n in lens)
    pairs = sum(min(n - T + t + 1, W) if W else n - T + t + 1 for n in lens for t in range(T) if n - T + t >= 0)
    new = case["batch"] * T
    b = tokens * Hk * D * 2 * _SIZE["nvfp4"] + new * Hq * (D * 4 + 4)
    return {"bytes": b + 4 * (tokens // case["page"] + 2 * case["batch"]), "flops": 4 * pairs * Hq * D}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "rotary":
        s = _rotary_inputs(case, seed)
        return _turn(case, s["x"], s["positions"])
    if op == "place":
        s = _place_inputs(case, seed)
        ps, kv = case["page"], []
        for x, scale in ((_turn(case, s["k"], s["positions"]), s["k_scale"]), (s["v"].double(), s["v_scale"])):
            c = torch.zeros((s["num_pages"], ps, case["kv_heads"], case["dim"]), dtype=torch.float64, device="cuda")
            if case["kv"] == "fp8":                            # the cache holds the values over their scale
                x = (x / scale.double()[:, None]).clamp(-448, 448)
            c.flatten(0, 1)[s["slots"].long()] = x
            kv.append(c.transpose(1, 2))
        return {"q": _turn(case, s["q"], s["positions"]), "k_cache": kv[0], "v_cache": kv[1]}
    if op == "cache4":
        s = _place_inputs(case, seed)
        return {x: _nearest(s[x].double(), s[x + "_scale"].double()) for x in "kv"}
    return _exact_attn(case, seed)


def _turn(case, x, positions):
    """The rotation as a product of complex numbers."""
    R, f, base = case["rot"], case["factor"], case["base"]
    if case["scaling"] == "ntk":
        base *= f ** (R / (R - 2.0))
    freq, gain = [], 1.0
    for i in range(R // 2):
        w = math.exp(-2.0 * i / R * math.log(base))
        turns = _ORIGINAL * w / (2 * math.pi)                  # over the positions trained on
        if case["scaling"] == "linear":
            w /= f
        elif case["scaling"] == "wavelength":
            keep = 1.0 if turns > 4 else 0.0 if turns < 1 else (turns - 1) / 3
            w *= keep + (1 - keep) / f
        elif case["scaling"] == "yarn":
            edge = [math.log(_ORIGINAL / (2 * math.pi * b)) * R / (2 * math.log(base)) for b in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(R - 1, math.ceil(edge[1]))
            t = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            w *= (1 - t) + t / f
            gain = 1 + math.log(f) / 10
        freq.append(w)
    a = torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(a, gain), a)[:, None, :]
    y = x.double().clone()
    head = y[..., :R].unflatten(-1, (R // 2, 2) if case["inter"] else (2, R // 2))
    if not case["inter"]:
        head = head.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
    y[..., :R] = (z if case["inter"] else z.transpose(-1, -2)).flatten(-2)
    return y


def _nearest(x, scale):
    """Each value replaced by the nearest one that its block can hold."""
    blocks = x.unflatten(-1, (-1, 16))
    b = (blocks.abs().amax(-1) / (6 * scale[:, None])).clamp(max=448).float().to(torch.float8_e4m3fn).double()
    unit = (b * scale[:, None])[..., None]
    grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    best, far = torch.zeros_like(blocks), torch.full_like(blocks, math.inf)
    for v in grid:
        d = (blocks.abs() - v * unit).abs()
        best, far = torch.where(d < far, (v * unit).expand_as(d), best), torch.minimum(d, far)
    return (best * blocks.sign()).flatten(-2)


def _exact_attn(case, seed):
    """Request by request and draft by draft, over the tokens that the draft sees."""
    T, Hq, Hk, D, ps = (case[k] for k in ("draft", "q_heads", "kv_heads", "dim", "page"))
    B, W = case["batch"], case["window"]
    s = {}
    s["k_scale"], s["v_scale"] = _scales(Hk, "nvfp4")
    s.update(_attn_inputs(case, seed, _plain_pool(case, s)))
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    grid = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(B):
        n = lens[b]
        first = max(0, n - T - W + 1) if W else 0              # the first token that any draft sees
        first -= first % ps
        ids = s["table"][b, first // ps:-(-n // ps)].long()
        kv = []
        for x in "kv":
            codes = s[x + "_codes"][ids].transpose(0, 1).reshape(Hk, -1, D // 2)[:, :n - first].int()
            val = torch.stack([grid[codes % 16], grid[codes // 16]], -1).reshape(Hk, n - first, D // 16, 16)
            blk = s[x + "_blocks"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
            blk = blk.transpose(0, 1).reshape(Hk, -1, D // 16)[:, :n - first]
            kv.append((val * blk[..., None]).flatten(-2) * s[x + "_scale"].double()[:, None, None])
        q = s["q"][b * T:(b + 1) * T].double().reshape(T, Hk, Hq // Hk, D)
        for t in range(T):
            p = n - T + t
            if p < 0:
                continue
            lo = max(0, p - W + 1) - first if W else 0
            sc = torch.einsum("hgd,hnd->hgn", q[t], kv[0][:, lo:p + 1 - first]) / math.sqrt(D)
            l = torch.logsumexp(sc, -1)
            o = torch.einsum("hgn,hnd->hgd", torch.exp(sc - l[..., None]), kv[1][:, lo:p + 1 - first])
            out[b, t], lse[b, t] = o.reshape(Hq, D), l.reshape(Hq)
    return {"out": out, "lse": lse}
