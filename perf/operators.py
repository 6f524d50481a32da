"""Cases that measure the operators of a hybrid decode step beside the SSM layers.

Four operators, each one pass as a serving loop makes it:

  pages       the page table of a batch: pages handed out and taken back on the GPU, with the slot and
              the position of every new token. A pass is a draft round whose drafts are all rejected
              ("round": extend by T, roll T back), or a batch turned over ("admit": every request leaves,
              new prompts of given lengths come). Either leaves the table as it found it.
  attention   the new tokens' keys and values written to their slots of a paged cache, and the attention of
              the new tokens over it (one token a request, or T drafts), optionally in a sliding window.
  add_norm    a block's output, optionally normalised, gated and scaled, added to the residual stream, and the
              norm of the sum that the next block reads.
  gated_norm  the norm after an SSM mixer, fused with its gate (Mamba-2: the gated product is normalised in
              groups; Gated DeltaNet: each head is normalised and then gated).

The plain forms are elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "bf16": 2, "fp8": 1}
_EPS = 1e-6


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # a draft round of a small serving batch: the table's own latency, twice
        dict(name="pages_round_b64_t4", op="pages", mode="round", batch=64, page=16, draft=4, lo=100, hi=9000),
        # a large batch turned over: 256 prompts of 1 to 32k tokens get their pages and slots
        dict(name="pages_admit_b256_32k", op="pages", mode="admit", batch=256, page=16, draft=1, lo=1, hi=32768),
        # one request, one token, a short context: latency
        dict(name="attn_b1_ctx777", op="attention", batch=1, q_heads=32, kv_heads=8, dim=128, page=16, draft=1,
             window=0, lo=777, hi=777, io="bf16", kv="bf16"),
        # the serving batch at ordinary, ragged contexts, four query heads to a cache head
        dict(name="attn_b256_ragged", op="attention", batch=256, q_heads=32, kv_heads=8, dim=128, page=16, draft=1,
             window=0, lo=17, hi=4500, io="bf16", kv="bf16"),
        # few long requests over an FP8 cache: the split over the length carries it
        dict(name="attn_fp8_b8_ctx128k", op="attention", batch=8, q_heads=32, kv_heads=8, dim=128, page=64, draft=1,
             window=0, lo=100001, hi=131072, io="bf16", kv="fp8"),
        # a speculative round: 4 drafts of 16 query heads to a cache head, wide heads
        dict(name="attn_draft4_b64_d256", op="attention", batch=64, q_heads=16, kv_heads=2, dim=256, page=32, draft=4,
             window=0, lo=1000, hi=9999, io="bf16", kv="bf16"),
        # sliding-window layers: as many cache heads as query heads, most pages out of the window
        dict(name="attn_window_b128_d64", op="attention", batch=128, q_heads=16, kv_heads=16, dim=64, page=16, draft=1,
             window=1000, lo=5, hi=6000, io="bf16", kv="bf16"),
        # FP32 throughout, as in the small FP32 decode configuration
        dict(name="attn_f32_b4", op="attention", batch=4, q_heads=8, kv_heads=8, dim=64, page=16, draft=1,
             window=0, lo=500, hi=2047, io="f32", kv="f32"),
        # between two blocks of a one-request decode: latency
        dict(name="add_norm_b1", op="add_norm", rows=1, dim=4096, res="bf16", io="bf16", post=False, gate="none"),
        # prompt tokens through a block with norms on both sides, a gate per channel, FP32 residual stream
        dict(name="add_norm_rows16k_sandwich", op="add_norm", rows=16384, dim=4096, res="f32", io="bf16", post=True,
             gate="channel"),
        # after the Mamba-2 mixer of the serving layer: 128 heads of 64 in 8 groups
        dict(name="gated_norm_mamba2_b256", op="gated_norm", rows=256, dim=8192, group=1024, first=False, io="bf16"),
        # after the Gated DeltaNet mixer on prompt tokens: 32 heads of 128
        dict(name="gated_norm_gdn_rows16k", op="gated_norm", rows=16384, dim=4096, group=128, first=True, io="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "attention", "attention", "attention", "add_norm", "gated_norm"])
    if op == "pages":
        mode = rng.choice(["round", "admit"])
        batch = _log(rng, 1, 1000)
        hi = _log(rng, 20, min(60000, max(21, 8_000_000 // batch)))
        return dict(op=op, mode=mode, batch=batch, page=rng.choice([16, 32, 64, 128]), draft=rng.randint(1, 8),
                    lo=rng.randint(1, hi), hi=hi)
    if op == "attention":
        kv, io = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp8", "bf16"), ("fp8", "bf16"), ("f32", "f32")])
        dim = rng.choice([64, 128, 256])
        kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        batch = _log(rng, 1, 400)
        # at most 1 GB of cache, so that no case costs more than the largest listed one
        most = max(64, 500_000_000 // (batch * kv_heads * dim * _SIZE[kv] * 2))
        hi = _log(rng, 32, min(most, 150000))
        # at most 20 GFLOP: many drafts of many heads go with shorter contexts
        most = max(1, int(20e9 / (4 * batch * hi * kv_heads * group * dim)))
        draft = min(most, rng.choice([1, 1, 1, 2, 3, 4, 5, 8]))
        return dict(op=op, batch=batch, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    page=rng.choice([16, 32, 48, 64, 128]), draft=draft, window=rng.choice([0, 0, 0, _log(rng, 1, 5000)]),
                    lo=rng.randint(max(1, hi // 20), hi), hi=hi, io=io, kv=kv)
    rows = _log(rng, 1, 16000)
    if op == "add_norm":
        dim = _log(rng, 128, max(128, min(8192, 64_000_000 // rows)))
        dim -= rng.choice([0, dim % 8, dim % 8, dim % 8])      # odd ones among them
        return dict(op=op, rows=rows, dim=dim, res=rng.choice(["bf16", "f32"]), io=rng.choice(["bf16", "bf16", "f32"]),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "row"]))
    first = rng.random() < 0.5
    group = rng.choice([64, 128, 256]) if first else 8 * _log(rng, 8, 256)
    most = max(1, min(64, 16384 // group, 60_000_000 // (rows * group)))
    return dict(op=op, rows=rows, dim=group * _log(rng, 1, most) if most > 1 else group, group=group, first=first,
                io=rng.choice(["bf16", "bf16", "f32"]))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _lens(case, seed=0):
    """Request lengths spread evenly over lo..hi (a golden-ratio sequence), in an order that the seed turns."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    v = [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(n)]
    k = seed % n
    return v[k:] + v[:k]


def _visible(case, length):
    """Per draft, the number of cached tokens it sees."""
    T, W = case["draft"], case["window"]
    out = []
    for t in range(T):
        p = length - T + t
        out.append(0 if p < 0 else min(p + 1, W) if W else p + 1)
    return out


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _inputs(case, seed):
    return {"pages": _pages_inputs, "attention": _attn_inputs, "add_norm": _add_inputs,
            "gated_norm": _gated_inputs}[case["op"]](case, seed)


def _pages_inputs(case, seed):
    B, ps = case["batch"], case["page"]
    lens = _lens(case, seed)
    rows = -(-(case["hi"] + case["draft"]) // ps)              # the longest request, with its drafts
    need = sum(-(-(n + case["draft"]) // ps) for n in lens)
    num = need + max(8, need // 8)                             # a pool with some room
    g = _gen(seed)
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    total = B * case["draft"] if case["mode"] == "round" else sum(lens)
    return {"free0": order, "lens0": torch.tensor(lens, dtype=torch.int32, device="cuda"), "max_pages": rows,
            "num_pages": num, "total": total,
            "zeros": torch.zeros(B, dtype=torch.int32, device="cuda")}


def _attn_inputs(case, seed):
    B, T, Hq, Hk, D, ps = (case[k] for k in ("batch", "draft", "q_heads", "kv_heads", "dim", "page"))
    g = _gen(seed)
    lens = _lens(case, seed)
    held = [-(-n // ps) for n in lens]
    max_pages = max(held) + 1
    num = sum(held) + 3
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    held_d = torch.tensor(held, dtype=torch.int64, device="cuda")
    j = torch.arange(max_pages, device="cuda")[None, :]
    at = (held_d.cumsum(0) - held_d)[:, None] + j
    inside = j < held_d[:, None]
    table = torch.where(inside, order[at.clamp(max=num - 1)], -1).to(torch.int32)
    ks = (0.010 + 0.0002 * torch.arange(Hk, device="cuda")).float()
    vs = (0.006 + 0.0001 * torch.arange(Hk, device="cuda")).float()
    caches = []
    for s, scale in ((1.0, ks), (0.5, vs)):
        c = torch.empty((num, Hk, ps, D), dtype=_DT[case["kv"]], device="cuda")
        step = max(1, (1 << 28) // (Hk * ps * D))
        for i in range(0, num, step):                          # in pieces: the FP32 draw is the larger one
            x = _randn(g, min(step, num - i), Hk, ps, D) * s
            if case["kv"] == "fp8":
                x = (x / scale[:, None, None]).clamp(-448, 448)
            c[i:i + step] = x.to(c.dtype)
        caches.append(c)
    qkv = _randn(g, B * T, Hq + 2 * Hk, D)                     # one projection's output: q, k and v are slices
    qkv[:, Hq + Hk:] *= 0.5
    qkv = qkv.to(_DT[case["io"]])
    # a request shorter than its drafts has no slot for the first of them
    pos = lens_d.long()[:, None] - T + torch.arange(T, device="cuda")[None, :]
    page = torch.gather(table.long(), 1, pos.clamp(min=0) // ps)
    slots = torch.where(pos < 0, -1, page * ps + pos % ps).to(torch.int32)
    return {"k_cache": caches[0], "v_cache": caches[1], "table": table, "lens": lens_d, "slots": slots.reshape(-1),
            "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:], "k_scale": ks, "v_scale": vs,
            "max_len": max(lens), "max_pages": max_pages, "num_pages": num}


def _add_inputs(case, seed):
    g = _gen(seed)
    n, d = case["rows"], case["dim"]
    io = _DT[case["io"]]
    s = {"u": (_randn(g, n, d) * 3).to(_DT[case["res"]]), "x": _randn(g, n, d).to(io), "w": 1 + 0.1 * _randn(g, d),
         "w_post": (1 + 0.1 * _randn(g, d)) if case["post"] else None, "gate": None, "scale": 0.7}
    if case["gate"] == "channel":
        s["gate"] = torch.sigmoid(_randn(g, d)).to(io)
    elif case["gate"] == "row":
        s["gate"] = torch.sigmoid(_randn(g, n, d)).to(io)
    return s


def _gated_inputs(case, seed):
    g = _gen(seed)
    n, d = case["rows"], case["dim"]
    zy = _randn(g, n, 2 * d).to(_DT[case["io"]])               # the gate is a slice of a wider projection
    w = 1 + 0.1 * _randn(g, case["group"] if case["first"] else d)
    return {"y": _randn(g, n, d).to(_DT[case["io"]]), "z": zy[:, :d], "w": w}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "pages":
        B = case["batch"]
        s["slots"] = torch.empty(s["total"], dtype=torch.int32, device="cuda")
        s["positions"] = torch.empty(s["total"], dtype=torch.int32, device="cuda")
    if case["op"] == "attention":
        s["out"] = torch.empty((case["batch"], case["draft"], case["q_heads"], case["dim"]), dtype=_DT[case["io"]],
                               device="cuda")
        s["lse"] = torch.empty((case["batch"], case["draft"], case["q_heads"]), dtype=torch.float32, device="cuda")
    if case["op"] == "add_norm":
        s["u_out"], s["n_out"] = torch.empty_like(s["u"]), torch.empty_like(s["x"])
    if case["op"] == "gated_norm":
        s["out"] = torch.empty_like(s["y"])
    if not own:
        if case["op"] == "pages":                              # the batch as it is before the pass: its pages held
            s["table"] = torch.full((B, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
            s["lens"], s["free"] = s["zeros"].clone(), s["free0"].clone()
            s["nfree"] = torch.full((1,), s["num_pages"], dtype=torch.int32, device="cuda")
            n = int(s["lens0"].sum())
            _plain_extend(s, s["lens0"], n)
        return s
    import hybrid_ssm_decode_gb300 as rssm
    if case["op"] == "pages":
        s["pages"] = rssm.PageTable(case["batch"], case["page"], s["num_pages"], s["max_pages"], free=s["free0"])
        n = int(s["lens0"].sum())
        tmp = torch.empty(n, dtype=torch.int32, device="cuda")
        s["pages"].extend(tmp, new=s["lens0"])
    if case["op"] == "attention":
        fp8 = case["kv"] == "fp8"
        s["attn"] = rssm.Attention(s["k_cache"], s["v_cache"], batch=case["batch"], q_heads=case["q_heads"],
                                   max_pages=s["max_pages"], max_draft=case["draft"], window=case["window"],
                                   in_dtype=case["io"], k_scale=s["k_scale"] if fp8 else None,
                                   v_scale=s["v_scale"] if fp8 else None)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return {"pages": _run_pages, "attention": _run_attn, "add_norm": _run_add,
            "gated_norm": _run_gated}[state["case"]["op"]](state)


def _run_pages(s):
    c = s["case"]
    if own:
        p = s["pages"]
        if c["mode"] == "round":
            p.extend(s["slots"], T=c["draft"], positions=s["positions"])
            p.rollback(c["draft"], s["zeros"])
        else:
            p.truncate(s["zeros"])
            p.extend(s["slots"], new=s["lens0"], positions=s["positions"])
        return {"slots": s["slots"], "positions": s["positions"], "lens": p.lens, "table": p.table, "free": p.free_count}
    if c["mode"] == "round":
        slots, positions = _plain_extend(s, torch.full_like(s["lens"], c["draft"]), s["total"])
        _plain_truncate(s, s["lens"] - c["draft"] + s["zeros"])
    else:
        _plain_truncate(s, s["zeros"])
        slots, positions = _plain_extend(s, s["lens0"], s["total"])
    return {"slots": slots, "positions": positions, "lens": s["lens"], "table": s["table"], "free": s["nfree"]}


def _plain_extend(s, new, total):
    """Pages for `new` tokens more a request, in the order of the requests; their slots and positions."""
    ps, table, lens, nfree = s["case"]["page"], s["table"], s["lens"].long(), s["nfree"].long()
    new = new.long()
    held, want = (lens + ps - 1) // ps, (lens + new + ps - 1) // ps
    need = torch.where(want <= s["max_pages"], want - held, 0)
    served = (want <= s["max_pages"]) & ((need == 0) | (need.cumsum(0) <= nfree))
    take = torch.where(served, need, 0)
    base = nfree - take.sum()
    j = torch.arange(s["max_pages"], device="cuda")[None, :] - held[:, None]
    at = (base + take.cumsum(0) - take)[:, None] + j
    fresh = (j >= 0) & (j < take[:, None])
    s["table"] = torch.where(fresh, s["free"][at.clamp(0, s["num_pages"] - 1)], table)
    first = new.cumsum(0) - new
    r = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), new, output_size=total)
    pos = lens[r] + torch.arange(total, device="cuda") - first[r]
    ok = served[r]
    slots = torch.where(ok, s["table"][r, (pos // ps).clamp(max=s["max_pages"] - 1)] * ps + pos % ps, -1)
    s["lens"] = (lens + torch.where(served, new, 0)).to(torch.int32)
    s["nfree"] = base.to(torch.int32)
    return slots.to(torch.int32), torch.where(ok, pos, -1).to(torch.int32)


def _plain_truncate(s, keep):
    """Each request cut to `keep` tokens; the pages that it no longer fills go back to the free list."""
    ps, table, lens = s["case"]["page"], s["table"], s["lens"].long()
    keep = torch.minimum(lens, keep.long())
    held, left = (lens + ps - 1) // ps, (keep + ps - 1) // ps
    back = held - left
    j = torch.arange(s["max_pages"], device="cuda")[None, :]
    gone = (j >= left[:, None]) & (j < held[:, None])
    at = (s["nfree"].long() + back.cumsum(0) - back - left)[:, None] + j
    free = torch.cat([s["free"], s["free"][:1]])               # one place more takes what does not go back
    free[torch.where(gone, at, s["num_pages"])] = table
    s["free"] = free[:-1]
    s["table"] = torch.where(gone, -1, table)
    s["lens"] = keep.to(torch.int32)
    s["nfree"] = (s["nfree"] + back.sum()).to(torch.int32)


def _run_attn(s):
    c = s["case"]
    B, T, Hq, Hk, D, ps = (c[k] for k in ("batch", "draft", "q_heads", "kv_heads", "dim", "page"))
    if own:
        a = s["attn"]
        a.append(s["k"], s["v"], s["slots"])
        a.decode(s["out"], s["q"], s["lens"], s["table"], T=T, lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    fp8 = c["kv"] == "fp8"
    slots = s["slots"].long()
    keep = slots >= 0
    old = slots.clamp(min=0)
    for cache, new, scale in ((s["k_cache"], s["k"], s["k_scale"]), (s["v_cache"], s["v"], s["v_scale"])):
        if fp8:
            new = (new.float() / scale[:, None]).clamp(-448, 448)
        new = new.to(cache.dtype)
        if fp8:                                                # indexed writes move the codes as bytes
            cache, new = cache.view(torch.uint8), new.view(torch.uint8)
        new = torch.where(keep[:, None, None], new, cache[old // ps, :, old % ps])
        cache[old // ps, :, old % ps] = new
    L = s["max_len"]
    pages = s["table"][:, :-(-L // ps)].clamp(min=0).long()
    pos = torch.arange(pages.shape[1] * ps, device="cuda")

    def rows(cache, scale):                                    # [B][Hk][tokens][D] in 32 bits
        x = cache.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() if fp8 else cache[pages].float()
        if fp8:
            x = x * scale[:, None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)

    p = s["lens"].long()[:, None] - T + torch.arange(T, device="cuda")[None, :]        # [B][T]
    seen = pos[None, None, :] <= p[:, :, None]
    if c["window"]:
        seen = seen & (pos[None, None, :] > p[:, :, None] - c["window"])
    any_row = seen.any(1)[:, None, :, None]
    q = s["q"].float().reshape(B, T, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)
    score = torch.matmul(q, rows(s["k_cache"], s["k_scale"]).transpose(-1, -2)) / math.sqrt(D)
    score = score.reshape(B, Hk, T, Hq // Hk, -1).masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    w = torch.where(total > 0, e / total, 0.0).reshape(B, Hk, T * (Hq // Hk), -1)
    v = torch.where(any_row, rows(s["v_cache"], s["v_scale"]), 0.0)
    o = torch.matmul(w, v).reshape(B, Hk, T, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = (torch.log(total) + top).reshape(B, Hk, T, Hq // Hk).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return {"out": o.to(_DT[c["io"]]), "lse": lse, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_add(s):
    if own:
        import hybrid_ssm_decode_gb300 as rssm
        rssm.add_norm(s["n_out"], s["u"], s["w"], x=s["x"], u_out=s["u_out"], w_post=s["w_post"], gate=s["gate"],
                      scale=s["scale"], eps=_EPS)
        return {"u": s["u_out"], "n": s["n_out"]}
    a = s["x"].float()
    if s["w_post"] is not None:
        a = a * torch.rsqrt((a * a).mean(-1, keepdim=True) + _EPS) * s["w_post"]
    if s["gate"] is not None:
        a = a * s["gate"].float()
    u = s["u"].float() + s["scale"] * a
    n = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + _EPS) * s["w"]
    return {"u": u.to(s["u"].dtype), "n": n.to(s["x"].dtype)}


def _run_gated(s):
    c = s["case"]
    if own:
        import hybrid_ssm_decode_gb300 as rssm
        rssm.gated_norm(s["out"], s["y"], s["z"], s["w"], group=c["group"], norm_first=c["first"], eps=_EPS)
        return s["out"]
    y, z = s["y"].float(), s["z"].float()
    gate = z / (1 + torch.exp(-z))
    v = y if c["first"] else y * gate
    v = v.reshape(c["rows"], -1, c["group"])
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + _EPS)
    if c["first"]:
        return (v * s["w"]).reshape(c["rows"], -1).mul(gate).to(s["y"].dtype)
    return (v.reshape(c["rows"], -1) * s["w"]).to(s["y"].dtype)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "pages":
        ps, B = case["page"], case["batch"]
        lens = _lens(case)
        if case["mode"] == "round":
            tokens = B * case["draft"]
            moved = sum(-(-(n + case["draft"]) // ps) - -(-n // ps) for n in lens)
        else:
            tokens = sum(lens)
            moved = sum(-(-n // ps) for n in lens)
        # slots and positions; each page out of the free list, into the table, and back; lengths and counts
        return {"bytes": 8 * tokens + 16 * moved + 24 * B, "flops": 0}
    if op == "attention":
        T, Hq, Hk, D = (case[k] for k in ("draft", "q_heads", "kv_heads", "dim"))
        io, kv = _SIZE[case["io"]], _SIZE[case["kv"]]
        lens = _lens(case)
        tokens = sum(min(n, case["window"] + T - 1) if case["window"] else n for n in lens)
        pairs = sum(sum(_visible(case, n)) for n in lens)
        new = case["batch"] * T
        b = tokens * Hk * D * 2 * kv + new * (Hq * D * 2 + Hk * D * 2) * io + new * Hk * D * 2 * kv + new * Hq * 4
        return {"bytes": b + 4 * (tokens // case["page"] + 2 * case["batch"] + new), "flops": 4 * pairs * Hq * D}
    n, d, io = case["rows"], case["dim"], _SIZE[case["io"]]
    if op == "add_norm":
        b = n * d * 2 * (_SIZE[case["res"]] + io) + 4 * d * (2 if case["post"] else 1)
        b += {"none": 0, "channel": d * io, "row": n * d * io}[case["gate"]]
        return {"bytes": b, "flops": n * d * (10 if case["post"] else 6)}
    return {"bytes": 3 * n * d * io + 4 * (case["group"] if case["first"] else d), "flops": 8 * n * d}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "pages":
        return None                                            # whole numbers
    s = _inputs(case, seed)
    if case["op"] == "attention":
        return _exact_attn(case, s)
    if case["op"] == "add_norm":
        x, u = s["x"].double(), s["u"].double()
        if s["w_post"] is not None:
            x = x / (x.square().sum(1, keepdim=True) / case["dim"] + _EPS).sqrt() * s["w_post"].double()
        if s["gate"] is not None:
            x = x * s["gate"].double()
        u = u + s["scale"] * x
        return {"u": u, "n": u / (u.square().sum(1, keepdim=True) / case["dim"] + _EPS).sqrt() * s["w"].double()}
    y, z, w = s["y"].double(), s["z"].double(), s["w"].double()
    out = torch.empty_like(y)
    gate = z * torch.sigmoid(z)
    for i in range(0, case["dim"], case["group"]):
        j = slice(i, i + case["group"])
        if case["first"]:
            v = y[:, j]
            out[:, j] = v / (v.square().sum(1, keepdim=True) / case["group"] + _EPS).sqrt() * w * gate[:, j]
        else:
            v = y[:, j] * gate[:, j]
            out[:, j] = v / (v.square().sum(1, keepdim=True) / case["group"] + _EPS).sqrt() * w[j]
    return out


def _exact_attn(case, s):
    """Request by request and draft by draft, over the tokens that the draft sees."""
    T, Hq, Hk, D, ps = (case[k] for k in ("draft", "q_heads", "kv_heads", "dim", "page"))
    B, W, fp8 = case["batch"], case["window"], case["kv"] == "fp8"
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(B):
        n = lens[b]
        first = max(0, n - T - W + 1) if W else 0              # the first token that any draft sees
        first -= first % ps
        ids = s["table"][b, first // ps:-(-n // ps)].long()
        kv = []
        for cache, new, scale in ((s["k_cache"], s["k"], s["k_scale"]), (s["v_cache"], s["v"], s["v_scale"])):
            x = cache.view(torch.uint8)[ids].view(cache.dtype) if fp8 else cache[ids]
            x = x.transpose(0, 1).reshape(Hk, -1, D)[:, :n - first].double()
            for t in range(max(0, T - n), T):                  # the new tokens, as they lie in the cache
                v = new[b * T + t].double()
                if fp8:
                    v = (v / scale.double()[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
                x[:, n - T + t - first] = v
            kv.append(x * scale.double()[:, None, None] if fp8 else x)
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
    return {"out": out, "lse": lse, "k_cache": None, "v_cache": None}
