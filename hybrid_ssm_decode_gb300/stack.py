"""Synthetic decode stacks: Mamba-2 layers alone (M2Stack), and Mamba-2 and
attention layers in a given order (HybridStack).

The pages set the SSM-kernel speedup beside a smaller speedup of the whole
decode step ("ReplaySSM beschleunigt das Decoding von Hybridmodellen ...",
section "Wichtige Details"; "NVIDIA ve Dao AI Lab, ... ReplaySSM'i sundu",
section "Durum trafiğini azaltma ve rollback'ın basitleştirilmesi"): the SSM
layer is one part of a step that also runs the layer's projections. This
module builds that step from random-weight parts, so the SSM layer's share
and the step-level speedup can be measured without a trained model.

One layer, for the hidden state u [B][d_model] (bf16), with d_inner = H * P
and d_model = d_inner / 2 (the Mamba-2 expansion factor of 2):

    n  = u / rms(u)                                  RMS normalisation
    x  = n W_x,  z = n W_z                           [B][d_inner] = [B][H][P]
    Bt = n W_B,  Ct = n W_C                          [B][G][N]
    dt = softplus(n W_dt + dt_bias)                  [B][H]
    y  = SSM decode step (x, Bt, Ct, dt)             librssm, this layer's state
    u  = u + (y * silu(z)) W_out                     residual

The projections are plain bf16 GEMMs (cuBLAS through torch.matmul) and the
element-wise steps are torch operations: they are the same in the replay and
conventional stacks, which differ only in the SSM layer's mode. Weights are
N(0, 1/fan_in), drawn from a seeded torch generator on the device.
"""
from __future__ import annotations

from dataclasses import dataclass

import synth

from . import Attention, Layer, PageTable, add_norm, gated_norm, make_config


@dataclass(frozen=True)
class StackShape:
    layers: int
    batch: int
    heads: int = 128
    head_dim: int = 64
    state_dim: int = 128
    groups: int = 8
    k: int = 16

    @property
    def d_inner(self) -> int:
        return self.heads * self.head_dim

    @property
    def d_model(self) -> int:
        return self.d_inner // 2


class M2Stack:
    """`shape.layers` Mamba-2 layers with random projections on one GPU.

    mode: "replay" or "conventional" (the SSM layer's mode); ckpt / read_fmt
    as in make_config. The weights depend on `seed` only, so two stacks with
    the same seed and different modes compute the same function.
    """

    def __init__(self, shape: StackShape, mode="replay", ckpt="f32", read_fmt="none", seed=0,
                 device="cuda"):
        import torch
        self.shape, self.mode = shape, mode
        s = shape
        gen = torch.Generator(device=device)
        gen.manual_seed(1000 + seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device=device, dtype=torch.float32)
            return (w / rows ** 0.5).to(torch.bfloat16)

        self.weights = []
        self.layers = []
        for li in range(s.layers):
            w = {"x": weight(s.d_model, s.d_inner), "z": weight(s.d_model, s.d_inner),
                 "B": weight(s.d_model, s.groups * s.state_dim),
                 "C": weight(s.d_model, s.groups * s.state_dim),
                 "dt": weight(s.d_model, s.heads),
                 "out": weight(s.d_inner, s.d_model)}
            # dt_bias puts softplus(dt) near the synthetic workload's step sizes
            w["dt_bias"] = (torch.rand((s.heads,), generator=gen, device=device) * 2.0 - 4.0)
            self.weights.append(w)
            lw = synth.Mamba2Workload(f"stack_layer{li}", batch=s.batch, heads=s.heads,
                                      head_dim=s.head_dim, state_dim=s.state_dim, groups=s.groups,
                                      k=s.k, dtype="bf16", seed=seed * 1009 + li)
            A, D = synth.mamba2_params(lw)
            h0 = torch.from_numpy(synth.mamba2_state0(lw)).to(device)
            cfg = make_config(kind="mamba2", mode=mode, batch=s.batch, heads=s.heads,
                              head_dim=s.head_dim, state_dim=s.state_dim, groups=s.groups, k=s.k,
                              in_dtype="bf16", read_fmt=read_fmt, ckpt_dtype=ckpt)
            self.layers.append(Layer(cfg, torch.from_numpy(A).to(device), torch.from_numpy(D).to(device),
                                     h0))
        self.y = torch.empty((s.batch, 1, s.heads, s.head_dim), dtype=torch.bfloat16, device=device)

    def close(self):
        for layer in self.layers:
            layer.close()

    def step(self, u):
        """One decode step of every layer for the embeddings u [B][d_model]
        (bf16); returns the last layer's hidden state."""
        import torch
        import torch.nn.functional as F
        s = self.shape
        for w, layer in zip(self.weights, self.layers):
            uf = u.float()
            n = (uf * torch.rsqrt(uf.pow(2).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
            x = n @ w["x"]
            z = n @ w["z"]
            Bt = n @ w["B"]
            Ct = n @ w["C"]
            dt = F.softplus((n @ w["dt"]).float() + w["dt_bias"]).to(torch.bfloat16)
            layer.decode_step(self.y, 1, x=x, Bm=Bt, C=Ct, dt=dt)
            g = self.y.view(s.batch, s.d_inner) * F.silu(z)
            u = u + g @ w["out"]
        return u

    def ssm_inputs(self, u):
        """The SSM layers' inputs (x, B, C, dt) for the embeddings u, per layer,
        with u passed through unchanged (to time the SSM layers alone)."""
        import torch
        import torch.nn.functional as F
        out = []
        for w in self.weights:
            uf = u.float()
            n = (uf * torch.rsqrt(uf.pow(2).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
            dt = F.softplus((n @ w["dt"]).float() + w["dt_bias"]).to(torch.bfloat16)
            out.append((n @ w["x"], n @ w["B"], n @ w["C"], dt))
        return out


@dataclass(frozen=True)
class HybridShape:
    """A hybrid stack: `pattern` gives its layers in order, "M" a Mamba-2 layer
    and "A" an attention layer over a paged cache of `num_pages` pages."""
    pattern: str
    batch: int
    heads: int = 128               # Mamba-2: H, P, N, G, k
    head_dim: int = 64
    state_dim: int = 128
    groups: int = 8
    k: int = 16
    q_heads: int = 32              # attention
    kv_heads: int = 8
    attn_dim: int = 128
    page_size: int = 16
    num_pages: int = 4096
    max_pages: int = 512           # of one request
    window: int = 0
    max_draft: int = 1             # tokens a request may draft per step

    @property
    def d_inner(self) -> int:
        return self.heads * self.head_dim

    @property
    def d_model(self) -> int:
        return self.d_inner // 2


class HybridStack:
    """Mamba-2 and attention layers with random projections on one GPU, one
    decode step (or one round of drafts) at a time.

    For the residual stream u [B][T][d_model] (FP32), and layer after layer:

        u, n = add_norm(u, o)                  o: the layer before's output
        "M":  x, z, Bt, Ct, dt as in M2Stack;  y = SSM decode step
              o = gated_norm(y, z) W_out       normalised in G groups of d_inner
        "A":  q, k, v = n W_qkv;  with rope: q, k rotated to the tokens' positions
              k, v to the requests' new slots of the cache
              o = attention(q) W_o             over all tokens of the request

    All requests share one page table, which every attention layer's cache is
    laid out by. kv: "bf16", "fp8" or "nvfp4" (unit scales). rope: a Rope, or None
    for no positions. The weights depend on `seed` only. A request begins with no
    tokens.
    """

    def __init__(self, shape: HybridShape, kv="bf16", seed=0, device="cuda", rope=None):
        import torch
        s = self.shape = shape
        if not s.pattern or set(s.pattern) - {"M", "A"}:
            raise ValueError(f"pattern: {s.pattern!r}, must be of M and A")
        if kv not in ("bf16", "fp8", "nvfp4"):
            raise ValueError(f"kv: {kv!r}, must be bf16, fp8 or nvfp4")
        if rope is not None and "A" in s.pattern:
            # here, and not in a step's append, when the page table has grown already
            if rope.rotary_dim > s.attn_dim:
                raise ValueError(f"rope: {rope.rotary_dim} rotated channels, heads have {s.attn_dim}")
            on = torch.empty(0, device=device).device
            if rope.turns.device != on:
                raise ValueError(f"rope: on {rope.turns.device}, must be on {on}")
        self.rope = rope
        gen = torch.Generator(device=device)
        gen.manual_seed(2000 + seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device=device, dtype=torch.float32)
            return (w / rows ** 0.5).to(torch.bfloat16)

        def norm(n):
            return 1 + 0.1 * torch.randn((n,), generator=gen, device=device, dtype=torch.float32)

        self.pages = PageTable(s.batch, s.page_size, s.num_pages, s.max_pages, device=device)
        self.weights, self.layers = [], []
        workspace = None
        for li, kind in enumerate(s.pattern):
            w = {"norm": norm(s.d_model)}
            if kind == "M":
                w.update(x=weight(s.d_model, s.d_inner), z=weight(s.d_model, s.d_inner),
                         B=weight(s.d_model, s.groups * s.state_dim), C=weight(s.d_model, s.groups * s.state_dim),
                         dt=weight(s.d_model, s.heads), out=weight(s.d_inner, s.d_model), gate=norm(s.d_inner))
                w["dt_bias"] = torch.rand((s.heads,), generator=gen, device=device) * 2.0 - 4.0
                lw = synth.Mamba2Workload(f"stack_layer{li}", batch=s.batch, heads=s.heads, head_dim=s.head_dim,
                                          state_dim=s.state_dim, groups=s.groups, k=s.k, dtype="bf16",
                                          seed=seed * 1009 + li)
                A, D = synth.mamba2_params(lw)
                cfg = make_config(kind="mamba2", batch=s.batch, heads=s.heads, head_dim=s.head_dim,
                                  state_dim=s.state_dim, groups=s.groups, k=s.k, max_draft=s.max_draft)
                self.layers.append(Layer(cfg, torch.from_numpy(A).to(device), torch.from_numpy(D).to(device)))
            else:
                w.update(qkv=weight(s.d_model, (s.q_heads + 2 * s.kv_heads) * s.attn_dim),
                         out=weight(s.q_heads * s.attn_dim, s.d_model))
                dtype = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "nvfp4": torch.uint8}[kv]
                row = s.attn_dim if kv != "nvfp4" else s.attn_dim // 2 + s.attn_dim // 16
                cache = torch.zeros((s.num_pages, 2, s.kv_heads, s.page_size, row), dtype=dtype, device=device)
                ones = torch.ones((s.kv_heads,), device=device) if kv != "bf16" else None
                layer = Attention(cache[:, 0], cache[:, 1], batch=s.batch, q_heads=s.q_heads, max_pages=s.max_pages,
                                  max_draft=s.max_draft, window=s.window, k_scale=ones, v_scale=ones, workspace=workspace)
                workspace = layer.workspace           # the layers run one after another: one workspace
                self.layers.append(layer)
            self.weights.append(w)
        self.final_norm = norm(s.d_model)
        self.buffers = {}

    def close(self):
        for layer in self.layers:
            layer.close()
        self.pages.close()

    def _buffers(self, T, device):
        import torch
        if T not in self.buffers:
            s, n = self.shape, self.shape.batch * T
            bf16, f32 = torch.bfloat16, torch.float32

            def new(dtype, *shape):
                return torch.empty(shape, dtype=dtype, device=device)

            self.buffers[T] = {"u": new(f32, n, s.d_model), "n": new(bf16, n, s.d_model), "y": new(bf16, n, s.d_inner),
                               "g": new(bf16, n, s.d_inner), "o": new(bf16, s.batch, T, s.q_heads, s.attn_dim),
                               "slots": new(torch.int32, n), "positions": new(torch.int32, n)}
        return self.buffers[T]

    def step(self, u):
        """One decode step for u [B][d_model], or a round of T drafts a request for
        [B][T][d_model] (float32); returns the final norm's output, bf16, of the
        same shape. A round of T > 1 drafts must be followed by verify. Where the
        page table refuses a request (errors, pages.refused), its output is of no
        use: verify turns a round's drafts down everywhere, but a single step's
        token has gone into its SSM layers, and the request must be ended."""
        import torch
        import torch.nn.functional as F
        s = self.shape
        T = 1 if u.dim() == 2 else u.shape[1]
        n_tok = s.batch * T
        b = self._buffers(T, u.device)
        self.pages.extend(b["slots"], T=T, positions=b["positions"] if self.rope else None)
        b["u"].copy_(u.reshape(n_tok, s.d_model))
        res, n, out = b["u"], b["n"], None
        for w, layer, kind in zip(self.weights, self.layers, s.pattern):
            add_norm(n, res, w["norm"], x=out, u_out=None if out is None else res)
            if kind == "M":
                dt = F.softplus((n @ w["dt"]).float() + w["dt_bias"]).to(torch.bfloat16)
                layer.decode_step(b["y"], T, x=n @ w["x"], Bm=n @ w["B"], C=n @ w["C"], dt=dt)
                gated_norm(b["g"], b["y"], n @ w["z"], w["gate"], group=s.d_inner // s.groups)
                out = b["g"] @ w["out"]
            else:
                qkv = (n @ w["qkv"]).view(n_tok, s.q_heads + 2 * s.kv_heads, s.attn_dim)
                q, k, v = qkv.split([s.q_heads, s.kv_heads, s.kv_heads], dim=1)
                if self.rope:
                    layer.append(k, v, b["slots"], rope=self.rope, positions=b["positions"], q=q, q_out=q)
                else:
                    layer.append(k, v, b["slots"])
                layer.decode(b["o"], q, self.pages.lens, self.pages.table, T=T)
                out = b["o"].view(n_tok, -1) @ w["out"]
        final = torch.empty_like(n)
        add_norm(final, res, self.final_norm, x=out)
        return final.view(u.shape)

    def verify(self, T, accepted):
        """After a round of T > 1 drafts: accepted[b] of them stay (device int32);
        none of a request that the page table refused."""
        kept = accepted * (1 - self.pages.refused)
        for layer, kind in zip(self.layers, self.shape.pattern):
            if kind == "M":
                layer.verify_rollback(kept)
        self.pages.rollback(T, accepted)

    def errors(self):
        """The error words of the page table and of every layer (synchronises)."""
        return [self.pages.get_error()] + [layer.get_error() for layer in self.layers]
