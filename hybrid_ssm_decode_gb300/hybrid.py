"""The attention side of a hybrid decode step on torch CUDA tensors: the page
table of a batch (``PageTable``), an attention layer over a paged cache
(``Attention``), and the norms around a block (``add_norm``, ``gated_norm``).

Each call checks its tensors' type, device (the current one), shape and strides,
and then makes one call of the C ABI (include/rssm.h) on the given stream, or torch's
current one. Nothing here synchronises or copies; a ValueError names the argument that
does not fit, and an RssmError a status of the library.

A decode step makes these calls by the dozen, and a kernel of theirs takes a few
microseconds, so what the checks conclude (strides, a filled configuration
struct) is kept by what they looked at: the tensors' types, devices, shapes and
strides, never their addresses. A call with a signature seen before is a look-up
and the C call.
"""
from __future__ import annotations

import hybrid_ssm_decode_gb300 as _r


_KEPT = 512          # signatures kept per kind of call


def _torch():
    import torch
    return torch


def _sig(t):
    """What the checks look at of a tensor (or None)."""
    return None if t is None else (t.dtype, t.get_device(), t.shape, t.stride())


def _keep(store, key, value):
    if len(store) >= _KEPT:
        store.clear()
    store[key] = value
    return value


def _raw_stream(device_index):
    """torch's current stream on a device, as an address."""
    torch = _torch()
    return torch.cuda.current_stream(device_index).cuda_stream


def _current_device():
    return _torch().cuda.current_device()


def _stream_of(stream, device_index):
    """The stream of a call on tensors of a device, which has to be the current
    one: the library launches there."""
    if device_index != _current_device():
        raise ValueError(f"tensors on cuda:{device_index}, but the current device is cuda:{_current_device()}")
    if stream is None:
        return _raw_stream(device_index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _bind():
    """The library's functions and torch's raw queries, once both are loaded."""
    global _lib, _raw_stream, _current_device
    if _lib is None:
        _lib = _r.load()
        raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            _raw_stream = raw
        _current_device = getattr(_torch()._C, "_cuda_getDevice", _current_device)
    return _lib


_lib = None


_DTYPES: dict = {}


def _dtype(t, name):
    """RSSM_F32 / RSSM_BF16 of a tensor."""
    if not _DTYPES:
        torch = _torch()
        _DTYPES.update({torch.float32: _r.RSSM_F32, torch.bfloat16: _r.RSSM_BF16})
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: dtype {t.dtype}, must be float32 or bfloat16")
    return d


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _cuda(device, name):
    _need(device.type == "cuda", f"{name}: on {device}, must be a CUDA device")


def _on(t, device, name):
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, must be on {device}")


def _ints(t, n, device, name):
    """A dense int32 vector of n entries."""
    torch = _torch()
    _on(t, device, name)
    _need(t.dtype == torch.int32 and t.numel() == n and t.is_contiguous(), f"{name}: must be {n} dense int32")


class PageTable:
    """The pages of a batch of requests (rssm_pages_*).

    `lens`, `table`, `free_count` and `refused` are views of the workspace, which
    the library alone writes: they are read where an attention layer wants them.
    `refused` (int32 [batch]) is 1 for a request whose last extend found no room.
    """

    def __init__(self, batch, page_size, num_pages, max_pages, free=None, device="cuda", stream=None):
        torch = _torch()
        self.handle = 0
        self.cfg = _r.PagesConfig(batch, page_size, num_pages, max_pages)
        self.layout = _r.rssm_pages_layout_for(self.cfg)
        self.workspace = torch.empty(self.layout.total_bytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device
        _cuda(self.device, "device")
        if free is not None:
            _ints(free, num_pages, self.device, "free")
        self._fn = _bind()
        self.handle = _r.rssm_pages_create(self.cfg, self.workspace, self.layout.total_bytes, free,
                                           _stream_of(stream, self.device.index))
        lay = self.layout

        def view(off, *shape):
            n = 1
            for s in shape:
                n *= s
            return self.workspace[off:off + 4 * n].view(torch.int32).view(*shape)

        self._seen = {}
        self.lens = view(lay.lens, batch)
        self.table = view(lay.table, batch, max_pages)
        self.free_count = view(lay.free_count, 1)
        self.refused = view(lay.refused, batch)

    def close(self):
        if self.handle:
            _r.rssm_pages_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def extend(self, slots, T=0, new=None, positions=None, stream=None):
        """Room for T tokens more in every request, or new[b] (int32, device)
        in request b; writes the new tokens' slots (and positions)."""
        key = (_sig(slots), _sig(new), _sig(positions), T == 0)
        n = self._seen.get(key)
        if n is None:
            _need((T == 0) != (new is None), "extend: give either T or new")
            n = slots.numel()
            _ints(slots, n, self.device, "slots")
            if positions is not None:
                _ints(positions, n, self.device, "positions")
            if new is not None:
                _ints(new, self.cfg.batch, self.device, "new")
            _keep(self._seen, key, n)
        st = self._fn.rssm_pages_extend(self.handle, T, None if new is None else new.data_ptr(), slots.data_ptr(),
                                        None if positions is None else positions.data_ptr(), n,
                                        _stream_of(stream, self.device.index))
        if st:
            _r._check("rssm_pages_extend", st)

    def rollback(self, T, accepted, stream=None):
        """Of the last T tokens of request b, accepted[b] stay; a request whose
        extend was refused stays as it is."""
        self._counts(accepted, "accepted")
        st = self._fn.rssm_pages_rollback(self.handle, T, accepted.data_ptr(), _stream_of(stream, self.device.index))
        if st:
            _r._check("rssm_pages_rollback", st)

    def truncate(self, keep, stream=None):
        """Cut request b to keep[b] tokens (0 ends it)."""
        self._counts(keep, "keep")
        st = self._fn.rssm_pages_truncate(self.handle, keep.data_ptr(), _stream_of(stream, self.device.index))
        if st:
            _r._check("rssm_pages_truncate", st)

    def _counts(self, t, name):
        key = _sig(t)
        if key not in self._seen:
            _ints(t, self.cfg.batch, self.device, name)
            _keep(self._seen, key, True)

    def get_error(self, stream=None):
        return _r.rssm_pages_get_error(self.handle, _stream_of(stream, self.device.index))


def _tokens(t, n, heads, dim, dtype, device, name):
    """Elements between consecutive tokens of t, [n][heads][dim] or any shape
    whose leading dimensions fold to n without a copy."""
    _on(t, device, name)
    _need(t.dtype == dtype, f"{name}: dtype {t.dtype}, must be {dtype}")
    if t.dim() < 3:
        _need(t.dim() == 2 and t.shape == (n, heads * dim) and t.stride(1) == 1,
              f"{name}: shape {tuple(t.shape)}, must be {(n, heads, dim)}")
        _need(n <= 1 or t.stride(0) >= heads * dim, f"{name}: tokens overlap")
        return t.stride(0) if n > 1 else heads * dim
    sh, st = t.shape, t.stride()
    _need(sh[-1] == dim and sh[-2] == heads and t.numel() == n * heads * dim,
          f"{name}: shape {tuple(sh)}, must be {(n, heads, dim)}")
    _need((st[-1] == 1 or dim == 1) and (st[-2] == dim or heads == 1), f"{name}: a token's heads must be dense")
    step, span = None, 1                    # the leading dimensions, from the inside
    for i in range(t.dim() - 3, -1, -1):
        if sh[i] == 1:
            continue
        if step is None:
            step = st[i]
        elif st[i] != step * span:
            raise ValueError(f"{name}: tokens must be evenly spaced")
        span *= sh[i]
    _need(step is None or step >= heads * dim, f"{name}: tokens overlap")
    return heads * dim if step is None else step


class Attention:
    """One attention layer over paged caches [num_pages][kv_heads][page_size][head_dim]
    (rssm_attn_*): float32 caches with float32 inputs, bfloat16 or
    float8_e4m3fn ones with bfloat16 inputs; float8 caches need k_scale and
    v_scale (float32 [kv_heads]). The caches may be slices of one tensor along
    a page ([num_pages][2][kv_heads]...).

    workspace: a uint8 tensor that layers on one stream share; None allocates
    one (`workspace_size` gives the bytes).
    """

    def __init__(self, k_cache, v_cache, batch, q_heads, max_pages, max_draft=1, window=0, scale=0.0, in_dtype=None,
                 k_scale=None, v_scale=None, workspace=None, stream=None):
        torch = _torch()
        self.handle = 0
        kinds = {torch.float32: (_r.RSSM_F32, "f32"), torch.bfloat16: (_r.RSSM_BF16, "bf16"),
                 torch.float8_e4m3fn: (_r.RSSM_KV_FP8, "bf16")}
        _need(k_cache.dtype in kinds, f"k_cache: dtype {k_cache.dtype}")
        kv, io = kinds[k_cache.dtype]
        io = in_dtype or io
        _need(io in _r.DTYPE, f"in_dtype: {io}")
        _need(k_cache.dim() == 4, "k_cache: must be [num_pages][kv_heads][page_size][head_dim]")
        pages, heads, ps, dim = k_cache.shape
        self.device = k_cache.device
        _cuda(self.device, "k_cache")
        for c, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _on(c, self.device, name)
            _need(c.dtype == k_cache.dtype and c.shape == k_cache.shape, f"{name}: k_cache and v_cache must be alike")
            _need(c.stride()[1:] == (ps * dim, dim, 1), f"{name}: a page must be dense")
        _need(k_cache.stride(0) == v_cache.stride(0) or pages == 1, "k_cache and v_cache: page strides differ")
        _need(k_cache.stride(0) >= heads * ps * dim or pages == 1, "k_cache and v_cache: pages overlap")
        fp8 = kv == _r.RSSM_KV_FP8
        for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _need((s is not None) == fp8, f"{name}: given for float8 caches, and only for them")
            if s is not None:
                _on(s, self.device, name)
                _need(s.dtype == torch.float32 and s.numel() == heads and s.is_contiguous(), f"{name}: must be {heads} dense float32")
        self.cfg = _r.AttnConfig(batch=batch, q_heads=q_heads, kv_heads=heads, head_dim=dim, page_size=ps,
                                 num_pages=pages, max_pages=max_pages, max_draft=max_draft, in_dtype=_r.DTYPE[io],
                                 kv_dtype=kv, window=window, scale=scale,
                                 page_stride=k_cache.stride(0) if pages > 1 else 0)
        self.dtype = torch.float32 if io == "f32" else torch.bfloat16
        need = _r.rssm_attn_workspace_size(self.cfg)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        _on(workspace, self.device, "workspace")
        _need(workspace.is_contiguous(), "workspace: must be dense")
        self.workspace = workspace
        self._tensors = (k_cache, v_cache, k_scale, v_scale)
        self._seen = {}
        self._fn = _bind()
        self.handle = _r.rssm_attn_create(self.cfg, k_cache, v_cache, k_scale, v_scale, workspace,
                                          workspace.numel() * workspace.element_size(),
                                          _stream_of(stream, self.device.index))

    def close(self):
        if self.handle:
            _r.rssm_attn_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, k, v, slots, stream=None):
        """Write the new tokens' keys and values ([tokens][kv_heads][head_dim],
        slices of a wider projection too) to their slots."""
        key = (_sig(k), _sig(v), _sig(slots))
        seen = self._seen.get(key)
        if seen is None:
            c, n = self.cfg, slots.numel()
            _ints(slots, n, self.device, "slots")
            seen = _keep(self._seen, key, (n, _tokens(k, n, c.kv_heads, c.head_dim, self.dtype, self.device, "k"),
                                           _tokens(v, n, c.kv_heads, c.head_dim, self.dtype, self.device, "v")))
        st = self._fn.rssm_attn_append(self.handle, seen[0], k.data_ptr(), seen[1], v.data_ptr(), seen[2],
                                       slots.data_ptr(), _stream_of(stream, self.device.index))
        if st:
            _r._check("rssm_attn_append", st)

    def decode(self, out, q, lens, table, T=1, lse=None, stream=None):
        """The attention of T new tokens a request: q and out
        [batch][T][q_heads][head_dim] (q may be a slice of a wider projection)."""
        key = (T, _sig(out), _sig(q), _sig(lens), _sig(table), _sig(lse))
        step = self._seen.get(key)
        if step is None:
            step = _keep(self._seen, key, self._check_decode(out, q, lens, table, T, lse))
        st = self._fn.rssm_attn_decode(self.handle, T, q.data_ptr(), step, lens.data_ptr(), table.data_ptr(),
                                       out.data_ptr(), None if lse is None else lse.data_ptr(),
                                       _stream_of(stream, self.device.index))
        if st:
            _r._check("rssm_attn_decode", st)

    def _check_decode(self, out, q, lens, table, T, lse):
        torch = _torch()
        c = self.cfg
        n = c.batch * T
        step = _tokens(q, n, c.q_heads, c.head_dim, self.dtype, self.device, "q")
        _ints(lens, c.batch, self.device, "lens")
        _ints(table, c.batch * c.max_pages, self.device, "table")
        _on(out, self.device, "out")
        _need(out.dtype == self.dtype and out.numel() == n * c.q_heads * c.head_dim and out.is_contiguous(),
              f"out: must be a dense {self.dtype} [{c.batch}][{T}][{c.q_heads}][{c.head_dim}]")
        if lse is not None:
            _on(lse, self.device, "lse")
            _need(lse.dtype == torch.float32 and lse.numel() == n * c.q_heads and lse.is_contiguous(),
                  f"lse: must be a dense float32 [{c.batch}][{T}][{c.q_heads}]")
        return step

    def get_error(self, stream=None):
        return _r.rssm_attn_get_error(self.handle, _stream_of(stream, self.device.index))


def _rows(t, rows, dim, device, name):
    """Elements between the rows of t, whose leading dimensions fold to `rows`."""
    _on(t, device, name)
    if t.dim() == 2:
        sh, st = t.shape, t.stride()
        if sh[1] == dim and sh[0] == rows and (st[1] == 1 or dim == 1):
            _need(rows <= 1 or st[0] >= dim, f"{name}: rows overlap")
            return st[0] if rows > 1 else dim
    _need(t.numel() == rows * dim and t.shape[-1] == dim, f"{name}: shape {tuple(t.shape)}, must hold {(rows, dim)}")
    _need(t.is_contiguous(), f"{name}: rows must be evenly spaced and dense")
    return dim


def _by_ref(cfg):
    return _r.ctypes.byref(cfg)


def _weights(w, n, device, name):
    _on(w, device, name)
    _need(w.dtype == _torch().float32 and w.numel() == n and w.is_contiguous(), f"{name}: must be {n} dense float32")


_add_seen: dict = {}


def add_norm(n_out, u, w, x=None, u_out=None, w_post=None, gate=None, scale=1.0, eps=1e-6, w_offset=0.0, stream=None):
    """u_out = u + scale * gate * post(x) and n_out = rmsnorm(u_out) * w (rssm_add_norm).

    u, u_out [rows][dim] float32 or bfloat16; x, gate, n_out [rows][dim] of one
    such type; gate may be [dim], the same for all rows; w, w_post float32
    [dim]. u_out may be u, n_out may be x; u_out or n_out may be None.
    """
    key = (_sig(u), _sig(n_out), _sig(w), _sig(x), _sig(u_out), _sig(w_post), _sig(gate), scale, eps, w_offset)
    cfg = _add_seen.get(key)
    if cfg is None:
        cfg = _keep(_add_seen, key, _check_add(n_out, u, w, x, u_out, w_post, gate, scale, eps, w_offset))
    st = _lib.rssm_add_norm(cfg, u.data_ptr(), None if x is None else x.data_ptr(),
                            None if w_post is None else w_post.data_ptr(), None if gate is None else gate.data_ptr(),
                            None if w is None else w.data_ptr(), None if u_out is None else u_out.data_ptr(),
                            None if n_out is None else n_out.data_ptr(), _stream_of(stream, u.get_device()))
    if st:
        _r._check("rssm_add_norm", st)


def _check_add(n_out, u, w, x, u_out, w_post, gate, scale, eps, w_offset):
    """The configuration struct of add_norm, by reference."""
    _bind()
    dim = u.shape[-1]
    rows = u.numel() // dim if dim else 0
    dev = u.device
    _cuda(dev, "u")
    cfg = _r.AddNormConfig(rows=rows, dim=dim, res_dtype=_dtype(u, "u"), eps=eps, scale=scale, w_offset=w_offset,
                           u_stride=_rows(u, rows, dim, dev, "u"))
    kind = None
    for t, name, field in ((x, "x", "x_stride"), (n_out, "n_out", "n_out_stride")):
        if t is None:
            continue
        d = _dtype(t, name)
        _need(kind in (None, d), "x and n_out: must have one dtype")
        kind = d
        setattr(cfg, field, _rows(t, rows, dim, dev, name))
    cfg.dtype = cfg.res_dtype if kind is None else kind
    if u_out is not None:
        _need(u_out.dtype == u.dtype, "u_out: must have u's dtype")
        cfg.u_out_stride = _rows(u_out, rows, dim, dev, "u_out")
    if gate is not None:
        _need(_dtype(gate, "gate") == cfg.dtype, "gate: must have x's dtype")
        if gate.dim() == 1:
            _on(gate, dev, "gate")
            _need(gate.numel() == dim and (gate.stride(0) == 1 or dim == 1), f"gate: must be {dim} dense values")
        else:
            cfg.gate_stride = _rows(gate, rows, dim, dev, "gate")
    for t, name in ((w, "w"), (w_post, "w_post")):
        if t is not None:
            _weights(t, dim, dev, name)
    return _by_ref(cfg)


_gated_seen: dict = {}


def gated_norm(out, y, z, w, group=None, norm_first=False, act="silu", eps=1e-6, w_offset=0.0, stream=None):
    """The norm after an SSM mixer, with its gate (rssm_gated_norm).

    norm_first=False: rmsnorm(y * act(z)) * w in groups of `group` columns
    (the Mamba-2 block); True: rmsnorm(y) * w * act(z) (the Gated DeltaNet
    block, one group per head). y, z, out [rows][dim] of one type; w float32
    [dim] or [group]. out may be y.
    """
    key = (_sig(y), _sig(z), _sig(out), _sig(w), group, norm_first, act, eps, w_offset)
    cfg = _gated_seen.get(key)
    if cfg is None:
        cfg = _keep(_gated_seen, key, _check_gated(out, y, z, w, group, norm_first, act, eps, w_offset))
    st = _lib.rssm_gated_norm(cfg, y.data_ptr(), z.data_ptr(), w.data_ptr(), out.data_ptr(),
                              _stream_of(stream, y.get_device()))
    if st:
        _r._check("rssm_gated_norm", st)


def _check_gated(out, y, z, w, group, norm_first, act, eps, w_offset):
    """The configuration struct of gated_norm, by reference."""
    _bind()
    dim = y.shape[-1]
    rows = y.numel() // dim if dim else 0
    dev = y.device
    _cuda(dev, "y")
    d = _dtype(y, "y")
    _need(z.dtype == y.dtype and out.dtype == y.dtype, "z and out: must have y's dtype")
    group = dim if group is None else group
    _need(act in _r.GATE, f"act: {act}, must be one of {sorted(_r.GATE)}")
    _need(w.numel() in (dim, group), f"w: {w.numel()} values, must be {dim} or {group}")
    _weights(w, w.numel(), dev, "w")
    cfg = _r.GatedNormConfig(rows=rows, dim=dim, group=group, w_dim=w.numel(), dtype=d, norm_first=int(norm_first),
                             act=_r.GATE[act], eps=eps, w_offset=w_offset, y_stride=_rows(y, rows, dim, dev, "y"),
                             z_stride=_rows(z, rows, dim, dev, "z"), out_stride=_rows(out, rows, dim, dev, "out"))
    return _by_ref(cfg)
