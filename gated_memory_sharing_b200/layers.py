"""Device-resident layers over the C ABI: a Mamba scan layer that produces the
memory readout M, and Gated Memory Units that reuse it.

These hold the weights and workspaces in torch-allocated device memory and
call the ABI entry points; they do no arithmetic of their own.
"""

from __future__ import annotations

import torch

from . import abi


def io_dtype(io: int) -> torch.dtype:
    return torch.bfloat16 if io == abi.BF16 else torch.float32


def to_device(a, io: int, device="cuda") -> torch.Tensor:
    """float32 numpy array (already rounded to the I/O type) -> device tensor."""
    return torch.from_numpy(a).to(device=device).to(io_dtype(io)).contiguous()


def to_device_f32(a, device="cuda") -> torch.Tensor:
    return torch.from_numpy(a).to(device=device, dtype=torch.float32).contiguous()


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


class ScanLayer:
    """The Mamba layer whose readout is the shared memory M."""

    def __init__(self, w: dict, d_model: int, io: int, device="cuda"):
        self.io = io
        self.dtype = io_dtype(io)
        self.d_inner, self.d_state = w["A"].shape
        self.d_conv = w["conv_w"].shape[1]
        self.dt_rank = w["dt_rank"]
        self.d_model = d_model
        self.conv_w = to_device(w["conv_w"], io, device)
        self.conv_b = to_device(w["conv_b"], io, device)
        self.x_proj_w = to_device(w["x_proj_w"], io, device)
        self.dt_proj_w = to_device(w["dt_proj_w"], io, device)
        self.dt_bias = to_device_f32(w["dt_bias"], device)
        self.A = to_device_f32(w["A"], device)
        self.D = to_device_f32(w["D"], device)
        self.abi_w = abi.make_weights(self.conv_w, self.conv_b, self.x_proj_w, self.dt_proj_w,
                                      self.dt_bias, self.A, self.D)
        self.device = device
        self._ws = {}

    def dims(self, batch: int, seqlen: int) -> abi.Dims:
        return abi.make_dims(batch, seqlen, self.d_model, self.d_inner, self.d_state, self.d_conv,
                             self.dt_rank, self.io)

    def _workspace(self, key, nbytes):
        ws = self._ws.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = workspace(nbytes, self.device)
            self._ws[key] = ws
        return ws

    def new_state(self, batch: int):
        h = torch.zeros(batch, self.d_inner, self.d_state, dtype=torch.float32, device=self.device)
        cs = torch.zeros(batch, self.d_inner, self.d_conv, dtype=self.dtype, device=self.device)
        return h, cs

    def prefill(self, u, ssm_state=None, conv_state=None, M=None, fresh=None, stream=None):
        """u [B, L, Di] -> M [B, L, Di].  Without states (or with fresh=True)
        the prompt starts from zero state; otherwise it continues the given
        states.  States are returned and updated in place."""
        B, L, _ = u.shape
        if fresh is None:
            fresh = ssm_state is None
        if ssm_state is None:
            ssm_state, conv_state = self.new_state(B)
        if M is None:
            M = torch.empty_like(u)
        d = self.dims(B, L)
        ws = self._workspace(("prefill", B, L), abi.sambay_scan_prefill_workspace(d))
        abi.sambay_scan_prefill(self.abi_w, d, u, M, ssm_state, conv_state, fresh, ws, stream)
        return M, ssm_state, conv_state

    def step(self, u_t, ssm_state, conv_state, m_t=None, stream=None):
        """u_t [B, Di] -> m_t [B, Di]; states updated in place."""
        B = u_t.shape[0]
        if m_t is None:
            m_t = torch.empty_like(u_t)
        d = self.dims(B, 1)
        ws = self._workspace(("step", B), abi.sambay_scan_step_workspace(d))
        abi.sambay_scan_step(self.abi_w, d, u_t, m_t, ssm_state, conv_state, ws, stream)
        return m_t


class GMULayer:
    """Y = (M ⊙ SiLU(X W1^T)) W2 (+ X)."""

    def __init__(self, W1, W2, io: int, device="cuda"):
        self.io = io
        self.W1 = to_device(W1, io, device)
        self.W2 = to_device(W2, io, device)
        self.d_inner, self.d_model = W1.shape
        self.device = device
        self._ws = {}

    def dims(self, rows: int) -> abi.Dims:
        return abi.make_dims(rows, 1, self.d_model, self.d_inner, 16, 4, 4, self.io)

    def _workspace(self, key, nbytes):
        ws = self._ws.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = workspace(nbytes, self.device)
            self._ws[key] = ws
        return ws

    def forward(self, X, M, residual=False, Y=None, stream=None):
        rows = X.shape[0]
        if Y is None:
            Y = torch.empty_like(X)
        d = self.dims(rows)
        ws = self._workspace(("fwd", rows), abi.gmu_forward_workspace(d, rows))
        abi.gmu_forward(d, rows, X, M, self.W1, self.W2, X if residual else None, Y, ws, stream)
        return Y

    def step(self, X, M, residual=False, Y=None, stream=None):
        rows = X.shape[0]
        if Y is None:
            Y = torch.empty_like(X)
        d = self.dims(rows)
        ws = self._workspace(("step", rows), abi.gmu_step_workspace(d, rows))
        abi.gmu_step(d, rows, X, M, self.W1, self.W2, X if residual else None, Y, ws, stream)
        return Y


class DecodeChain:
    """One decode token through the scan and a stack of GMU layers that reuse
    its readout: m_t = scan step(u_t); X <- X + GMU_l(X, m_t) for each layer,
    as one sambay_decode_step call (states and X updated in place)."""

    def __init__(self, scan: ScanLayer, gmus):
        self.scan = scan
        self.gmus = list(gmus)
        self.layers = abi.make_gmu_layers([(g.W1, g.W2) for g in self.gmus])
        self._ws = {}

    def step(self, u_t, ssm_state, conv_state, X, m_t=None, stream=None):
        B = u_t.shape[0]
        if m_t is None:
            m_t = torch.empty_like(u_t)
        d = self.scan.dims(B, 1)
        n = len(self.gmus)
        ws = self._ws.get(B)
        need = abi.sambay_decode_step_workspace(d, n)
        if ws is None or ws.numel() < need:
            ws = workspace(need, self.scan.device)
            self._ws[B] = ws
        abi.sambay_decode_step(self.scan.abi_w, d, u_t, m_t, ssm_state, conv_state, self.layers, n,
                               X if n else None, ws, stream)
        return m_t


class MambaLayer:
    """The whole Mamba layer whose scan readout is the shared memory M:
    u = X W_in^T, y = scan(u) (= M), out = (y ⊙ SiLU(X W_z^T)) W_out + X.
    The gated output projection is the GMU's computation with W1 = W_z and
    W2 = W_out, so it runs through gmu_forward / gmu_step."""

    def __init__(self, w: dict, bw: dict, d_model: int, io: int, device="cuda"):
        self.scan = ScanLayer(w, d_model, io, device)
        self.W_in = to_device(bw["W_in"], io, device)
        self.gate = GMULayer(bw["W_z"], bw["W_out"], io, device)
        self.io, self.device = io, device
        self.d_model, self.d_inner = d_model, self.scan.d_inner
        self._ws = {}

    def _proj(self, X2, u2, stream):
        rows = X2.shape[0]
        d = self.gate.dims(rows)
        ws = self._ws.get(rows)
        need = abi.sambay_in_proj_workspace(d, rows)
        if ws is None or ws.numel() < need:
            ws = workspace(need, self.device)
            self._ws[rows] = ws
        abi.sambay_in_proj(d, rows, X2, self.W_in, u2, ws, stream)

    def prefill(self, X, ssm_state=None, conv_state=None, fresh=None, stream=None):
        """X [B, L, Dm] -> (out [B, L, Dm], M [B, L, Di], ssm_state, conv_state)."""
        B, L, Dm = X.shape
        X2 = X.reshape(B * L, Dm)
        u = torch.empty(B, L, self.d_inner, dtype=X.dtype, device=X.device)
        self._proj(X2, u.view(B * L, self.d_inner), stream)
        M, h, cs = self.scan.prefill(u, ssm_state, conv_state, fresh=fresh, stream=stream)
        out = self.gate.forward(X2, M.view(B * L, self.d_inner), residual=True, stream=stream)
        return out.view(B, L, Dm), M, h, cs

    def step(self, x_t, ssm_state, conv_state, stream=None):
        """x_t [B, Dm] -> (out_t [B, Dm], m_t [B, Di]); states updated in place."""
        u_t = torch.empty(x_t.shape[0], self.d_inner, dtype=x_t.dtype, device=x_t.device)
        self._proj(x_t, u_t, stream)
        m_t = self.scan.step(u_t, ssm_state, conv_state, stream=stream)
        out = self.gate.step(x_t, m_t, residual=True, stream=stream)
        return out, m_t


class MLPMemory:
    """SambaY-MLP's memory: the SwiGLU hidden activation SiLU(X W_g^T) ⊙ (X W_u^T)."""

    def __init__(self, W_g, W_u, io: int, device="cuda"):
        self.W_g = to_device(W_g, io, device)
        self.W_u = to_device(W_u, io, device)
        self.d_ff, self.d_model = W_g.shape
        self.io, self.device = io, device
        self._ws = {}

    def forward(self, X, M=None, stream=None):
        rows = X.shape[0]
        if M is None:
            M = torch.empty(rows, self.d_ff, dtype=X.dtype, device=X.device)
        d = abi.make_dims(rows, 1, self.d_model, self.d_ff, 16, 4, 4, self.io)
        ws = self._ws.get(rows)
        need = abi.sambay_mlp_memory_workspace(d, rows)
        if ws is None or ws.numel() < need:
            ws = workspace(need, self.device)
            self._ws[rows] = ws
        abi.sambay_mlp_memory(d, rows, X, self.W_g, self.W_u, M, ws, stream)
        return M


class Mamba2Scan:
    """The SambaY-2 memory: a Mamba-2 (SSD) layer's readout over a prompt."""

    def __init__(self, w: dict, io: int = abi.BF16, device="cuda"):
        self.io = io
        self.dtype = io_dtype(io)
        self.nheads = int(w["A"].shape[0])
        self.headdim = int(w["P"])
        self.d_state = int(w["N"])
        self.channels, self.d_conv = w["conv_w"].shape
        self.conv_w = to_device(w["conv_w"], io, device)
        self.conv_b = to_device(w["conv_b"], io, device)
        self.dt_bias = to_device_f32(w["dt_bias"], device)
        self.A = to_device_f32(w["A"], device)
        self.D = to_device_f32(w["D"], device)
        self.abi_w = abi.SsdWeights(self.conv_w.data_ptr(), self.conv_b.data_ptr(), self.dt_bias.data_ptr(),
                                    self.A.data_ptr(), self.D.data_ptr())
        self.device = device
        self._ws = {}

    def dims(self, batch: int, seqlen: int) -> abi.SsdDims:
        return abi.SsdDims(batch, seqlen, self.nheads, self.headdim, self.d_state, self.d_conv, self.io)

    def new_state(self, batch: int):
        h = torch.zeros(batch, self.nheads, self.headdim, self.d_state, dtype=torch.float32, device=self.device)
        cs = torch.zeros(batch, self.channels, self.d_conv, dtype=self.dtype, device=self.device)
        return h, cs

    def prefill(self, xbc, dt_raw, ssm_state=None, conv_state=None, M=None, fresh=None, stream=None):
        """xbc [B, L, C], dt_raw [B, L, H] -> M [B, L, H * P]; states as for
        ScanLayer.prefill (returned, updated in place)."""
        B, L, _ = xbc.shape
        if fresh is None:
            fresh = ssm_state is None
        if ssm_state is None:
            ssm_state, conv_state = self.new_state(B)
        if M is None:
            M = torch.empty(B, L, self.nheads * self.headdim, dtype=self.dtype, device=self.device)
        d = self.dims(B, L)
        n = abi.sambay_ssd_prefill_workspace(d)
        ws = self._ws.get((B, L))
        if ws is None:
            ws = workspace(n, self.device)
            self._ws[(B, L)] = ws
        abi.sambay_ssd_prefill(self.abi_w, d, xbc, dt_raw, M, ssm_state, conv_state, fresh, ws, stream)
        return M, ssm_state, conv_state

    def step(self, xbc_t, dt_raw_t, ssm_state, conv_state, m_t=None, stream=None):
        """xbc_t [B, C], dt_raw_t [B, H] -> m_t [B, H * P]; states updated in place."""
        B = xbc_t.shape[0]
        if m_t is None:
            m_t = torch.empty(B, self.nheads * self.headdim, dtype=self.dtype, device=self.device)
        d = self.dims(B, 1)
        n = abi.sambay_ssd_step_workspace(d)
        ws = self._ws.get(("step", B))
        if ws is None:
            ws = workspace(n, self.device)
            self._ws[("step", B)] = ws
        abi.sambay_ssd_step(self.abi_w, d, xbc_t, dt_raw_t, m_t, ssm_state, conv_state, ws, stream)
        return m_t


# What a call of the 4-bit cache asks for every time, without torch's wrappers.
_I32 = torch.int32
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


class KV4Cache:
    """The one KV cache of the cross-decoder in 4 bits: rows are quantised as
    they are written (4.5 bits an element), read back, and attended over.

    Pages of ``page_tokens`` tokens from a pool of ``num_pages``; ``table``
    [B, pages a sequence] int32 says which page holds which tokens (by default
    each sequence has its own pages, in order).  The table may be changed in
    place between calls, on the stream of the calls.  ``k_exp`` / ``v_exp``
    [Hkv] int32: the power of two of each head's rows (see :meth:`exponents`),
    fixed for the cache's life.  These tensors and ``pages`` are the cache's own
    (calls use their addresses): another one cannot be put in their place.

    Positions, lengths and counts are int32 tensors on the device.  Indices
    outside the table, the pool or a call's rows are skipped and recorded
    (``abi.sambay_device_status``).  Workspaces come from torch's allocator
    call by call, so calls on different streams and captured graphs share none.
    """

    def __init__(self, batch: int, kv_heads: int, head_dim: int, max_tokens: int, page_tokens: int = 64,
                 io: int = abi.BF16, num_pages=None, table=None, k_exp=None, v_exp=None, device="cuda"):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"the cache lies on a GPU, not on {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        each = -(-max_tokens // page_tokens)
        if table is None:
            if num_pages is None:
                num_pages = batch * each
            if num_pages < batch * each:
                raise ValueError(f"{num_pages} pages are not enough for {batch} sequences of {each} pages: give a table")
            table = torch.arange(batch * each, dtype=torch.int32, device=self.device).view(batch, each)
        elif num_pages is None:
            raise ValueError("a table needs num_pages, the pool's size")
        self._dev = self.device.index
        self.io, self.dtype = io, io_dtype(io)
        self.batch, self.kv_heads, self.head_dim, self.page_tokens = batch, kv_heads, head_dim, page_tokens
        self._own = {"table": table, "k_exp": k_exp, "v_exp": v_exp}
        if table.dim() != 2 or table.shape[0] != batch:
            raise ValueError(f"table is [{batch}, pages]: got {tuple(table.shape)}")
        self._index(table, "table", None)
        for name, e in (("k_exp", k_exp), ("v_exp", v_exp)):
            if e is not None:
                self._index(e, name, kv_heads)
        self.dims = abi.Kv4Dims(batch, kv_heads, head_dim, page_tokens, num_pages, table.shape[1], io)
        nbytes = abi.sambay_kv4_cache_bytes(self.dims)
        if nbytes == 0:
            raise ValueError("unsupported sizes: head_dim 64 or 128, page_tokens a power of two in 16 .. 1024, "
                             "at most 2^30 tokens a sequence")
        with torch.cuda.device(self.device):
            # zeros: a page that was never written reads as zeros
            self._own["pages"] = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.abi_cache = abi.make_kv4_cache(self.pages, table, k_exp, v_exp)
        self._plans, self._row_shapes = {}, set()

    def _fixed(name):
        def put(self, t):
            if t is not self._own[name]:                 # `cache.table += 1` puts the same tensor back
                raise ValueError(f"{name} belongs to the cache: change it in place")
        return property(lambda self: self._own[name], put)

    table, k_exp, v_exp, pages = map(_fixed, ("table", "k_exp", "v_exp", "pages"))
    del _fixed

    @staticmethod
    def exponents(rows) -> torch.Tensor:
        """[Hkv] int32 for rows [..., Hkv, dh]: the least e in -64 .. 64 for
        which the largest of these values is not past what a block can hold,
        2688 * 2^e.  Infinities and NaN do not count: they take their own block
        of 16 values only, not their head."""
        size = rows.detach().abs()
        size = torch.where(torch.isfinite(size), size, 0)
        amax = size.amax(-1).reshape(-1, rows.shape[-2]).amax(0).double()
        e = torch.ceil(torch.log2(torch.clamp(amax, min=2.0 ** -60) / 2688.0))
        return torch.clamp(e, -64, 64).to(torch.int32)

    # ------------------------------------------------------------- checks
    # (a condition that holds costs one expression; what is wrong is found and said by the functions)

    def _index(self, t, name, n):
        if t.dtype is not _I32 or t.get_device() != self._dev or not t.is_contiguous() or (
                n is not None and t.numel() != n):
            raise ValueError(f"{name}: {'' if n is None else n} int32, dense, on {self.device}: "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")

    def _rows(self, t, name, shape, dense=True):
        if t.dtype is not self.dtype or t.get_device() != self._dev or t.shape != shape or (
                dense and not t.is_contiguous()):
            raise ValueError(f"{name}: {self.dtype} {tuple(shape)}{', dense,' if dense else ''} on {self.device}: "
                             f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")

    def _row_shape(self, shape):
        """Takes [B, T, Hkv, dh] in among the shapes that rows may have."""
        if len(shape) != 4 or shape[0] != self.batch or shape[1] < 1 or tuple(shape[2:]) != (self.kv_heads, self.head_dim):
            raise ValueError(f"rows are [{self.batch}, tokens, {self.kv_heads}, {self.head_dim}], got {tuple(shape)}")
        self._row_shapes.add(shape)

    def _stride(self, t, name):
        """Elements between a sequence's consecutive tokens (0: dense); heads
        and values are dense and sequences follow at the same stride."""
        B, T, H, D = t.shape
        s = t.stride()
        token = s[1] if T > 1 else s[0] if B > 1 else H * D
        if s[3] != 1 or (H > 1 and s[2] != D) or (B > 1 and s[0] != T * token) or token < H * D:
            raise ValueError(f"{name}: strides {s} are not [tokens * stride, stride, {D}, 1]")
        return token

    def _on(self, stream):
        """(the stream's handle, what makes the cache's device and the stream
        current, or None where they are)."""
        if stream is None:
            return (_current_stream(self._dev),
                    None if _current_device() == self._dev else torch.cuda.device(self._dev))
        if isinstance(stream, int):
            # (torch takes the handle 0 as a wish for a stream of its pool)
            stream = (torch.cuda.ExternalStream(stream, device=self.device) if stream
                      else torch.cuda.default_stream(self.device))
        if stream.device != self.device:
            raise ValueError(f"a stream of {stream.device} for a cache on {self.device}")
        return stream.cuda_stream, torch.cuda.stream(stream)

    # ------------------------------------------------------------- calls

    def write(self, K, V, pos, count=None, stream=None):
        """Quantise rows K, V [B, T, Hkv, dh] into positions pos[b] .. of each
        sequence (count[b] of them, or all T).  Rows may be slices of wider
        ones (a fused projection's).  Calls that write tokens of the same 16 of
        a sequence (positions 16 j .. 16 j + 15) must be ordered."""
        shape, dtype, dev = K.shape, self.dtype, self._dev
        if shape not in self._row_shapes:
            self._row_shape(shape)
        if K.dtype is not dtype or K.get_device() != dev:
            self._rows(K, "K", shape, False)
        if V.dtype is not dtype or V.get_device() != dev or V.shape != shape:
            self._rows(V, "V", shape, False)
        n = self.batch
        if pos.dtype is not _I32 or pos.get_device() != dev or pos.numel() != n or not pos.is_contiguous():
            self._index(pos, "pos", n)
        if count is not None and (count.dtype is not _I32 or count.get_device() != dev or count.numel() != n
                                  or not count.is_contiguous()):
            self._index(count, "count", n)
        ks = 0 if K.is_contiguous() else self._stride(K, "K")
        vs = 0 if V.is_contiguous() else self._stride(V, "V")
        handle, within = self._on(stream)
        if within is None:
            abi.sambay_kv4_write(self.abi_cache, self.dims, shape[1], K, V, pos, count, ks, vs, handle)
        else:
            with within:
                abi.sambay_kv4_write(self.abi_cache, self.dims, shape[1], K, V, pos, count, ks, vs, handle)

    def read(self, pos, tokens: int, count=None, K=None, V=None, stream=None):
        """The rows K, V [B, tokens, Hkv, dh] that positions pos[b] .. stand
        for (count[b] of them, or all); rows from count[b] on are left as they
        were (zeros in tensors made here)."""
        n, dtype, dev = self.batch, self.dtype, self._dev
        if pos.dtype is not _I32 or pos.get_device() != dev or pos.numel() != n or not pos.is_contiguous():
            self._index(pos, "pos", n)
        if count is not None and (count.dtype is not _I32 or count.get_device() != dev or count.numel() != n
                                  or not count.is_contiguous()):
            self._index(count, "count", n)
        if K is None or V is None:
            shape = torch.Size((self.batch, tokens, self.kv_heads, self.head_dim))
        else:
            shape = K.shape
            if shape[1] != tokens:
                raise ValueError(f"K has {shape[1]} tokens a sequence, not {tokens}")
        if shape not in self._row_shapes:
            self._row_shape(shape)
        if K is not None and (K.dtype is not dtype or K.get_device() != dev or not K.is_contiguous()
                              or K.shape != shape):
            self._rows(K, "K", shape)
        if V is not None and (V.dtype is not dtype or V.get_device() != dev or not V.is_contiguous()
                              or V.shape != shape):
            self._rows(V, "V", shape)
        handle, within = self._on(stream)
        if within is None:
            return self._read(shape, K, V, pos, count, handle)
        with within:
            return self._read(shape, K, V, pos, count, handle)

    def _read(self, shape, K, V, pos, count, handle):
        K = self._made(shape, count) if K is None else K
        V = self._made(shape, count) if V is None else V
        abi.sambay_kv4_read(self.abi_cache, self.dims, shape[1], K, V, pos, count, handle)
        return K, V

    def attend(self, q, lens, count=None, scale: float = 0.0, out=None, stream=None):
        """out [B, T, Hq, dh] for the queries q of the newest T (or count[b])
        of each sequence's lens[b] cached tokens; q [B, Hq, dh] for one token
        a sequence.  Rows from count[b] on are left as they were (zeros in a
        tensor made here)."""
        shape, dtype, dev = q.shape, self.dtype, self._dev
        plan = self._plans.get(shape)
        if plan is None:
            plan = self._plan(shape)
        if q.dtype is not dtype or q.get_device() != dev or not q.is_contiguous():
            self._rows(q, "q", shape)
        if out is not None and (out.dtype is not dtype or out.get_device() != dev or not out.is_contiguous()
                                or out.shape != shape):
            self._rows(out, "out", shape)
        n = self.batch
        if lens.dtype is not _I32 or lens.get_device() != dev or lens.numel() != n or not lens.is_contiguous():
            self._index(lens, "lens", n)
        if count is not None and (count.dtype is not _I32 or count.get_device() != dev or count.numel() != n
                                  or not count.is_contiguous()):
            self._index(count, "count", n)
        handle, within = self._on(stream)
        if within is None:
            return self._attend(plan, q, lens, count, scale, out, handle)
        with within:
            return self._attend(plan, q, lens, count, scale, out, handle)

    def _plan(self, shape):
        """(query heads, tokens, workspace bytes) for queries of this shape."""
        if len(shape) not in (3, 4) or shape[0] != self.batch or shape[-1] != self.head_dim or 0 in shape:
            raise ValueError(f"q: [{self.batch}, tokens, heads, {self.head_dim}] or without tokens, got {tuple(shape)}")
        heads, tokens = shape[-2], shape[1] if len(shape) == 4 else 1
        plan = heads, tokens, abi.sambay_cross_attn_decode_kv4_workspace(self.dims, heads, tokens)
        self._plans[shape] = plan
        return plan

    def _attend(self, plan, q, lens, count, scale, out, handle):
        heads, tokens, ws_bytes = plan
        if out is None:
            out = self._made(q.shape, count)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device) if ws_bytes else None
        abi.sambay_cross_attn_decode_kv4(self.abi_cache, self.dims, heads, tokens, q, out, lens, count, scale, ws,
                                         ws_bytes, handle)
        return out

    def _made(self, shape, count):
        """A new tensor of the current stream (that of the call)."""
        return (torch.empty if count is None else torch.zeros)(shape, dtype=self.dtype, device=self.device)
