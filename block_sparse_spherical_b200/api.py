"""torch-tensor front end of the BSA C ABI.

PyTorch supplies device memory and the current stream; each call marshals
tensors into one C-ABI call (abi.py) and the kernels in libbsa.so do all the
work. Inputs must be contiguous CUDA tensors in the layouts of include/bsa.h.
"""
from __future__ import annotations

import torch

from . import abi


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return abi.BSA_BF16
    if t.dtype == torch.float32:
        return abi.BSA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _require(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def config_for(q: torch.Tensor, block_size: int, top_n: int, window_blocks: int = 1,
               scale: float = 0.0) -> abi.BsaConfig:
    b, h, n, d = q.shape
    return abi.BsaConfig(b, h, n, d, block_size, top_n, window_blocks, _dtype_code(q), scale)


class BSA:
    """A BSA forward pass of fixed shape with its workspace held on the device.

    Calling the object runs pool -> compress/select -> fine attention on the
    current stream (three kernels) and returns `out` ([B, H, N, d], q's dtype).
    """

    def __init__(self, batch: int, heads: int, n_tokens: int, head_dim: int, block_size: int,
                 top_n: int, window_blocks: int = 1, dtype=torch.bfloat16, scale: float = 0.0,
                 device="cuda"):
        self.cfg = abi.BsaConfig(batch, heads, n_tokens, head_dim, block_size, top_n, window_blocks,
                                 abi.BSA_BF16 if dtype == torch.bfloat16 else abi.BSA_F32, scale)
        self.shape = (batch, heads, n_tokens, head_dim)
        self.dtype = dtype
        self.m = n_tokens // block_size
        self.workspace_bytes = abi.bsa_workspace_size(self.cfg)
        self.workspace = torch.zeros(self.workspace_bytes, dtype=torch.uint8, device=device)
        self.sel_idx = torch.empty((batch, heads, self.m, top_n), dtype=torch.int32, device=device)

    @classmethod
    def from_config(cls, cfg, device="cuda", scale: float = 0.0) -> "BSA":
        return cls(cfg.batch, cfg.heads, cfg.n_tokens, cfg.head_dim, cfg.block_size, cfg.top_n,
                   cfg.window_blocks, torch.bfloat16 if cfg.dtype == "bf16" else torch.float32, scale,
                   device)

    def __call__(self, q, k, v, gates, out=None) -> torch.Tensor:
        for name, t in (("q", q), ("k", k), ("v", v)):
            _require(t, name, self.dtype, self.shape)
        _require(gates, "gates", torch.float32, self.shape[:3] + (3,))
        if out is None:
            out = torch.empty_like(q)
        _require(out, "out", self.dtype, self.shape)
        abi.bsa_forward(self.cfg, q, k, v, gates, out, self.sel_idx, self.workspace, self.workspace_bytes)
        return out

    def check_status(self) -> int:
        """Synchronise and return the kernels' status code (0 = OK); resets it."""
        return abi.bsa_check_status(self.workspace)


class BSAStream:
    """BSA forwards over a sequence of batches held in pinned host memory, with the host-device
    copies overlapped with the computation.

    run(batches, outs) enqueues, for batch i: its inputs copied in on a copy stream into device
    buffer set i % 2, the forward (bsa_forward) on a compute stream, and its output copied back on
    a third stream into outs[i]; so batch i+1's inputs move in and batch i-1's output moves out
    while batch i computes. Events order the reuse of each buffer set (inputs: after the forward
    two batches back has read them; output: after the copy-out two batches back has read it).
    run returns once everything is enqueued; synchronize() waits for it. The host tensors must
    stay alive and unchanged until then. The device buffers (and the layer's workspace and index
    array) are marked as used by the streams that touch them, so that memory freed with this object
    is not handed out again while a copy or a forward on one of them is still pending.
    """

    def __init__(self, layer: BSA):
        self.layer = layer
        dev = layer.workspace.device
        b, h, n, d = layer.shape
        self.streams = [torch.cuda.Stream(dev) for _ in range(3)]   # copy in, compute, copy out
        self.bufs = [dict(q=torch.empty(layer.shape, dtype=layer.dtype, device=dev),
                          k=torch.empty(layer.shape, dtype=layer.dtype, device=dev),
                          v=torch.empty(layer.shape, dtype=layer.dtype, device=dev),
                          gates=torch.empty((b, h, n, 3), dtype=torch.float32, device=dev),
                          out=torch.empty(layer.shape, dtype=layer.dtype, device=dev)) for _ in range(2)]
        for buf in self.bufs:
            for t in buf.values():
                for st in self.streams:
                    t.record_stream(st)
        layer.workspace.record_stream(self.streams[1])
        layer.sel_idx.record_stream(self.streams[1])
        self.in_done = [torch.cuda.Event() for _ in range(2)]
        self.cmp_done = [torch.cuda.Event() for _ in range(2)]
        self.out_done = [torch.cuda.Event() for _ in range(2)]
        self._used = [False, False]

    def run(self, batches, outs) -> None:
        s_in, s_cmp, s_out = self.streams
        for i, ((q, k, v, gates), o) in enumerate(zip(batches, outs)):
            for name, t in (("q", q), ("k", k), ("v", v), ("gates", gates), ("out", o)):
                if t.is_cuda or not t.is_pinned():
                    raise ValueError(f"{name} of batch {i} must be a pinned host tensor")
            j = i % 2
            buf = self.bufs[j]
            with torch.cuda.stream(s_in):
                if self._used[j]:
                    s_in.wait_event(self.cmp_done[j])
                for name, t in (("q", q), ("k", k), ("v", v), ("gates", gates)):
                    buf[name].copy_(t, non_blocking=True)
                self.in_done[j].record(s_in)
            with torch.cuda.stream(s_cmp):
                s_cmp.wait_event(self.in_done[j])
                if self._used[j]:
                    s_cmp.wait_event(self.out_done[j])
                self.layer(buf["q"], buf["k"], buf["v"], buf["gates"], out=buf["out"])
                self.cmp_done[j].record(s_cmp)
            with torch.cuda.stream(s_out):
                s_out.wait_event(self.cmp_done[j])
                o.copy_(buf["out"], non_blocking=True)
                self.out_done[j].record(s_out)
            self._used[j] = True

    def synchronize(self) -> None:
        for st in self.streams:
            st.synchronize()


class BSATrain(BSA):
    """A BSA layer of fixed shape for training: forward() saves what backward() needs.

    forward(q, k, v, gates) -> out; backward(dout) -> (dq, dk, dv, dgates), with the
    selected blocks held fixed. bf16, block 64, head_dim 64. The saved tensors and
    both workspaces live on the device between the two calls.
    """

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        b, h, n, d = self.shape
        dev = self.workspace.device
        self.o_cg = torch.empty((b, h, self.m, d), dtype=torch.float32, device=dev)
        self.lse_cg = torch.empty((b, h, self.m), dtype=torch.float32, device=dev)
        self.o_fg = torch.empty(self.shape, dtype=self.dtype, device=dev)
        self.o_l = torch.empty(self.shape, dtype=self.dtype, device=dev)
        self.lse_fine = torch.empty((b, h, n, 2), dtype=torch.float32, device=dev)
        self.bwd_workspace_bytes = abi.bsa_backward_workspace_size(self.cfg)
        self.bwd_workspace = torch.zeros(self.bwd_workspace_bytes, dtype=torch.uint8, device=dev)
        self._saved = None

    def __call__(self, q, k, v, gates, out=None) -> torch.Tensor:
        return self.forward(q, k, v, gates, out)

    def forward(self, q, k, v, gates, out=None) -> torch.Tensor:
        for name, t in (("q", q), ("k", k), ("v", v)):
            _require(t, name, self.dtype, self.shape)
        _require(gates, "gates", torch.float32, self.shape[:3] + (3,))
        if out is None:
            out = torch.empty_like(q)
        _require(out, "out", self.dtype, self.shape)
        abi.bsa_forward_train(self.cfg, q, k, v, gates, out, self.sel_idx, self.o_cg, self.lse_cg, self.o_fg,
                              self.o_l, self.lse_fine, self.workspace, self.workspace_bytes)
        self._saved = (q, k, v, gates)
        return out

    def backward(self, dout, grads=None):
        """Gradients (dq, dk, dv, dgates) of the last forward() for dL/dout = dout."""
        if self._saved is None:
            raise RuntimeError("backward() needs a forward() first")
        q, k, v, gates = self._saved
        _require(dout, "dout", self.dtype, self.shape)
        if grads is None:
            grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(gates))
        dq, dk, dv, dg = grads
        abi.bsa_backward(self.cfg, q, k, v, gates, dout, self.sel_idx, self.o_cg, self.lse_cg, self.o_fg, self.o_l,
                         self.lse_fine, dq, dk, dv, dg, self.bwd_workspace, self.bwd_workspace_bytes)
        return dq, dk, dv, dg

    def check_backward_status(self) -> int:
        """Synchronise and return the backward kernels' status code (0 = OK); resets it."""
        return abi.bsa_check_status(self.bwd_workspace)


class LatLonToHealpix:
    """Cross-attention interpolation from a lat-lon grid to the HEALPix NESTED pixels at nside.

    The plan (16 neighbours and relative positions per pixel) is built once on the
    device; calling the object with k_src, v_src [B, nlat*nlon, d] (bf16 or fp32) and
    the query map wq [d, 3] (fp32) returns [B, 12*nside^2, d].
    """

    def __init__(self, nside: int, nlat: int, nlon: int, device="cuda"):
        self.nside, self.nlat, self.nlon = nside, nlat, nlon
        self.npix = 12 * nside * nside
        self.nbr = torch.empty((self.npix, 16), dtype=torch.int32, device=device)
        self.rel = torch.empty((self.npix, 16, 3), dtype=torch.float32, device=device)
        abi.bsa_latlon_healpix_plan(nside, nlat, nlon, self.nbr, self.rel)
        self._ws = None            # the keys' 3-float position-space images, sized on first use

    def __call__(self, k_src, v_src, wq, scale: float = 0.0, out=None, status_word=None):
        b, n_src, d = k_src.shape
        if n_src != self.nlat * self.nlon:
            raise ValueError(f"k_src must hold {self.nlat * self.nlon} grid points, got {n_src}")
        _require(k_src, "k_src")
        _require(v_src, "v_src", k_src.dtype, k_src.shape)
        _require(wq, "wq", torch.float32, (d, 3))
        if out is None:
            out = torch.empty((b, self.npix, d), dtype=k_src.dtype, device=k_src.device)
        _require(out, "out", k_src.dtype, (b, self.npix, d))
        need = abi.bsa_latlon_workspace_size(b, n_src)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=k_src.device)
        abi.bsa_latlon_to_healpix(b, self.npix, n_src, d, _dtype_code(k_src), scale, self.nbr, self.rel, wq, k_src,
                                  v_src, out, self._ws, self._ws.numel(), status_word)
        return out


def _raw_stream(index: int) -> int:
    """The current stream of a device (the cheap way, where this torch has it: it is asked in every call)."""
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get is not None else torch.cuda.current_stream(index).cuda_stream


class _DenseLayer:
    """What the layers of fixed sizes below share: their device, status word and calls on it.

    A call runs on the layer's device and that device's current stream, whichever device is current.
    Workspaces come from torch's allocator anew in each call (on that stream, or from a capturing
    graph's own pool), so that one layer may be called from several streams and graphs at once.
    """

    def __init__(self, batch, heads, kv_heads, head_dim, dtype, scale, device):
        # float32 is a type of the library that these operators lack: the C call refuses it (BSA_ERR_UNSUPPORTED)
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"dtype must be bfloat16, got {dtype}")
        self.kv_heads = heads if kv_heads is None else kv_heads
        self.dtype, self.scale = dtype, scale
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = self.status.device
        if not self.status.is_cuda:
            raise ValueError(f"the layer needs a CUDA device, got {device}")
        self._status_ptr = self.status.data_ptr()
        self._code = abi.BSA_BF16 if dtype == torch.bfloat16 else abi.BSA_F32

    def _take(self, t, name, shape, dtype=None) -> int:
        """The address of a tensor of the layer's device, of this shape and dtype, contiguous."""
        dtype = self.dtype if dtype is None else dtype
        try:                                # what a good tensor passes at once
            if t.shape == shape and t.dtype is dtype and t.device == self.device and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:
            pass
        _require(t, name, dtype, shape)
        raise ValueError(f"{name} must be on {self.device}, got {t.device}")

    def _lengths(self, t, name, count):
        return None if t is None else self._take(t, name, (count,), torch.int32)

    def _output(self, t, name, shape, like):
        """An output of the caller's, or a new one like an input that was checked, and its address."""
        if t is None:
            t = torch.empty_like(like)
            return t, t.data_ptr()
        return t, self._take(t, name, shape)

    def _run(self, call, args, workspace_bytes):
        """One call of the C ABI on the layer's device and its current stream, with a workspace."""
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self._run(call, args, workspace_bytes)
        ws = torch.empty(workspace_bytes, dtype=torch.uint8, device=self.device) if workspace_bytes else None
        call(self.cfg, *args, None if ws is None else ws.data_ptr(), workspace_bytes, self._status_ptr,
             _raw_stream(self.device.index))

    def _capturing(self) -> bool:
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return torch.cuda.is_current_stream_capturing()
        return torch.cuda.is_current_stream_capturing()

    def check_status(self) -> int:
        """Synchronise the device (a layer's calls may be on any of its streams) and return the kernels'
        status code (0 = OK); resets it."""
        torch.cuda.synchronize(self.device)
        with torch.cuda.device(self.device):
            return abi.bsa_check_status(self.status)


class CrossAttention(_DenseLayer):
    """Attention of n_q query rows a head to an encoder's n_k states (include/bsa.h: bsa_cross_attention).

    Calling the object with q [B, H, n_q, d], k and v [B, H_kv, n_k, d] (bf16, d 64 or 128, H a multiple
    of H_kv) and, for a padded batch, key_len [B] (int32, 0 to n_k) returns out [B, H, n_q, d]. States
    behind key_len are never used; a batch entry without states gives zero rows.
    """

    def __init__(self, batch: int, heads: int, n_q: int, n_k: int, head_dim: int, kv_heads: int | None = None,
                 dtype=torch.bfloat16, scale: float = 0.0, device="cuda"):
        super().__init__(batch, heads, kv_heads, head_dim, dtype, scale, device)
        self.cfg = abi.BsaCrossConfig(batch, heads, self.kv_heads, n_q, n_k, head_dim, self._code, scale)
        self.workspace_bytes = abi.bsa_cross_workspace_size(self.cfg)
        self.batch = batch
        self.shape = (batch, heads, n_q, head_dim)
        self.kv_shape = (batch, self.kv_heads, n_k, head_dim)

    def _forward(self, q, k, v, key_len, out, lse=None, low=None):
        args = (self._take(q, "q", self.shape), self._take(k, "k", self.kv_shape), self._take(v, "v", self.kv_shape),
                self._lengths(key_len, "key_len", self.batch))
        out, address = self._output(out, "out", self.shape, q)
        self._run(abi.bsa_cross_attention, (*args, address, *(None if t is None else t.data_ptr() for t in (lse, low))),
                  self.workspace_bytes)
        return out

    def __call__(self, q, k, v, key_len=None, out=None) -> torch.Tensor:
        return self._forward(q, k, v, key_len, out)


class CrossAttentionTrain(CrossAttention):
    """A CrossAttention layer for training.

    forward(q, k, v, key_len) -> out; backward(dout) -> (dq, dk, dv) of the last forward(). Its q, k, v,
    key_len and out are kept by reference until then and have to stay as they are (and with them, of
    the layer's own, the rows' log-sum-exp and what rounding out to bf16 left off). A backward() captured
    into a graph reads them in every replay: what a forward() outside of a capture saved is then kept as
    long as the layer is.
    """

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.bwd_workspace_bytes = abi.bsa_cross_backward_workspace_size(self.cfg)
        self._saved = self._stream = None
        self._captured = False
        self._replayed = []                 # what captured backwards read and no graph's memory pool holds

    def __call__(self, q, k, v, key_len=None, out=None) -> torch.Tensor:
        return self.forward(q, k, v, key_len, out)

    def forward(self, q, k, v, key_len=None, out=None) -> torch.Tensor:
        lse = torch.empty(self.shape[:3], dtype=torch.float32, device=self.device)
        low = torch.empty(self.shape, dtype=self.dtype, device=self.device)
        out = self._forward(q, k, v, key_len, out, lse, low)
        self._saved, self._stream = (q, k, v, key_len, out, lse, low), _raw_stream(self.device.index)
        self._captured = self._capturing()
        return out

    def backward(self, dout, grads=None):
        """Gradients (dq, dk, dv) of the last forward() for dL/dout = dout; into `grads` where it gives them."""
        if self._saved is None:
            raise RuntimeError("backward() needs a forward() first")
        saved = self._saved
        if _raw_stream(self.device.index) != self._stream:
            # a later forward() drops these, and may hold the last reference to any of them: their memory must not
            # be handed out before this call has read it
            for t in saved:
                if t is not None:
                    t.record_stream(torch.cuda.current_stream(self.device))
        if not self._captured and self._capturing():
            self._replayed.append(saved)
        grads = tuple(grads or (None,) * 3)
        if len(grads) != 3:                 # the C call takes its arguments by position
            raise ValueError(f"grads must be dq, dk and dv, got {len(grads)} of them")
        outs = [self._output(t, name, shape, like) for t, name, shape, like in
                zip(grads, ("dq", "dk", "dv"), (self.shape, self.kv_shape, self.kv_shape), saved)]
        args = (*(None if t is None else t.data_ptr() for t in saved), self._take(dout, "dout", self.shape),
                *(address for _, address in outs))
        self._run(abi.bsa_cross_attention_backward, args, self.bwd_workspace_bytes)
        return tuple(t for t, _ in outs)


class PrefixAttention(_DenseLayer):
    """Attention of an ensemble's members to a prefix they share and to states of their own, in one
    softmax (include/bsa.h: bsa_prefix_attention).

    The batch is `groups` ensembles of batch / groups consecutive members. Calling the object with q
    [B, H, n_q, d], k_prefix and v_prefix [groups, H_kv, n_prefix, d], k_own and v_own [B, H_kv, n_own, d]
    (bf16) and, where buffers are not full, prefix_len [groups] and own_len [B] (int32, 0 allowed) returns
    [B, H, n_q, d]. The prefix is read once for a group's members together.
    """

    def __init__(self, batch: int, heads: int, n_q: int, n_prefix: int, n_own: int, head_dim: int,
                 kv_heads: int | None = None, groups: int = 1, dtype=torch.bfloat16, scale: float = 0.0,
                 device="cuda"):
        super().__init__(batch, heads, kv_heads, head_dim, dtype, scale, device)
        self.cfg = abi.BsaPrefixConfig(batch, groups, heads, self.kv_heads, n_q, n_prefix, n_own, head_dim,
                                       self._code, scale)
        self.workspace_bytes = abi.bsa_prefix_workspace_size(self.cfg)
        self.batch, self.groups = batch, groups
        self.shape = (batch, heads, n_q, head_dim)
        self.prefix_shape = (groups, self.kv_heads, n_prefix, head_dim)
        self.own_shape = (batch, self.kv_heads, n_own, head_dim)

    def __call__(self, q, k_prefix, v_prefix, k_own, v_own, prefix_len=None, own_len=None,
                 out=None) -> torch.Tensor:
        args = (self._take(q, "q", self.shape), self._take(k_prefix, "k_prefix", self.prefix_shape),
                self._take(v_prefix, "v_prefix", self.prefix_shape),
                self._lengths(prefix_len, "prefix_len", self.groups), self._take(k_own, "k_own", self.own_shape),
                self._take(v_own, "v_own", self.own_shape), self._lengths(own_len, "own_len", self.batch))
        out, address = self._output(out, "out", self.shape, q)
        self._run(abi.bsa_prefix_attention, (*args, address), self.workspace_bytes)
        return out


def forward(q, k, v, gates, block_size: int, top_n: int, window_blocks: int = 1, scale: float = 0.0,
            return_indices: bool = False):
    """One-shot BSA forward (allocates a workspace; use BSA for repeated calls)."""
    b, h, n, d = q.shape
    bsa = BSA(b, h, n, d, block_size, top_n, window_blocks, q.dtype, scale, q.device)
    out = bsa(q, k, v, gates)
    return (out, bsa.sel_idx) if return_indices else out


def pool(q, k, v, block_size: int):
    """Block means of q, k, v -> three float32 tensors [B, H, m, d]."""
    b, h, n, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, q.dtype, q.shape)
    cfg = config_for(q, block_size, 1, 0)
    outs = [torch.empty((b, h, n // block_size, d), dtype=torch.float32, device=q.device) for _ in range(3)]
    abi.bsa_pool(cfg, q, k, v, *outs)
    return tuple(outs)


def compress_select(qbar, kbar, vbar, top_n: int, block_size: int, dtype=torch.bfloat16,
                    scale: float = 0.0):
    """Compressed branch + top-n from pooled tensors -> (o_cg_block [B,H,m,d], sel_idx [B,H,m,n])."""
    b, h, m, d = qbar.shape
    for name, t in (("qbar", qbar), ("kbar", kbar), ("vbar", vbar)):
        _require(t, name, torch.float32, qbar.shape)
    cfg = abi.BsaConfig(b, h, m * block_size, d, block_size, top_n, 0,
                        abi.BSA_BF16 if dtype == torch.bfloat16 else abi.BSA_F32, scale)
    o_cg = torch.empty_like(qbar)
    idx = torch.empty((b, h, m, top_n), dtype=torch.int32, device=qbar.device)
    abi.bsa_compress_select(cfg, qbar, kbar, vbar, o_cg, idx)
    return o_cg, idx


def fine_attention(q, k, v, gates, o_cg_block, sel_idx, block_size: int, window_blocks: int = 1,
                   scale: float = 0.0, status_word=None, out=None):
    """Selection + local branches and gated combine from given o_cg_block and sel_idx."""
    b, h, n, d = q.shape
    top_n = sel_idx.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, q.dtype, q.shape)
    _require(gates, "gates", torch.float32, (b, h, n, 3))
    _require(o_cg_block, "o_cg_block", torch.float32, (b, h, n // block_size, d))
    _require(sel_idx, "sel_idx", torch.int32, (b, h, n // block_size, top_n))
    cfg = config_for(q, block_size, top_n, window_blocks, scale)
    if out is None:
        out = torch.empty_like(q)
    abi.bsa_fine_attention(cfg, q, k, v, gates, o_cg_block, sel_idx, out, status_word)
    return out
