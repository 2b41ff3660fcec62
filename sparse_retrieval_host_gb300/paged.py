"""Paged 8-bit KV cache: requests of different lengths over one pool of blocks.

``PagedKV8`` owns a library handle (scratch, error word), the block table, the
request lengths, the stack of free blocks and, per layer, the pools of e4m3
codes and block scales (or adopts the caller's tensors). One serving step is

    cu, pos, slot = cache.resize(new_len, n_new)       # block tables, positions, slots
    q, k = cache.norm_rope(q, k, pos=pos, ...)         # RMS norm + rotation
    cache.append(k, v, cu)                             # rows into the cache
    out = cache.attend(q, cu, scale=...)               # attention over it

and ``resize`` with shorter lengths gives rejected drafted tokens back. All work
runs in the library's kernels (kv8_* of include/srh.h); PyTorch allocates
tensors and names streams. Calls on one cache are ordered by the caller. A call
on a ``stream`` of its own waits for nothing on the current one; the tensors that it
is given may be let go as soon as it returns.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import abi

_STYLES = {"pairs": abi.KV8_ROPE_PAIRS, "halves": abi.KV8_ROPE_HALVES}
_BF16 = (torch.bfloat16, torch.int16)      # int16: bf16 bit patterns, as DecodeStep holds them


def _public_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle without making a Stream object (2 us of a 10 us call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)


class PagedKV8:
    """Cache of ``layers`` layers for up to ``batch`` requests of up to
    ``max_blocks * block_tokens`` tokens each.

    ``shared_kv``: rows are latent rows, V = K (one pool per layer).
    ``buffers``: tensors to use instead of new ones, by name: ``table`` int32
    [batch][max_blocks], ``len`` int32 [batch], ``free`` int32 [n_blocks],
    ``n_free`` int32 [1], and for a one-layer cache ``k_codes`` / ``v_codes``
    uint8 [n_blocks][n_kv_heads][block_tokens][head_dim] (blocks may be strided),
    ``k_scale`` / ``v_scale`` fp32 [n_blocks][n_kv_heads].
    """

    def __init__(self, *, batch: int, n_kv_heads: int, head_dim: int, block_tokens: int, n_blocks: int, max_blocks: int,
                 shared_kv: bool = False, layers: int = 1, device: str = "cuda", buffers: Optional[dict] = None):
        self.cache = None
        buf = dict(buffers or {})
        if layers < 1:
            raise ValueError("layers must be >= 1")
        if layers > 1 and any(k in buf for k in ("k_codes", "k_scale", "v_codes", "v_scale")):
            raise ValueError("pools can be given for a one-layer cache only")
        if shared_kv and (buf.get("v_codes") is not buf.get("k_codes") or buf.get("v_scale") is not buf.get("k_scale")):
            if "v_codes" in buf or "v_scale" in buf:
                raise ValueError("a shared cache has one pool")
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError("the cache lives on a CUDA device")
        self.device = torch.device("cuda", torch.cuda.current_device() if dev.index is None else dev.index)
        self.batch, self.Hk, self.D, self.bs = batch, n_kv_heads, head_dim, block_tokens
        self.n_blocks, self.max_blocks, self.shared = n_blocks, max_blocks, bool(shared_kv)
        shape = (n_blocks, n_kv_heads, block_tokens, head_dim)
        stride = 0
        for name in ("k_codes", "v_codes"):
            t = buf.get(name)
            if t is None:
                continue
            inner = (block_tokens * head_dim, head_dim, 1)
            if t.dtype != torch.uint8 or tuple(t.shape) != shape or t.stride()[1:] != inner or t.device != self.device:
                raise ValueError(f"{name} must be uint8 {shape} on {self.device}, dense within a block")
            if n_blocks > 1 and t.stride(0) < t[0].numel():
                raise ValueError(f"{name}: blocks must not overlap")
            if stride and n_blocks > 1 and t.stride(0) != stride:
                raise ValueError("k_codes and v_codes must have the same block stride")
            stride = t.stride(0) if n_blocks > 1 else 0
        cfg = abi.Kv8Config(batch, n_kv_heads, head_dim, block_tokens, n_blocks, max_blocks, int(self.shared), stride)
        with torch.cuda.device(self.device):
            self.cache = abi.kv8_create(cfg)

        def tensor(name, shp, dtype, make):
            t = buf.get(name)
            if t is None:
                return make()
            if t.dtype != dtype or tuple(t.shape) != tuple(shp) or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{name} must be a dense {dtype} {tuple(shp)} on {self.device}")
            return t

        i32 = dict(dtype=torch.int32, device=self.device)
        self.table = tensor("table", (batch, max_blocks), torch.int32, lambda: torch.full((batch, max_blocks), -1, **i32))
        self.len = tensor("len", (batch,), torch.int32, lambda: torch.zeros(batch, **i32))
        # block 0 is on top of the stack
        self.free = tensor("free", (n_blocks,), torch.int32,
                           lambda: torch.arange(n_blocks - 1, -1, -1, **i32))
        self.n_free = tensor("n_free", (1,), torch.int32, lambda: torch.full((1,), n_blocks, **i32))
        self.k_codes, self.k_scale, self.v_codes, self.v_scale, self._pool = [], [], [], [], []
        for _ in range(layers):
            for part, codes, scale in (("k", self.k_codes, self.k_scale), ("v", self.v_codes, self.v_scale)):
                if part == "v" and self.shared:
                    codes.append(self.k_codes[-1])
                    scale.append(self.k_scale[-1])
                    continue
                c = buf.get(part + "_codes")
                if c is None:
                    # the block stride of a given pool holds for both
                    width = stride or n_kv_heads * block_tokens * head_dim
                    c = torch.zeros((n_blocks, width), dtype=torch.uint8, device=self.device)
                    c = c[:, :n_kv_heads * block_tokens * head_dim].view(shape)
                codes.append(c)
                scale.append(tensor(part + "_scale", (n_blocks, n_kv_heads), torch.float32,
                                    lambda: torch.ones((n_blocks, n_kv_heads), device=self.device)))
            pool = abi.Kv8Pool(self.k_codes[-1].data_ptr(), self.k_scale[-1].data_ptr(),
                               self.v_codes[-1].data_ptr(), self.v_scale[-1].data_ptr())
            self._pool.append(ctypes.byref(pool))
        # what every call passes, taken once: the cache's own tensors stay where they are
        self._lib = abi.load()
        self._index = self.device.index
        self._table, self._len = self.table.data_ptr(), self.len.data_ptr()
        self._free, self._n_free = self.free.data_ptr(), self.n_free.data_ptr()

    # ------------------------------------------------------------------ checks
    def _raise(self, rc: int, where: str) -> None:
        raise abi.SrhError(rc, where, self._lib.kv8_last_error(self.cache).decode(errors="replace"))

    def _s(self, stream) -> int:
        if stream is None:
            return _current_stream(self.device.index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _empty(self, shape, dtype, stream) -> torch.Tensor:
        """A new output of a call on ``stream``: its memory belongs to that stream."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        s = torch.cuda.ExternalStream(stream, self.device) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _keep(self, stream, *tensors) -> None:
        """Memory of a call's tensors is not handed out again before ``stream`` is through with them."""
        s = torch.cuda.ExternalStream(stream, self.device) if isinstance(stream, int) else stream
        for t in tensors:
            if t is not None:
                t.record_stream(s)

    def _rows(self, t: torch.Tensor, name: str, heads: Optional[int] = None, dim: Optional[int] = None) -> int:
        """Row stride (elements) of a bf16 [rows][heads][dim] tensor with dense rows."""
        if t.dtype not in _BF16 or t.dim() != 3 or t.get_device() != self._index:
            raise ValueError(f"{name} must be bf16 [rows][heads][dim] on {self.device}")
        n, h, d = t.shape
        if (heads is not None and h != heads) or (dim is not None and d != dim):
            raise ValueError(f"{name} must have {heads} heads of {dim}")
        st = t.stride()
        if (d > 1 and st[2] != 1) or (h > 1 and st[1] != d):
            raise ValueError(f"{name}: the heads of a row must be dense")
        return st[0] if n > 1 else h * d

    def _ints(self, t: torch.Tensor, name: str, n: Optional[int] = None, dtype=torch.int32) -> None:
        if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name} must be a dense 1-d {dtype} on {self.device}")
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name} must have {n} entries")

    def _requests(self, cu: torch.Tensor) -> int:
        self._ints(cu, "cu")
        n = cu.shape[0] - 1
        if not 1 <= n <= self.batch:
            raise ValueError("cu must have an entry per request and one more")
        return n

    # ------------------------------------------------------------------ the step
    def resize(self, new_len: torch.Tensor, n_new: int = 0, *, out=None, stream=None):
        """Requests 0 .. len(new_len)-1 to ``new_len`` tokens (int32, on the GPU),
        blocks taken or given back. ``n_new``: room for new tokens (their number,
        or more). Returns ``cu`` int32 [n + 1] and, with ``n_new``, ``pos`` int32 and
        ``slot`` int64 of the new tokens (else None, None); ``out`` gives the
        three tensors to write. Slots behind the last new token (all of them after
        a refusal) are negative. Asynchronous; see kv8_resize for refusals."""
        self._ints(new_len, "new_len")
        n = new_len.shape[0]
        if not 1 <= n <= self.batch:
            raise ValueError("new_len must have 1 .. batch entries")
        if n_new < 0:
            raise ValueError("n_new must be >= 0")
        if out is None:
            cu = self._empty(n + 1, torch.int32, stream)
            pos = self._empty(n_new, torch.int32, stream) if n_new else None
            slot = self._empty(n_new, torch.int64, stream) if n_new else None
        else:
            cu, pos, slot = out
            self._ints(cu, "cu", n + 1)
            if n_new:
                self._ints(pos, "pos", n_new)
                self._ints(slot, "slot", n_new, torch.int64)
            else:
                pos = slot = None
        rc = self._lib.kv8_resize(self.cache, new_len.data_ptr(), n, self._len, self._table, self._free, self._n_free,
                                  cu.data_ptr(), pos.data_ptr() if n_new else None, slot.data_ptr() if n_new else None,
                                  n_new, self._s(stream))
        if rc:
            self._raise(rc, "kv8_resize")
        if stream is not None:
            self._keep(stream, new_len, cu, pos, slot)
        return cu, pos, slot

    def norm_rope(self, q: Optional[torch.Tensor] = None, k: Optional[torch.Tensor] = None, *, pos=None, inv_freq=None,
                  rot_dim: int = 0, rot_off: int = 0, style: str = "pairs", eps: float = 1e-6, q_weight=None, k_weight=None,
                  q_out=None, k_out=None, q_slot=None, k_slot=None, stream=None):
        """RMS norm of every head of ``q`` and ``k`` (bf16 [tokens][heads][dim]; either
        may be None) and rotation of dims [rot_off, rot_off + rot_dim) by
        ``pos`` * ``inv_freq`` (fp64 [rot_dim / 2]). ``*_slot`` (int64): token t's
        row goes to row slot[t] of ``*_out`` (negative: nowhere), which is then
        required. Returns (q_out, k_out)."""
        if style not in _STYLES:
            raise ValueError("style must be pairs or halves")
        first = q if q is not None else k
        if first is None or first.dim() != 3:
            raise ValueError("q or k must be bf16 [tokens][heads][dim]")
        n, _, d = first.shape
        if rot_dim:
            if pos is None or inv_freq is None:
                raise ValueError("rot_dim needs pos and inv_freq")
            self._ints(pos, "pos", n)
            self._ints(inv_freq, "inv_freq", rot_dim // 2, torch.float64)
        parts, outs = [], []
        for x, w, out, slot, name in ((q, q_weight, q_out, q_slot, "q"), (k, k_weight, k_out, k_slot, "k")):
            if x is None:
                parts.append(None)
                outs.append(None)
                continue
            row = self._rows(x, name, None, d)
            if x.shape[0] != n:
                raise ValueError("q and k must have the same tokens")
            if w is not None and (w.dtype != torch.float32 or tuple(w.shape) != (d,) or not w.is_contiguous()
                                  or w.device != self.device):
                raise ValueError(f"{name}_weight must be fp32 [{d}] on {self.device}")
            if slot is not None:
                self._ints(slot, name + "_slot", n, torch.int64)
                if out is None:
                    raise ValueError(f"{name}_slot needs {name}_out")
            if out is None:
                out, out_row = self._empty(x.shape, x.dtype, stream), x.shape[1] * d
            else:
                out_row = self._rows(out, name + "_out", x.shape[1], d)
                if slot is None and out.shape[0] != n:
                    raise ValueError(f"{name}_out must have a row per token")
            parts.append(abi.Kv8Heads(x.data_ptr(), row, out.data_ptr(), out_row, None if w is None else w.data_ptr(),
                                      x.shape[1], None if slot is None else slot.data_ptr(),
                                      0 if slot is None else out.shape[0]))
            outs.append(out)
        if n:
            rc = self._lib.kv8_norm_rope(self.cache, parts[0], parts[1], n, d, pos.data_ptr() if rot_dim else None,
                                         inv_freq.data_ptr() if rot_dim else None, rot_dim, rot_off, _STYLES[style], eps,
                                         self._s(stream))
            if rc:
                self._raise(rc, "kv8_norm_rope")
            if stream is not None:
                self._keep(stream, q, k, pos, inv_freq, q_weight, k_weight, q_slot, k_slot, *outs)
        return outs[0], outs[1]

    def append(self, k: torch.Tensor, v: Optional[torch.Tensor], cu: torch.Tensor, *, layer: int = 0, stream=None) -> None:
        """The last ``cu[b+1] - cu[b]`` tokens of each request from rows ``cu[b]`` .. of
        ``k`` and ``v`` (bf16 [rows][n_kv_heads][head_dim]; ``v`` None when shared)."""
        n = self._requests(cu)
        kr = self._rows(k, "k", self.Hk, self.D)
        if (v is None) != self.shared:
            raise ValueError("v is given exactly when the cache is not shared")
        vr = 0
        if v is not None:
            vr = self._rows(v, "v", self.Hk, self.D)
            if v.shape[0] != k.shape[0]:
                raise ValueError("k and v must have the same rows")
        if k.shape[0]:
            rc = self._lib.kv8_append(self.cache, self._pool[layer], self._table, self._len, cu.data_ptr(), n, k.data_ptr(),
                                      kr, None if v is None else v.data_ptr(), vr, k.shape[0], self._s(stream))
            if rc:
                self._raise(rc, "kv8_append")
            if stream is not None:
                self._keep(stream, k, v, cu)

    def attend(self, q: torch.Tensor, cu: torch.Tensor, *, scale: float, window: int = 0, out=None, layer: int = 0,
               stream=None) -> torch.Tensor:
        """Attention of each request's last ``cu[b+1] - cu[b]`` tokens (rows of ``q``,
        bf16 [rows][heads][head_dim]) over its cache, causal, with an optional
        window. Rows of ``out`` behind the last request are left as they are."""
        n = self._requests(cu)
        qr = self._rows(q, "q", None, self.D)
        if out is None:
            out, orow = self._empty(q.shape, q.dtype, stream), q.shape[1] * self.D
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        else:
            orow = self._rows(out, "out", None, self.D)
        if q.shape[0]:
            rc = self._lib.kv8_attend(self.cache, self._pool[layer], self._table, self._len, cu.data_ptr(), n, q.data_ptr(),
                                      qr, q.shape[0], q.shape[1], scale, window, out.data_ptr(), orow, self._s(stream))
            if rc:
                self._raise(rc, "kv8_attend")
            if stream is not None:
                self._keep(stream, q, cu, out)
        return out

    # ------------------------------------------------------------------ status
    def check_error(self) -> int:
        """Waits for the device; the sticky error word as a code (kv8_check_error)."""
        return abi.kv8_check_error(self.cache)

    def close(self) -> None:
        if getattr(self, "cache", None):
            abi.kv8_destroy(self.cache)
            self.cache = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass
