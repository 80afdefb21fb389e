"""Torch-facing binding of libmamba2pool.so: argument marshalling only.

Tensors supply device pointers, dtypes and row strides; the stream is
torch's current stream.  Every computation runs in the HIP kernels of the
library, and a missing library raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
from ctypes import byref, c_uint64, c_void_p

import numpy as np
import torch

from ._ffi import M2_BF16, M2_F32, Int8StoreDesc, LayerParams, Mamba2Error, PoolDesc, check, lib

_DT = {torch.float32: M2_F32, torch.bfloat16: M2_BF16}


def _code_of(dtype: torch.dtype) -> int:
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    return _DT[dtype]


def _dtype_code(t: torch.Tensor) -> int:
    return _code_of(t.dtype)


def _rows(t: torch.Tensor, name: str):
    # the stride of a dimension of one element, and every stride of an empty tensor, may be anything
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1 and t.numel() > 0):
        raise ValueError(f"{name} must be a 2-D tensor with a contiguous last dimension")
    return c_void_p(t.data_ptr()), t.stride(0)


def _stream():
    return c_void_p(torch.cuda.current_stream().cuda_stream)


def _host_i32(a):
    if a is None:
        return None, None
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return arr, arr.ctypes.data_as(c_void_p)


class LayerWeights:
    """fp32 device parameters of one layer: A, D, dt_bias [H], conv_w [Cd, W], conv_b [Cd].
    A gated-delta layer has no D and may have no conv_b: pass None."""

    def __init__(self, A, D, dt_bias, conv_w, conv_b):
        self.tensors = [None if t is None else t.contiguous() for t in (A, D, dt_bias, conv_w, conv_b)]
        for t in self.tensors:
            if t is not None and t.dtype != torch.float32:
                raise TypeError("layer parameters must be float32")
        self.A, self.D, self.dt_bias, self.conv_w, self.conv_b = self.tensors
        self.struct = LayerParams(*(None if t is None else t.data_ptr() for t in self.tensors))

    @classmethod
    def from_numpy(cls, p: dict, device="cuda"):
        f = lambda k: torch.as_tensor(np.asarray(p[k], np.float32), device=device)
        return cls(f("A"), f("D"), f("dt_bias"), f("conv_w"), f("conv_b"))


class Pool:
    """Slot pool over caller-owned tensors ssm [L, S, H, P, N] and conv [L, S, Cd, W-1]."""

    def __init__(self, ssm: torch.Tensor, conv: torch.Tensor, nheads: int, head_dim: int, d_state: int,
                 n_groups: int, conv_kernel: int, family: int = 0):
        if not (ssm.is_contiguous() and conv.is_contiguous()):
            raise ValueError("pool tensors must be contiguous")
        self.ssm, self.conv = ssm, conv
        self.nheads, self.head_dim, self.d_state = nheads, head_dim, d_state
        self.n_groups, self.conv_kernel = n_groups, conv_kernel
        self.family = family               # 0: Mamba2, 1: Mamba1 (nheads = D channels, head_dim 1), 2: GDN, 3: KDA
        self.intermediate = nheads * head_dim
        self.conv_dim = self.intermediate + (0 if family == 1 else 2 * n_groups * d_state)
        self.num_layers, self.num_slots = ssm.shape[0], ssm.shape[1]
        desc = PoolDesc(self.num_layers, self.num_slots, nheads, head_dim, d_state, n_groups, conv_kernel,
                        _dtype_code(ssm), _dtype_code(conv), family, ssm.data_ptr(), conv.data_ptr(),
                        ssm.numel() * ssm.element_size(), conv.numel() * conv.element_size())
        h = c_void_p()
        check(lib().mamba2_pool_create(byref(desc), byref(h)))
        self._h = h

    @classmethod
    def allocate(cls, num_layers, num_slots, nheads, head_dim, d_state, n_groups, conv_kernel,
                 ssm_dtype=torch.bfloat16, conv_dtype=torch.bfloat16, device="cuda"):
        cd = nheads * head_dim + 2 * n_groups * d_state
        ssm = torch.zeros((num_layers, num_slots, nheads, head_dim, d_state), dtype=ssm_dtype, device=device)
        conv = torch.zeros((num_layers, num_slots, cd, conv_kernel - 1), dtype=conv_dtype, device=device)
        return cls(ssm, conv, nheads, head_dim, d_state, n_groups, conv_kernel)

    @classmethod
    def allocate_mamba1(cls, num_layers, num_slots, d_inner, d_state, conv_kernel, ssm_dtype=torch.bfloat16,
                        conv_dtype=torch.bfloat16, device="cuda"):
        """A Mamba1 pool: ssm [L, S, D, 1, N] (the (D, N) state) and conv [L, S, D, W-1]."""
        ssm = torch.zeros((num_layers, num_slots, d_inner, 1, d_state), dtype=ssm_dtype, device=device)
        conv = torch.zeros((num_layers, num_slots, d_inner, conv_kernel - 1), dtype=conv_dtype, device=device)
        return cls(ssm, conv, d_inner, 1, d_state, 1, conv_kernel, family=1)

    @classmethod
    def allocate_gdn(cls, num_layers, num_slots, num_v_heads, head_v_dim, head_k_dim, num_k_heads, conv_kernel,
                     device="cuda"):
        """A GDN pool: ssm [L, S, Hv, dv, dk] and conv [L, S, 2*Hk*dk + Hv*dv, W-1] (channels q, k, v),
        both bf16; decoded and prefilled by the gdn_* calls."""
        cd = num_v_heads * head_v_dim + 2 * num_k_heads * head_k_dim
        ssm = torch.zeros((num_layers, num_slots, num_v_heads, head_v_dim, head_k_dim), dtype=torch.bfloat16,
                          device=device)
        conv = torch.zeros((num_layers, num_slots, cd, conv_kernel - 1), dtype=torch.bfloat16, device=device)
        return cls(ssm, conv, num_v_heads, head_v_dim, head_k_dim, num_k_heads, conv_kernel, family=2)

    @classmethod
    def allocate_kda(cls, num_layers, num_slots, num_heads, head_dim, conv_kernel, device="cuda"):
        """A KDA pool (state only: no recurrence here): ssm [L, S, H, d, d] fp32 and conv
        [L, S, 3*H*d, W-1] bf16."""
        ssm = torch.zeros((num_layers, num_slots, num_heads, head_dim, head_dim), dtype=torch.float32, device=device)
        conv = torch.zeros((num_layers, num_slots, 3 * num_heads * head_dim, conv_kernel - 1), dtype=torch.bfloat16,
                           device=device)
        return cls(ssm, conv, num_heads, head_dim, head_dim, num_heads, conv_kernel, family=3)

    def mamba1_decode_step(self, layer: int, w: LayerWeights, slots: torch.Tensor, x, B, C, z, dt, y,
                           slots_host=None):
        """One Mamba1 token per row of slots (device int32): x, z, dt rows of D, B and C rows of N;
        w.A is the (D, N) decay matrix."""
        if slots.dtype != torch.int32:
            raise TypeError("slots must be int32")
        _, sh_ptr = _host_i32(slots_host)
        io = _dtype_code(x)
        for t in (B, C, z, dt):
            if _dtype_code(t) != io:
                raise TypeError("x, B, C, z and dt must share one dtype")
        xp, xs = _rows(x, "x")
        bp, bs = _rows(B, "B")
        cp, cs = _rows(C, "C")
        zp, zs = _rows(z, "z")
        dp, ds = _rows(dt, "dt")
        yp, ys = _rows(y, "y")
        check(lib().mamba1_decode_step(self._h, layer, byref(w.struct), slots.numel(), c_void_p(slots.data_ptr()),
                                       sh_ptr, xp, xs, bp, bs, cp, cs, zp, zs, dp, ds, io, yp, ys,
                                       _dtype_code(y), _stream()))
        return y

    def mamba1_workspace_size(self, num_seqs: int, total_tokens: int, chunk_size: int = 0,
                              max_ckpt: int = 0) -> int:
        n = c_uint64()
        check(lib().mamba1_prefill_workspace_size(self._h, num_seqs, total_tokens, chunk_size, max_ckpt,
                                                  byref(n)))
        return n.value

    def mamba1_prefill(self, layer: int, w: LayerWeights, cu_seqlens, slots, has_init, x, B, C, z, dt, y,
                       start_pos=None, chunk_size: int = 0, ckpt_interval: int = 0, ckpt_slots=None,
                       workspace: torch.Tensor | None = None):
        """Mamba1 prefill of packed sequences (rows x, z, dt of D; B, C of N); cu_seqlens, slots,
        has_init, start_pos and ckpt_slots [num_seqs][max_ckpt] are host arrays; chunk_size 0 lets
        the library choose the chunking."""
        cu, _ = _host_i32(cu_seqlens)
        sl, sl_p = _host_i32(slots)
        hi = np.ascontiguousarray(np.asarray(has_init, dtype=np.uint8))
        sp, sp_p = _host_i32(start_pos)   # sp keeps the array alive through the call
        ns = len(sl)
        max_ck, ck_p = 0, None
        if ckpt_slots is not None:
            ck = np.ascontiguousarray(np.asarray(ckpt_slots, dtype=np.int32).reshape(ns, -1))
            max_ck = ck.shape[1]
            ck_p = ck.ctypes.data_as(c_void_p)
        total = int(cu[-1]) if len(cu) else 0
        if workspace is None:
            workspace = torch.empty(self.mamba1_workspace_size(ns, total, chunk_size, max_ck), dtype=torch.uint8,
                                    device=self.ssm.device)
        io = _dtype_code(x)
        for t in (B, C, z, dt):
            if _dtype_code(t) != io:
                raise TypeError("x, B, C, z and dt must share one dtype")
        xp, xs = _rows(x, "x")
        bp, bs = _rows(B, "B")
        cp, cs = _rows(C, "C")
        zp, zs = _rows(z, "z")
        dp, ds = _rows(dt, "dt")
        yp, ys = _rows(y, "y")
        check(lib().mamba1_prefill(
            self._h, layer, byref(w.struct), ns, cu.ctypes.data_as(c_void_p), sl_p,
            hi.ctypes.data_as(c_void_p), sp_p, xp, xs, bp, bs, cp, cs, zp, zs, dp, ds, io, yp, ys,
            _dtype_code(y), chunk_size, ckpt_interval, ck_p, max_ck, c_void_p(workspace.data_ptr()),
            workspace.numel(), _stream()))
        return y

    def close(self):
        if getattr(self, "_h", None):
            lib().mamba2_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def info(self):
        s, c = c_uint64(), c_uint64()
        check(lib().mamba2_pool_info(self._h, byref(s), byref(c)))
        return s.value, c.value

    def split_xbc(self, u: torch.Tensor):
        """Views x, B, C of packed pre-conv rows u [rows, Cd]."""
        I, GN = self.intermediate, self.n_groups * self.d_state
        return u[:, :I], u[:, I:I + GN], u[:, I + GN:]

    # ------------------------------------------------------------------ decode
    def decode_step(self, layer: int, w: LayerWeights, slots: torch.Tensor, x, B, C, z, dt, y,
                    slots_host=None):
        """One token per row of slots (device int32); writes y in place and updates the pool."""
        if slots.dtype != torch.int32:
            raise TypeError("slots must be int32")
        _, sh_ptr = _host_i32(slots_host)
        io = _dtype_code(x)
        for t in (B, C, z, dt):
            if _dtype_code(t) != io:
                raise TypeError("x, B, C, z and dt must share one dtype")
        xp, xs = _rows(x, "x")
        bp, bs = _rows(B, "B")
        cp, cs = _rows(C, "C")
        zp, zs = _rows(z, "z")
        dp, ds = _rows(dt, "dt")
        yp, ys = _rows(y, "y")
        check(lib().mamba2_decode_step(self._h, layer, byref(w.struct), slots.numel(), c_void_p(slots.data_ptr()),
                                       sh_ptr, xp, xs, bp, bs, cp, cs, zp, zs, dp, ds, io, yp, ys,
                                       _dtype_code(y), _stream()))
        return y

    def decode_multi(self, layer: int, w: LayerWeights, slots_in: torch.Tensor, slots_out: torch.Tensor,
                     x, B, C, z, dt, y, slots_in_host=None, slots_out_host=None):
        """num_tokens = slots_out.shape[1] decode tokens per row of slots_in (device int32), rows
        b*num_tokens + t of x, B, C, z, dt and y; the state after token t goes to slots_out[b, t]."""
        if slots_in.dtype != torch.int32 or slots_out.dtype != torch.int32:
            raise TypeError("slots must be int32")
        if slots_out.dim() != 2 or slots_out.shape[0] != slots_in.numel() or not slots_out.is_contiguous():
            raise ValueError("slots_out must be a contiguous [batch, num_tokens] tensor")
        _, si_p = _host_i32(slots_in_host)
        _, so_p = _host_i32(None if slots_out_host is None else np.asarray(slots_out_host).reshape(-1))
        io = _dtype_code(x)
        for t in (B, C, z, dt):
            if _dtype_code(t) != io:
                raise TypeError("x, B, C, z and dt must share one dtype")
        xp, xs = _rows(x, "x")
        bp, bs = _rows(B, "B")
        cp, cs = _rows(C, "C")
        zp, zs = _rows(z, "z")
        dp, ds = _rows(dt, "dt")
        yp, ys = _rows(y, "y")
        check(lib().mamba2_decode_multi(self._h, layer, byref(w.struct), slots_in.numel(), slots_out.shape[1],
                                        c_void_p(slots_in.data_ptr()), c_void_p(slots_out.data_ptr()), si_p, so_p,
                                        xp, xs, bp, bs, cp, cs, zp, zs, dp, ds, io, yp, ys, _dtype_code(y),
                                        _stream()))
        return y

    # ------------------------------------------------------------------ prefill
    def workspace_size(self, cu_seqlens, chunk_size: int = 256, start_pos=None, ckpt_interval: int = 0,
                       ckpt_slots=None) -> int:
        """Workspace bytes of a prefill call with these host arguments (the library counts the chunks)."""
        cu, cu_p = _host_i32(cu_seqlens)
        ns = len(cu) - 1
        _, sp_p = _host_i32(start_pos)
        ck_p, max_ck = None, 0
        if ckpt_slots is not None:
            ck = np.ascontiguousarray(np.asarray(ckpt_slots, dtype=np.int32).reshape(ns, -1))
            ck_p, max_ck = ck.ctypes.data_as(c_void_p), ck.shape[1]
        n = c_uint64()
        check(lib().mamba2_prefill_workspace_size(self._h, ns, cu_p, sp_p, chunk_size, ckpt_interval, ck_p, max_ck,
                                                  byref(n)))
        return n.value

    def prefill(self, layer: int, w: LayerWeights, cu_seqlens, slots, has_init, x, B, C, z, dt, y,
                start_pos=None, chunk_size: int = 256, ckpt_interval: int = 0, ckpt_slots=None,
                workspace: torch.Tensor | None = None):
        """Chunked prefill of packed sequences; cu_seqlens/slots/has_init/start_pos/ckpt_slots are host arrays."""
        cu, cu_p = _host_i32(cu_seqlens)
        sl, sl_p = _host_i32(slots)
        hi = np.ascontiguousarray(np.asarray(has_init, dtype=np.uint8))
        sp, sp_p = _host_i32(start_pos)
        ns = len(sl)
        max_ck = 0
        ck_p = None
        if ckpt_slots is not None:
            ck = np.ascontiguousarray(np.asarray(ckpt_slots, dtype=np.int32).reshape(ns, -1))
            max_ck = ck.shape[1]
            ck_p = ck.ctypes.data_as(c_void_p)
        if workspace is None:
            need = self.workspace_size(cu, chunk_size, sp, ckpt_interval, ckpt_slots)
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=self.ssm.device)
        io = _dtype_code(x)
        xp, xs = _rows(x, "x")
        bp, bs = _rows(B, "B")
        cp, cs = _rows(C, "C")
        zp, zs = _rows(z, "z")
        dp, ds = _rows(dt, "dt")
        yp, ys = _rows(y, "y")
        check(lib().mamba2_prefill_chunked(
            self._h, layer, byref(w.struct), ns, cu.ctypes.data_as(c_void_p), sl_p,
            hi.ctypes.data_as(c_void_p), sp_p, xp, xs, bp, bs, cp, cs, zp, zs, dp, ds, io, yp, ys,
            _dtype_code(y), chunk_size, ckpt_interval, ck_p, max_ck, c_void_p(workspace.data_ptr()),
            workspace.numel(), _stream()))
        return y

    def prefill_noalloc(self, layer: int, w: LayerWeights, cu_seqlens, slots, has_init, x, B, C, z, dt, y,
                        start_pos=None, chunk_size: int = 256, ckpt_interval: int = 0, ckpt_slots=None):
        """prefill() with its scratch in the library's static per-GPU array instead of a workspace."""
        cu, _ = _host_i32(cu_seqlens)
        sl, sl_p = _host_i32(slots)
        hi = np.ascontiguousarray(np.asarray(has_init, dtype=np.uint8))
        _, sp_p = _host_i32(start_pos)
        ns = len(sl)
        max_ck, ck_p = 0, None
        if ckpt_slots is not None:
            ck = np.ascontiguousarray(np.asarray(ckpt_slots, dtype=np.int32).reshape(ns, -1))
            max_ck, ck_p = ck.shape[1], ck.ctypes.data_as(c_void_p)
        xp, xs = _rows(x, "x")
        bp, bs = _rows(B, "B")
        cp, cs = _rows(C, "C")
        zp, zs = _rows(z, "z")
        dp, ds = _rows(dt, "dt")
        yp, ys = _rows(y, "y")
        check(lib().mamba2_prefill_chunked_noalloc(
            self._h, layer, byref(w.struct), ns, cu.ctypes.data_as(c_void_p), sl_p, hi.ctypes.data_as(c_void_p),
            sp_p, xp, xs, bp, bs, cp, cs, zp, zs, dp, ds, _dtype_code(x), yp, ys, _dtype_code(y), chunk_size,
            ckpt_interval, ck_p, max_ck, _stream()))
        return y

    # ------------------------------------------------------------------ gated delta rule (GDN pools)
    def split_qkv(self, u: torch.Tensor):
        """Views q, k, v of packed pre-conv rows u [rows, Cd] of a GDN layer."""
        qk = self.n_groups * self.d_state
        return u[:, :qk], u[:, qk:2 * qk], u[:, 2 * qk:]

    def _gdn_rows(self, w: LayerWeights, rows: int, q, k, v, a, b, o, exact: bool):
        """Pointers, strides and dtypes of a gated-delta call's row tensors, checked against the pool."""
        dev, qk = self.ssm.device, self.n_groups * self.d_state
        io = _dtype_code(q)
        args = []
        for t, name, width in ((q, "q", qk), (k, "k", qk), (v, "v", self.intermediate), (a, "a", self.nheads),
                               (b, "b", self.nheads), (o, "o", self.intermediate)):
            if t.device != dev:
                raise ValueError(f"{name} is on {t.device}, the pool on {dev}")
            if t is not o and _dtype_code(t) != io:
                raise TypeError("q, k, v, a and b must share one dtype")
            p, stride = _rows(t, name)
            if t.shape[1] != width or (t.shape[0] != rows if exact else t.shape[0] < rows):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {rows} rows of {width}")
            # the stride of a single row is never used, and a view of one row may have any
            args += [p, width if rows <= 1 else stride]
        for t, name, shape in ((w.A, "A", (self.nheads,)), (w.dt_bias, "dt_bias", (self.nheads,)),
                               (w.conv_w, "conv_w", (self.conv_dim, self.conv_kernel)),
                               (w.conv_b, "conv_b", (self.conv_dim,))):
            if t is not None and (t.device != dev or tuple(t.shape) != shape):
                raise ValueError(f"{name} must be a {shape} tensor on {dev}")
        return args[:10] + [io] + args[10:] + [_dtype_code(o)]

    def _slots(self, t: torch.Tensor, name: str):
        if t.dtype != torch.int32 or not t.is_contiguous() or t.device != self.ssm.device:
            raise TypeError(f"{name} must be a contiguous int32 tensor on the pool's device")
        return c_void_p(t.data_ptr())

    def gdn_decode_step(self, layer: int, w: LayerWeights, slots: torch.Tensor, q, k, v, a, b, o, slots_host=None):
        """One gated-delta token per row of slots (device int32); writes o in place and updates the pool."""
        sl = self._slots(slots, "slots")
        host, host_p = _host_i32(slots_host)
        if host is not None and host.size != slots.numel():
            raise ValueError("slots_host must have one entry per row")
        rows = self._gdn_rows(w, slots.numel(), q, k, v, a, b, o, True)
        with torch.cuda.device(self.ssm.device):
            check(lib().mamba2_gdn_decode_step(self._h, layer, byref(w.struct), slots.numel(), sl, host_p, *rows,
                                               _stream()))
        return o

    def gdn_decode_multi(self, layer: int, w: LayerWeights, slots_in: torch.Tensor, slots_out: torch.Tensor,
                         q, k, v, a, b, o, slots_in_host=None, slots_out_host=None):
        """num_tokens = slots_out.shape[1] gated-delta tokens per row of slots_in (device int32), rows
        i*num_tokens + t of q, k, v, a, b and o; the state after token t goes to slots_out[i, t]."""
        si, so = self._slots(slots_in, "slots_in"), self._slots(slots_out, "slots_out")
        if slots_out.dim() != 2 or slots_out.shape[0] != slots_in.numel():
            raise ValueError("slots_out must be a contiguous [batch, num_tokens] tensor")
        hi, hi_p = _host_i32(slots_in_host)
        ho, ho_p = _host_i32(None if slots_out_host is None else np.asarray(slots_out_host).reshape(-1))
        if (hi is not None and hi.size != slots_in.numel()) or (ho is not None and ho.size != slots_out.numel()):
            raise ValueError("host slots must match the device slots")
        rows = self._gdn_rows(w, slots_out.numel(), q, k, v, a, b, o, True)
        with torch.cuda.device(self.ssm.device):
            check(lib().mamba2_gdn_decode_multi(self._h, layer, byref(w.struct), slots_in.numel(), slots_out.shape[1],
                                                si, so, hi_p, ho_p, *rows, _stream()))
        return o

    @staticmethod
    def _ckpt_table(ckpt_slots, ns: int):
        if ckpt_slots is None:
            return None, None, 0
        # without sequences the table has no rows to tell its width by
        ck = np.ascontiguousarray(np.asarray(ckpt_slots, dtype=np.int32).reshape(ns, -1 if ns else 0))
        return ck, ck.ctypes.data_as(c_void_p), ck.shape[1]

    def gdn_workspace_size(self, cu_seqlens, start_pos=None, ckpt_interval: int = 0, ckpt_slots=None,
                           io_dtype=torch.bfloat16, o_dtype=torch.bfloat16) -> int:
        """Workspace bytes of a gdn_prefill call with these host arguments and dtypes."""
        cu, cu_p = _host_i32(cu_seqlens)
        ns = len(cu) - 1
        sp, sp_p = _host_i32(start_pos)
        if sp is not None and sp.size != ns:
            raise ValueError("start_pos must have one entry per sequence")
        ck, ck_p, max_ck = self._ckpt_table(ckpt_slots, ns)
        n = c_uint64()
        check(lib().mamba2_gdn_prefill_workspace_size(self._h, ns, cu_p, sp_p, ckpt_interval, ck_p, max_ck,
                                                      _code_of(io_dtype), _code_of(o_dtype), byref(n)))
        return n.value

    def gdn_prefill(self, layer: int, w: LayerWeights, cu_seqlens, slots, has_init, q, k, v, a, b, o, start_pos=None,
                    ckpt_interval: int = 0, ckpt_slots=None, workspace: torch.Tensor | None = None):
        """Chunked gated-delta prefill of packed sequences; cu_seqlens, slots, has_init, start_pos and
        ckpt_slots [num_seqs][max_ckpt] are host arrays.  Rows behind cu_seqlens[-1] are left alone."""
        cu, cu_p = _host_i32(cu_seqlens)
        ns = len(cu) - 1
        sl, sl_p = _host_i32(slots)
        hi = np.ascontiguousarray(np.asarray(has_init, dtype=np.uint8))
        sp, sp_p = _host_i32(start_pos)
        if ns < 0 or sl.size != ns or hi.size != ns or (sp is not None and sp.size != ns):
            raise ValueError("cu_seqlens has one entry more than slots, has_init and start_pos")
        ck, ck_p, max_ck = self._ckpt_table(ckpt_slots, ns)
        rows = self._gdn_rows(w, int(cu[-1]), q, k, v, a, b, o, False)
        if workspace is None:
            need = self.gdn_workspace_size(cu, sp, ckpt_interval, ck, q.dtype, o.dtype)
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=self.ssm.device)
        elif workspace.device != self.ssm.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the pool's device")
        with torch.cuda.device(self.ssm.device):
            check(lib().mamba2_gdn_prefill(
                self._h, layer, byref(w.struct), ns, cu_p, sl_p, hi.ctypes.data_as(c_void_p), sp_p, *rows, ckpt_interval,
                ck_p, max_ck, c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(), _stream()))
        return o

    # ------------------------------------------------------------------ beam search
    def beam_workspace_size(self, batch: int, beams: int, vocab: int) -> int:
        """Workspace bytes of a beam_step call."""
        n = c_uint64()
        check(lib().mamba2_beam_workspace_size(self._h, batch, beams, vocab, byref(n)))
        return n.value

    def beam_step(self, logits: torch.Tensor, scores, slots, tokens, parents, scores_out, slots_out, finished=None,
                  finished_out=None, eos_token: int = -1, slots_host=None, workspace: torch.Tensor | None = None):
        """One beam-search step for logits [batch, beams, vocab]: the best `beams` continuations of each
        request into tokens, parents, scores_out and slots_out ([batch*beams] each, best first), and the
        states of every layer where the new beams live.  finished / finished_out are uint8; an output may
        be the input of its kind."""
        if logits.dim() != 3 or (logits.stride(2) != 1 and logits.shape[2] > 1 and logits.numel() > 0) or (
                min(logits.shape[:2]) > 1 and logits.stride(0) != logits.shape[1] * logits.stride(1)):
            raise ValueError("logits must be [batch, beams, vocab] with evenly spaced rows and a contiguous last dimension")
        batch, beams, vocab = logits.shape
        dev, n = self.ssm.device, batch * beams
        if logits.device != dev:
            raise ValueError(f"logits are on {logits.device}, the pool on {dev}")
        ptrs = []
        for t, name, dt in ((scores, "scores", torch.float32), (finished, "finished", torch.uint8),
                            (slots, "slots", torch.int32), (tokens, "tokens", torch.int32),
                            (parents, "parents", torch.int32), (scores_out, "scores_out", torch.float32),
                            (finished_out, "finished_out", torch.uint8), (slots_out, "slots_out", torch.int32)):
            if t is None and name.startswith("finished"):
                ptrs.append(None)
                continue
            if t.dtype != dt or t.device != dev or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dt} tensor of {n} on {dev}")
            ptrs.append(c_void_p(t.data_ptr()))
        host, host_p = _host_i32(None if slots_host is None else np.asarray(slots_host).reshape(-1))
        if host is not None and host.size != n:
            raise ValueError("slots_host must have one entry per beam")
        if workspace is None:
            workspace = torch.empty(max(self.beam_workspace_size(batch, beams, vocab), 1), dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the pool's device")
        # the stride of a single row is never used; torch gives it any value
        stride = vocab if n <= 1 else logits.stride(1) if beams > 1 else logits.stride(0)
        with torch.cuda.device(dev):
            check(lib().mamba2_beam_step(self._h, batch, beams, vocab, c_void_p(logits.data_ptr()), stride,
                                         _dtype_code(logits), ptrs[0], ptrs[1], eos_token, ptrs[2], host_p, *ptrs[3:6],
                                         ptrs[6], ptrs[7], c_void_p(workspace.data_ptr()),
                                         workspace.numel() * workspace.element_size(), _stream()))
        return tokens, parents

    # ------------------------------------------------------------------ checkpoints
    def int8_store(self, num_entries: int) -> "Int8Store":
        """A zeroed int8 checkpoint store of num_entries entries for this pool's layers."""
        return Int8Store(self, num_entries)

    def int8_put(self, store: "Int8Store", layer: int, slots: torch.Tensor, entries: torch.Tensor,
                 slots_host=None, entries_host=None):
        """Quantize slot slots[i] into store entry entries[i] (device int32); layer -1 = all layers."""
        _, s_p = _host_i32(slots_host)
        _, e_p = _host_i32(entries_host)
        check(lib().mamba2_int8_store_put(self._h, byref(store.desc), layer, slots.numel(),
                                          c_void_p(slots.data_ptr()), c_void_p(entries.data_ptr()), s_p, e_p,
                                          _stream()))

    def int8_get(self, store: "Int8Store", layer: int, entries: torch.Tensor, slots: torch.Tensor,
                 entries_host=None, slots_host=None):
        """Restore store entry entries[i] into slot slots[i] (device int32); layer -1 = all layers."""
        _, e_p = _host_i32(entries_host)
        _, s_p = _host_i32(slots_host)
        check(lib().mamba2_int8_store_get(self._h, byref(store.desc), layer, entries.numel(),
                                          c_void_p(entries.data_ptr()), c_void_p(slots.data_ptr()), e_p, s_p,
                                          _stream()))

    def checkpoint(self, layer: int, src: torch.Tensor, dst: torch.Tensor, src_host=None, dst_host=None):
        """Copy both state objects slot src[i] -> dst[i] (device int32); layer -1 = all layers."""
        _, s_p = _host_i32(src_host)
        _, d_p = _host_i32(dst_host)
        check(lib().mamba2_checkpoint_states(self._h, layer, src.numel(), c_void_p(src.data_ptr()),
                                             c_void_p(dst.data_ptr()), s_p, d_p, _stream()))


class Int8Store:
    """int8 checkpoint store for a pool: codes int8 [E, L, H, P, N], scales fp32 [E, L, H, N],
    conv windows [E, L, Cd, W-1] in the pool's conv dtype, allocated on the pool's device."""

    def __init__(self, pool: Pool, num_entries: int):
        cb, sb, vb = c_uint64(), c_uint64(), c_uint64()
        check(lib().mamba2_int8_store_size(pool._h, num_entries, byref(cb), byref(sb), byref(vb)))
        L, H, P, N = pool.num_layers, pool.nheads, pool.head_dim, pool.d_state
        dev = pool.ssm.device
        self.codes = torch.zeros((num_entries, L, H, P, N), dtype=torch.int8, device=dev)
        self.scales = torch.zeros((num_entries, L, H, N), dtype=torch.float32, device=dev)
        self.conv = torch.zeros((num_entries, L) + tuple(pool.conv.shape[2:]), dtype=pool.conv.dtype, device=dev)
        for t, b in ((self.codes, cb), (self.scales, sb), (self.conv, vb)):
            assert t.numel() * t.element_size() == b.value
        self.num_entries = num_entries
        self.desc = Int8StoreDesc(num_entries, 0, self.codes.data_ptr(), self.scales.data_ptr(),
                                  self.conv.data_ptr(), cb.value, sb.value, vb.value)


__all__ = ["Pool", "LayerWeights", "Int8Store", "Mamba2Error"]
