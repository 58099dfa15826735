"""Device-side marshalling for the C ABI: uploads a layer's host arrays into torch CUDA
tensors, fills ``moe_weights`` with their addresses and owns the handle and workspaces.

Torch provides memory and streams only; every computation runs in ``libmoe.so``.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (MOE_DTYPE_BF16, MOE_DTYPE_F16, MOE_DTYPE_F32, MOE_FMT_INT4_ROWSCALE, MOE_FMT_NVFP4,
               moe_adapters_apply, moe_adapters_backward, moe_adapters_create, moe_adapters_desc,
               moe_adapters_destroy, moe_adapters_get_device_status, moe_adapters_weights,
               moe_adapters_workspace_size, moe_combine, moe_expert_ffn,
               moe_forward, moe_forward_fused, moe_forward_host, moe_group, moe_layer_create, moe_layer_desc,
               moe_layer_destroy, moe_route, moe_route_static, moe_sort_tokens, moe_sort_tokens_backward,
               moe_sort_workspace_size, moe_sorted_rows, moe_unsort_tokens, moe_unsort_tokens_backward,
               moe_weights, moe_workspace_size)

# torch dtype -> MOE_DTYPE_* (the layer's activations are fp16 bit patterns in uint16)
_DTYPE = {torch.float16: MOE_DTYPE_F16, torch.uint16: MOE_DTYPE_F16, torch.bfloat16: MOE_DTYPE_BF16,
          torch.float32: MOE_DTYPE_F32}


def _rows(t: torch.Tensor, shape: tuple, what: str) -> tuple:
    """(address, MOE_DTYPE_*, row stride) of a 2-D tensor whose rows are dense."""
    dtype = _DTYPE.get(t.dtype)
    if t.shape != shape or dtype is None or not t.is_cuda:
        stride = None
    else:
        stride = t.stride()
    if stride is None or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what}: a CUDA tensor {list(shape)} of fp16, bf16 or fp32 with dense rows is wanted, "
                         f"got {t.dtype} {list(t.shape)} with strides {t.stride()} on {t.device}")
    # (the stride of a single row may be any number)
    return t.data_ptr(), dtype, stride[0] if shape[0] > 1 else shape[1]


def _raw_stream(stream, index: int) -> int:
    """Handle of a stream, or of the current stream of device `index` (looked up without
    making a torch.cuda.Stream, which takes longer than a small launch)."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)


def _index(device: torch.device) -> int:
    return torch.cuda.current_device() if device.index is None else device.index


def _dense(t: torch.Tensor, dtype, numel: int, what: str) -> int:
    if t.dtype != dtype or t.numel() != numel or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{what}: a contiguous CUDA tensor of {numel} {dtype} is wanted, "
                         f"got {t.dtype} {list(t.shape)}")
    return t.data_ptr()

# host array key -> moe_weights field
_FIELD = {
    "Wr": "router_w", "bias": "router_bias", "g": "gate", "u": "up", "d": "down",
    "sg": "gate_scale", "su": "up_scale", "sd": "down_scale",
    "bg": "gate_bscale", "bu": "up_bscale", "bd": "down_bscale",
    "tg": "gate_tscale", "tu": "up_tscale", "td": "down_tscale",
    "sh_g": "shared_gate", "sh_u": "shared_up", "sh_d": "shared_down",
    "sh_sg": "shared_gate_scale", "sh_su": "shared_up_scale", "sh_sd": "shared_down_scale",
    "sh_bg": "shared_gate_bscale", "sh_bu": "shared_up_bscale", "sh_bd": "shared_down_bscale",
    "sh_tg": "shared_gate_tscale", "sh_tu": "shared_up_tscale", "sh_td": "shared_down_tscale",
}


def make_desc(d: dict, max_tokens: int) -> moe_layer_desc:
    return moe_layer_desc(hidden=d["H"], inter=d["I"], inter_shared=d["I_sh"], n_experts=d["E"],
                          top_k=d["k"], n_shared=d["n_shared"], routed_scaling=d["scaling"],
                          format=d["fmt"], max_tokens=max_tokens, top_p=float(d.get("top_p", 0.0)))


def _to_device(a, device) -> torch.Tensor:
    a = np.ascontiguousarray(np.asarray(a))
    if a.ndim == 0:
        a = a.reshape(1)
    return torch.from_numpy(a).to(device)


class DeviceLayer:
    """One layer resident in HBM plus its handle."""

    def __init__(self, desc: dict, host: dict | None = None, max_tokens: int = 1,
                 device="cuda", tensors: dict | None = None):
        self.d = dict(desc)
        self.device = torch.device(device)
        self.max_tokens = max_tokens
        if tensors is None:
            tensors = {k: _to_device(v, self.device) for k, v in host.items() if k in _FIELD}
        self.t = tensors
        w = moe_weights()
        for k, v in self.t.items():
            setattr(w, _FIELD[k], v.data_ptr())
        self.weights = w
        self.desc = make_desc(self.d, max_tokens)
        self.handle = moe_layer_create(self.desc, self.weights)
        self.index = _index(self.device)

    def clone_weights(self) -> "DeviceLayer":
        """A second layer with the same values at different HBM addresses."""
        return DeviceLayer(self.d, max_tokens=self.max_tokens, device=self.device,
                           tensors={k: v.clone() for k, v in self.t.items()})

    def close(self):
        if getattr(self, "handle", None):
            moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ workspace
    def workspace(self, T: int) -> torch.Tensor:
        n = moe_workspace_size(self.handle, T)
        if n == 0:
            raise ValueError(f"T={T} out of range for this handle")
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    # ------------------------------------------------------------------ calls
    @staticmethod
    def _stream(stream):
        return (stream or torch.cuda.current_stream()).cuda_stream

    def forward(self, x: torch.Tensor, ws: torch.Tensor, y: torch.Tensor | None = None,
                stream=None, fused: bool = False) -> torch.Tensor:
        """The layer (moe_forward); fused=True: the one-launch decode path
        (moe_forward_fused, T <= 16)."""
        T = x.shape[0]
        if y is None:
            y = torch.empty_like(x)
        fn = moe_forward_fused if fused else moe_forward
        fn(self.handle, x.data_ptr(), T, y.data_ptr(), ws.data_ptr(), ws.numel(), self._stream(stream))
        return y

    def forward_host(self, x_host: torch.Tensor, y_host: torch.Tensor, ws: torch.Tensor,
                     stream=None):
        moe_forward_host(self.handle, x_host.data_ptr(), x_host.shape[0], y_host.data_ptr(),
                         ws.data_ptr(), ws.numel(), self._stream(stream))

    def route(self, x, T, ws, logits_in=None, want_logits=False, stream=None):
        k, E = self.d["k"], self.d["E"]
        idx = torch.empty((T, k), dtype=torch.int32, device=self.device)
        w = torch.empty((T, k), dtype=torch.float32, device=self.device)
        lo = torch.empty((T, E), dtype=torch.float32, device=self.device) if want_logits else None
        moe_route(self.handle, x.data_ptr() if x is not None else None, T,
                  logits_in.data_ptr() if logits_in is not None else None,
                  lo.data_ptr() if lo is not None else None, idx.data_ptr(), w.data_ptr(),
                  ws.data_ptr(), ws.numel(), self._stream(stream))
        return idx, w, lo

    def route_static(self, x, T, logits_in=None, want_logits=False, stream=None):
        """moe_route with the library's static scratch instead of a workspace."""
        k, E = self.d["k"], self.d["E"]
        idx = torch.empty((T, k), dtype=torch.int32, device=self.device)
        w = torch.empty((T, k), dtype=torch.float32, device=self.device)
        lo = torch.empty((T, E), dtype=torch.float32, device=self.device) if want_logits else None
        moe_route_static(self.handle, x.data_ptr() if x is not None else None, T,
                         logits_in.data_ptr() if logits_in is not None else None,
                         lo.data_ptr() if lo is not None else None, idx.data_ptr(), w.data_ptr(),
                         self._stream(stream))
        return idx, w, lo

    def group(self, topk_idx, T, ws, stream=None):
        E = self.d["E"]
        dev = self.device
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(max(T * self.d["k"], 1), dtype=torch.int32, device=dev)
        unique = torch.empty(E, dtype=torch.int32, device=dev)
        nu = torch.empty(1, dtype=torch.int32, device=dev)
        moe_group(self.handle, topk_idx.data_ptr(), T, counts.data_ptr(), offsets.data_ptr(),
                  perm.data_ptr(), unique.data_ptr(), nu.data_ptr(), ws.data_ptr(), ws.numel(),
                  self._stream(stream))
        return counts, offsets, perm, unique, nu

    def expert_ffn(self, x, T, offsets, perm, ws, stream=None):
        H, k = self.d["H"], self.d["k"]
        ya = torch.empty((T * k, H), dtype=torch.float32, device=self.device)
        ys = torch.empty((T, H), dtype=torch.float32, device=self.device) if self.d["n_shared"] else None
        moe_expert_ffn(self.handle, x.data_ptr(), T, offsets.data_ptr(), perm.data_ptr(),
                       ya.data_ptr(), ys.data_ptr() if ys is not None else None, ws.data_ptr(),
                       ws.numel(), self._stream(stream))
        return ya, ys

    def combine(self, y_assign, y_shared, topk_w, T, stream=None):
        y = torch.empty((T, self.d["H"]), dtype=torch.uint16, device=self.device)
        moe_combine(self.handle, y_assign.data_ptr(),
                    y_shared.data_ptr() if y_shared is not None else None, topk_w.data_ptr(), T,
                    y.data_ptr(), self._stream(stream))
        return y

    # ------------------------------------------------------------------ sorted rows
    def sort_workspace(self, T: int) -> torch.Tensor:
        """A workspace of moe_sort_tokens alone (workspace(T) serves too)."""
        n = moe_sort_workspace_size(self.handle, T)
        if n == 0:
            raise ValueError(f"T={T} out of range for this handle")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def sorted_rows(self, T: int, align: int = 1) -> int:
        return moe_sorted_rows(self.handle, T, align)

    def sort_tokens(self, x, topk_idx, ws, align=1, out=None, stream=None):
        """(rows [n, H], row_of [T, k], counts [E], seg_offsets [E + 1]) of moe_sort_tokens;
        out: the same four tensors to write to."""
        T, H, k, E = x.shape[0], self.d["H"], self.d["k"], self.d["E"]
        if out is None:
            i32 = dict(dtype=torch.int32, device=self.device)
            out = (torch.empty((self.sorted_rows(T, align), H), dtype=x.dtype, device=self.device),
                   torch.empty((T, k), **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32))
        rows, row_of, counts, seg = out
        px, dtype, ldx = _rows(x, (T, H), "x")
        moe_sort_tokens(self.handle, px, dtype, ldx, _dense(topk_idx, torch.int32, T * k, "topk_idx"), T, align,
                        _dense(rows, x.dtype, rows.shape[0] * H, "rows"), rows.shape[0],
                        _dense(row_of, torch.int32, T * k, "row_of"), _dense(counts, torch.int32, E, "counts"),
                        _dense(seg, torch.int32, E + 1, "seg_offsets"), ws.data_ptr(), ws.numel(),
                        _raw_stream(stream, self.index))
        return out

    def sort_tokens_backward(self, drows, row_of, dx=None, stream=None):
        """dx [T, H] of moe_sort_tokens_backward (of drows' type unless dx is given)."""
        n, H, k = drows.shape[0], self.d["H"], self.d["k"]
        T = row_of.numel() // k
        if dx is None:
            dx = torch.empty((T, H), dtype=drows.dtype, device=self.device)
        pr, rdt = _dense(drows, drows.dtype, n * H, "drows"), _DTYPE[drows.dtype]
        px, xdt, ldx = _rows(dx, (T, H), "dx")
        moe_sort_tokens_backward(self.handle, pr, rdt, n, _dense(row_of, torch.int32, T * k, "row_of"), T, px, xdt,
                                 ldx, _raw_stream(stream, self.index))
        return dx

    def unsort_tokens(self, rows, row_of, topk_w, y_shared=None, y=None, stream=None):
        """y [T, H] of moe_unsort_tokens (of rows' type unless y is given)."""
        n, H, k = rows.shape[0], self.d["H"], self.d["k"]
        T = row_of.numel() // k
        if y is None:
            y = torch.empty((T, H), dtype=rows.dtype, device=self.device)
        py, ydt, ldy = _rows(y, (T, H), "y")
        moe_unsort_tokens(self.handle, _dense(rows, rows.dtype, n * H, "rows"), _DTYPE[rows.dtype], n,
                          _dense(row_of, torch.int32, T * k, "row_of"),
                          _dense(topk_w, torch.float32, T * k, "topk_w"),
                          None if y_shared is None else _dense(y_shared, torch.float32, T * H, "y_shared"), T, py,
                          ydt, ldy, _raw_stream(stream, self.index))
        return y

    def unsort_tokens_backward(self, dy, rows, row_of, topk_w, counts=None, seg_offsets=None, out=None, stream=None):
        """(drows [n, H], dw [T, k]) of moe_unsort_tokens_backward; out: the two tensors to
        write to."""
        n, H, k, E = rows.shape[0], self.d["H"], self.d["k"], self.d["E"]
        T = row_of.numel() // k
        if out is None:
            out = (torch.empty_like(rows), torch.empty((T, k), dtype=torch.float32, device=self.device))
        drows, dw = out
        pd, ddt, ldd = _rows(dy, (T, H), "dy")
        moe_unsort_tokens_backward(self.handle, pd, ddt, ldd, _dense(rows, rows.dtype, n * H, "rows"),
                                   _DTYPE[rows.dtype], n, _dense(row_of, torch.int32, T * k, "row_of"),
                                   _dense(topk_w, torch.float32, T * k, "topk_w"),
                                   None if counts is None else _dense(counts, torch.int32, E, "counts"),
                                   None if seg_offsets is None else
                                   _dense(seg_offsets, torch.int32, E + 1, "seg_offsets"), T,
                                   _dense(drows, rows.dtype, n * H, "drows"),
                                   _dense(dw, torch.float32, T * k, "dw"), _raw_stream(stream, self.index))
        return out


class DeviceAdapters:
    """A pool of low-rank adapters of one projection and its handle: a [n, R, K], b [n, N, R]
    (fp16 or bf16), scaling fp32 [n], rank int32 [n] or None; the tensors are borrowed."""

    def __init__(self, a, b, scaling, rank=None, max_tokens: int = 1):
        n, R, K = a.shape
        N = b.shape[1]
        if b.shape != (n, N, R) or a.dtype not in _DTYPE:
            raise ValueError(f"a {list(a.shape)} {a.dtype} and b {list(b.shape)} do not make a pool of adapters")
        self.n, self.R, self.K, self.N = n, R, K, N
        self.device, self.dtype = a.device, a.dtype
        self.t = (a, b, scaling, rank)
        w = moe_adapters_weights(a=_dense(a, a.dtype, n * R * K, "a"), b=_dense(b, a.dtype, n * N * R, "b"),
                                 scaling=_dense(scaling, torch.float32, n, "scaling"),
                                 rank=None if rank is None else _dense(rank, torch.int32, n, "rank"))
        self.desc = moe_adapters_desc(in_features=K, out_features=N, n_adapters=n, max_rank=R,
                                      dtype=_DTYPE[a.dtype], max_tokens=max_tokens)
        self.handle = moe_adapters_create(self.desc, w)
        self.index = _index(self.device)

    def close(self):
        if getattr(self, "handle", None):
            moe_adapters_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace(self, T: int) -> torch.Tensor:
        n = moe_adapters_workspace_size(self.handle, T)
        if n == 0:
            raise ValueError(f"T={T} out of range for this handle")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def status(self) -> int:
        return moe_adapters_get_device_status(self.handle)

    def _input(self, t, shape, what):
        p, dtype, ld = _rows(t, shape, what)
        if dtype != self.desc.dtype:
            raise ValueError(f"{what}: the pool's type {self.dtype} is wanted, got {t.dtype}")
        return p, ld

    def _base(self, base, out, shape, what):
        """Address and row stride of an optional addend of out's type."""
        if base is None:
            return None, 0
        p, dtype, ld = _rows(base, shape, what)
        if dtype != _DTYPE[out.dtype]:
            raise ValueError(f"{what}: the output's type {out.dtype} is wanted, got {base.dtype}")
        return p, ld

    def apply(self, x, adapter_of, ws, y_in=None, y=None, z=None, stream=None):
        """y = y_in + scaling * B (A x), each token through its own adapter (moe_adapters_apply);
        y may be y_in; z fp32 [T, R] receives A x for the gradient."""
        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.N), dtype=x.dtype if y_in is None else y_in.dtype, device=self.device)
        px, ldx = self._input(x, (T, self.K), "x")
        py, ydt, ldy = _rows(y, (T, self.N), "y")
        pb, ldb = self._base(y_in, y, (T, self.N), "y_in")
        moe_adapters_apply(self.handle, px, ldx, _dense(adapter_of, torch.int32, T, "adapter_of"), T, pb, ldb, py, ydt,
                           ldy, None if z is None else _dense(z, torch.float32, T * self.R, "z"), ws.data_ptr(),
                           ws.numel(), _raw_stream(stream, self.index))
        return y

    def backward(self, x, z, dy, adapter_of, ws, dx_in=None, dx=None, da=None, db=None, accumulate=False,
                 want_dx=True, want_dw=True, stream=None):
        """(dx, da, db) of moe_adapters_backward; da fp32 [n, R, K], db fp32 [n, N, R] (added to
        when accumulate is set); want_dx / want_dw = False leave dx / da and db out (None)."""
        T = dy.shape[0]
        f32 = dict(dtype=torch.float32, device=self.device)
        px = pz = pa = pb = pdx = pin = None
        ldx = ldi = lddx = ddt = 0
        pdy, lddy = self._input(dy, (T, self.N), "dy")
        if want_dx:
            if dx is None:
                dx = torch.empty((T, self.K), dtype=dy.dtype if dx_in is None else dx_in.dtype, device=self.device)
            pdx, ddt, lddx = _rows(dx, (T, self.K), "dx")
            pin, ldi = self._base(dx_in, dx, (T, self.K), "dx_in")
        if want_dw:
            new = torch.zeros if accumulate else torch.empty
            da = new((self.n, self.R, self.K), **f32) if da is None else da
            db = new((self.n, self.N, self.R), **f32) if db is None else db
            pa = _dense(da, torch.float32, self.n * self.R * self.K, "da")
            pb = _dense(db, torch.float32, self.n * self.N * self.R, "db")
            px, ldx = self._input(x, (T, self.K), "x")
            pz = _dense(z, torch.float32, T * self.R, "z")
        moe_adapters_backward(self.handle, px, ldx, pz, pdy, lddy, _dense(adapter_of, torch.int32, T, "adapter_of"), T,
                              pin, ldi, pdx, ddt, lddx, pa, pb, int(accumulate), ws.data_ptr(), ws.numel(),
                              _raw_stream(stream, self.index))
        return (dx if want_dx else None), (da if want_dw else None), (db if want_dw else None)


def fp16_bits_to_float(y_bits: torch.Tensor) -> np.ndarray:
    return y_bits.cpu().numpy().view(np.float16).astype(np.float64)
