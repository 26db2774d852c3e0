"""Matrix-aware optimizer steps (Muon, SOAP, Newton-Schulz) on NVIDIA B200,
with AdamW for a model's other tensors and clipping over all gradients.

A thin Python binding of the C ABI in ``include/mo.h``: it turns torch
tensors into device pointers and the current CUDA stream into a handle, and
allocates the workspace with torch.  Every step of the computation runs in the
sm_100a kernels of ``libmo.so``; when that library is missing, importing the
binding's entry points fails.
"""

import ctypes
import warnings
from ctypes import byref, c_int32, c_int64, c_size_t, c_void_p

from . import _lib
from ._lib import (AdamW8Moments, AdamW8Tensor, AdamWCfg, AdamWTensor, ClipCfg, GemmDesc, Grad, MuonCfg, MuonMat,
                   NsCfg, PackCfg, SoapCfg, SoapMat, SoapMuonCfg, SoapMuonMat, OP_MUON, OP_NS, OP_SOAP)

__all__ = ["Context", "MoError", "TensorList", "QUINTIC", "OP_MUON", "OP_SOAP", "OP_NS"]

QUINTIC = (3.4445, -4.7750, 2.0315)


class MoError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"mo status {status}: {message}")
        self.status = status


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_f32(t, name):
    import torch
    if t is None:
        return
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")


def _check_state_shapes(i, d, keys):
    """Shapes of one SOAP / SOAP-Muon matrix's tensors: the library gets
    pointers only, so a mismatch here would address memory out of bounds."""
    W = d["W"]
    if W.dim() != 2:
        raise ValueError(f"matrix {i}: W must be 2-D")
    m, n = W.shape
    for k in keys:
        t = d.get(k)
        if t is not None and tuple(t.shape) != (m, n):
            raise ValueError(f"matrix {i}: {k} must have W's shape {(m, n)}")
    for fac, q, side in (("L", "QL", m), ("R", "QR", n)):
        for k in (fac, q):
            t = d.get(k)
            if t is not None and tuple(t.shape) != (side, side):
                raise ValueError(f"matrix {i}: {k} must be {side} x {side}")


def _check_extent(t, name, rows, cols, ld, stride, batch, dtypes):
    """A strided batch of rows x cols matrices (row stride ld, matrix stride
    stride, in elements) must lie inside the contiguous tensor t."""
    import torch
    if not t.is_cuda or not t.is_contiguous() or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a contiguous CUDA tensor of dtype {dtypes}")
    if ld < cols:
        raise ValueError(f"{name}: leading dimension {ld} < row length {cols}")
    last = (batch - 1) * stride + (rows - 1) * ld + cols
    if rows > 0 and cols > 0 and last > t.numel():
        raise ValueError(f"{name}: the {batch} x {rows} x {cols} operand (ld {ld}, stride {stride}) "
                         f"needs {last} elements, the tensor has {t.numel()}")


_TYPES = {}      # torch dtype -> the library's type, and whether a check allows it (filled on first use)


def _type(t, name, i, device, types):
    """The library's type of a flat tensor, checked: the library gets pointers only."""
    if not _TYPES:
        import torch
        _TYPES.update({torch.float32: (_lib.F32, "f32"), torch.bfloat16: (_lib.BF16, "bf16"),
                       torch.float16: (_lib.F16, "f16"), torch.uint8: (None, "u8")})
    code, kind = _TYPES.get(t.dtype, (None, ""))
    if kind not in types or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"tensor {i}: {name} must be a contiguous CUDA tensor of type {' or '.join(types)}")
    if t.device.index != device:
        raise ValueError(f"tensor {i}: {name} is on {t.device}, the context on cuda:{device}")
    return code


def _same_numel(t, name, i, numel):
    if t.numel() != numel:
        raise ValueError(f"tensor {i}: {name} must have {numel} elements, it has {t.numel()}")


def _scalar(t, name, device, dtype):
    """Device pointer of a one-element tensor (None passes through)."""
    if t is None:
        return None
    if t.dtype != dtype or not t.is_cuda or t.numel() != 1:
        raise ValueError(f"{name} must be a one-element {dtype} CUDA tensor")
    if t.device.index != device:
        raise ValueError(f"{name} is on {t.device}, the context on cuda:{device}")
    return t.data_ptr()


_NOT_GIVEN = object()


class TensorList:
    """A prepared list for adamw_step, adamw8_step, adamw8_pack / adamw8_unpack or clip_grads.

    The library's checks and launch tables of a list whose tensors stay in
    place, for a program that makes it once and passes it to every step.  It
    holds the tensors.  Made by Context.adamw_tensors, adamw8_tensors,
    adamw8_moments and clip_tensors."""

    def __init__(self, kind, lib, handle, tensors, device):
        self.kind, self.lib, self.handle, self.tensors, self.device = kind, lib, handle, tensors, device

    def __len__(self):
        return len(self.tensors)

    def __reduce__(self):
        raise TypeError("a TensorList owns a handle of the library and is not copied: make another one")

    def __del__(self):
        try:
            self.lib.mo_list_destroy(self.handle)
        except Exception:
            pass


class Context:
    """One library context on one CUDA device, with a torch-owned workspace."""

    _warned = False         # of adamw8_step(seed=...), once

    def __init__(self, device=None):
        import torch
        self.lib = _lib.load()
        self.device = torch.cuda.current_device() if device is None else int(device)
        self._device = torch.device("cuda", self.device)
        self._torch = torch
        h = c_void_p()
        st = self.lib.mo_ctx_create(byref(h), self.device)
        if st != 0:
            raise MoError(st, "mo_ctx_create failed")
        self.handle = h
        self._workspace = None
        self.retired = []       # workspaces replaced during stream capture, kept alive
        self._batch_reserved = {}

    def close(self):
        if getattr(self, "handle", None):
            self.lib.mo_ctx_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------ workspace
    @property
    def workspace(self):
        """The attached workspace tensor (None when detached)."""
        return self._workspace

    @workspace.setter
    def workspace(self, value):
        """Only None may be assigned: it detaches the workspace in the library
        (reading its status word first) and drops the tensor.  Use
        attach_workspace() or reserve() to attach one."""
        if value is not None:
            raise ValueError("assign None to detach; use attach_workspace() or reserve() to attach")
        if self._workspace is not None:
            self._check(self.lib.mo_set_workspace(self.handle, None, 0, self._stream(None)))
            self._workspace = None
            self._batch_reserved.clear()

    # ------------------------------------------------------------ helpers
    def _stream(self, stream):
        import torch
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        return c_void_p(s.cuda_stream)

    def _check(self, st):
        if st != 0:
            raise MoError(st, self.lib.mo_last_error(self.handle).decode())

    def workspace_bytes(self, op, shapes):
        n = len(shapes)
        rows = (c_int64 * max(n, 1))(*[int(s[0]) for s in shapes])
        cols = (c_int64 * max(n, 1))(*[int(s[1]) for s in shapes])
        mn, full = c_size_t(), c_size_t()
        self._check(self.lib.mo_workspace_bytes(self.handle, op, rows, cols, n, byref(mn), byref(full)))
        return mn.value, full.value

    def attach_workspace(self, nbytes, stream=None):
        """Allocate ``nbytes`` of device memory with torch, as memory of
        ``stream``, and attach it.

        Library work already enqueued may still use a workspace this one
        replaces, on any stream, and the switch itself copies the old status
        word on ``stream``.  Outside stream capture the device is synchronised
        before the old buffer goes back to torch's allocator.  During capture
        nothing can be synchronised: eager work enqueued before the capture
        may still be running, and the captured copy reads the old buffer
        whenever the graph replays.  So a buffer replaced during capture is
        kept alive (``retired``) until the next attach outside capture."""
        import torch
        with torch.cuda.stream(stream):         # else the current stream might still be writing it
            buf = torch.empty(int(nbytes), dtype=torch.uint8, device=f"cuda:{self.device}")
        self._check(self.lib.mo_set_workspace(self.handle, c_void_p(buf.data_ptr()), buf.numel(),
                                              self._stream(stream)))
        old, self._workspace = self._workspace, buf
        if old is not None:
            if torch.cuda.is_current_stream_capturing():
                self.retired.append(old)
            else:
                torch.cuda.synchronize(self.device)
                self.retired.clear()
        del old
        return buf

    def reserve(self, op, shapes, full=True, stream=None):
        """Make sure the attached workspace fits ``op`` on ``shapes``."""
        mn, fb = self.workspace_bytes(op, shapes)
        need = fb if full else mn
        if self.workspace is None or self.workspace.numel() < need:
            self.attach_workspace(need, stream)

    def device_status(self, stream=None):
        v = c_int32()
        st = self.lib.mo_device_status(self.handle, self._stream(stream), byref(v))
        if st not in (0, _lib.MO_ERR_DEVICE):
            self._check(st)
        return v.value

    def profile(self, enable=True):
        self._check(self.lib.mo_profile_enable(self.handle, int(enable)))

    def profile_read(self):
        """{kind: (ms, executed_flops, launches)} since the last read."""
        n = len(_lib.KINDS)
        ms = (ctypes.c_double * n)()
        fl = (ctypes.c_double * n)()
        ln = (c_int64 * n)()
        self._check(self.lib.mo_profile_read(self.handle, ms, fl, ln, n))
        return {k: (ms[i], fl[i], ln[i]) for i, k in enumerate(_lib.KINDS)}

    # ------------------------------------------------------------ entry points
    def muon_step(self, W, G, B, *, lr=0.02, weight_decay=0.01, momentum=0.95, nesterov=True,
                  momentum_ema=False, ns_steps=5, coeffs=QUINTIC, eps=1e-7,
                  adjust_lr="match_rms_adamw", nonfinite=None, stream=None, reserve=True):
        """One Muon step on lists of fp32 CUDA matrices (G entries may be None)."""
        n = len(W)
        if not (len(G) == len(B) == n):
            raise ValueError("W, G and B must have the same length")
        mats = (MuonMat * max(n, 1))()
        for i in range(n):
            for t, nm in ((W[i], "W"), (G[i], "G"), (B[i], "momentum")):
                _check_f32(t, f"{nm}[{i}]")
            if W[i].dim() != 2 or (G[i] is not None and G[i].shape != W[i].shape) or B[i].shape != W[i].shape:
                raise ValueError(f"matrix {i}: W, G and momentum must be 2-D with one shape")
            mats[i] = MuonMat(W[i].shape[0], W[i].shape[1], _ptr(W[i]), _ptr(G[i]), _ptr(B[i]))
        if reserve:
            self.reserve(OP_MUON, [tuple(w.shape) for w in W], stream=stream)
        modes = {"match_rms_adamw": 0, "original": 1}
        cfg = MuonCfg(lr, weight_decay, momentum, int(nesterov), int(momentum_ema), ns_steps,
                      coeffs[0], coeffs[1], coeffs[2], eps, modes[adjust_lr],
                      _ptr(nonfinite))
        self._check(self.lib.muon_step(self.handle, mats, n, byref(cfg), self._stream(stream)))

    def ns_orthogonalize(self, inputs, outputs=None, *, ns_steps=5, coeffs=QUINTIC, eps=1e-7,
                         nonfinite=None, stream=None, reserve=True):
        """O_i = NS(in_i); returns the list of fp32 outputs."""
        import torch
        n = len(inputs)
        if outputs is None:
            outputs = [torch.empty_like(x) for x in inputs]
        ins = (c_void_p * max(n, 1))()
        outs = (c_void_p * max(n, 1))()
        rows = (c_int64 * max(n, 1))()
        cols = (c_int64 * max(n, 1))()
        for i, (x, y) in enumerate(zip(inputs, outputs)):
            _check_f32(x, f"in[{i}]")
            _check_f32(y, f"out[{i}]")
            if x.dim() != 2 or y.shape != x.shape:
                raise ValueError(f"matrix {i}: input and output must be 2-D with one shape")
            ins[i], outs[i] = x.data_ptr(), y.data_ptr()
            rows[i], cols[i] = x.shape
        if reserve:
            self.reserve(OP_NS, [tuple(x.shape) for x in inputs], stream=stream)
        cfg = NsCfg(ns_steps, coeffs[0], coeffs[1], coeffs[2], eps, _ptr(nonfinite))
        self._check(self.lib.ns_orthogonalize(self.handle, ins, outs, rows, cols, n, byref(cfg),
                                              self._stream(stream)))
        return outputs

    def _reserve_batch(self, op, rows, cols, n, stream):
        """reserve() for n matrices of one shape, remembered per workspace so
        that repeated calls on the same batch cost no workspace query."""
        key = (op, rows, cols, n)
        if self.workspace is not None and self._batch_reserved.get(key) == self.workspace.data_ptr():
            return
        self.reserve(op, [(rows, cols)] * n, stream=stream)
        self._batch_reserved[key] = self.workspace.data_ptr()

    @staticmethod
    def _check_batch(t, name, shape=None):
        _check_f32(t, name)
        if t.dim() != 3 or (shape is not None and tuple(t.shape) != tuple(shape)):
            raise ValueError(f"{name} must be a 3-D [n, rows, cols] tensor" +
                             (f" of shape {tuple(shape)}" if shape is not None else ""))

    def ns_orthogonalize_batch(self, X, out=None, *, ns_steps=5, coeffs=QUINTIC, eps=1e-7, nonfinite=None,
                               stream=None, reserve=True):
        """out[i] = NS(X[i]) for a contiguous fp32 tensor X of shape [n, rows,
        cols] (e.g. per-head matrices): one call whatever n is."""
        import torch
        self._check_batch(X, "X")
        if out is None:
            out = torch.empty_like(X)
        self._check_batch(out, "out", X.shape)
        n, r, c = X.shape
        if reserve:
            self._reserve_batch(OP_NS, r, c, n, stream)
        cfg = NsCfg(ns_steps, coeffs[0], coeffs[1], coeffs[2], eps, _ptr(nonfinite))
        self._check(self.lib.ns_orthogonalize_strided(self.handle, _ptr(X), r * c, _ptr(out), r * c, r, c, n,
                                                      byref(cfg), self._stream(stream)))
        return out

    def muon_step_batch(self, W, G, B, *, lr=0.02, weight_decay=0.01, momentum=0.95, nesterov=True,
                        momentum_ema=False, ns_steps=5, coeffs=QUINTIC, eps=1e-7,
                        adjust_lr="match_rms_adamw", nonfinite=None, stream=None, reserve=True):
        """One Muon step on n matrices of one shape held as contiguous fp32
        [n, rows, cols] tensors W, G and B."""
        self._check_batch(W, "W")
        self._check_batch(G, "G", W.shape)
        self._check_batch(B, "B", W.shape)
        n, r, c = W.shape
        if reserve:
            self._reserve_batch(OP_MUON, r, c, n, stream)
        modes = {"match_rms_adamw": 0, "original": 1}
        cfg = MuonCfg(lr, weight_decay, momentum, int(nesterov), int(momentum_ema), ns_steps,
                      coeffs[0], coeffs[1], coeffs[2], eps, modes[adjust_lr], _ptr(nonfinite))
        self._check(self.lib.muon_step_strided(self.handle, _ptr(W), _ptr(G), _ptr(B), r * c, r, c, n,
                                               byref(cfg), self._stream(stream)))

    def soap_step(self, mats, step, *, lr=3e-3, beta1=0.95, beta2=0.95, shampoo_beta=None,
                  eps=1e-8, weight_decay=0.0, bias_correction=True, nonfinite=None, stream=None,
                  reserve=True, refresh=True, damping=0.0):
        """One SOAP step.  ``mats`` is a list of dicts with keys W, G, M, V and
        optionally L, QL, R, QR (missing or None: identity basis on that side).
        ``refresh=False`` keeps the bases this step (factors still update).
        ``damping``: 0 is the pages' power step qr(L Q); a positive value
        runs it on L + damping * trace(L) I instead (an option)."""
        n = len(mats)
        arr = (SoapMat * max(n, 1))()
        for i, d in enumerate(mats):
            for k in ("W", "G", "M", "V", "L", "QL", "R", "QR"):
                _check_f32(d.get(k), f"{k}[{i}]")
            _check_state_shapes(i, d, ("G", "M", "V"))
            W = d["W"]
            arr[i] = SoapMat(W.shape[0], W.shape[1], _ptr(W), _ptr(d.get("G")), _ptr(d["M"]),
                             _ptr(d["V"]), _ptr(d.get("L")), _ptr(d.get("QL")), _ptr(d.get("R")),
                             _ptr(d.get("QR")))
        if reserve:
            need = c_size_t()
            self._check(self.lib.mo_soap_workspace_bytes(self.handle, arr, n, byref(need)))
            if self.workspace is None or self.workspace.numel() < need.value:
                self.attach_workspace(need.value, stream)
        sb = beta2 if shampoo_beta is None else shampoo_beta
        cfg = SoapCfg(lr, beta1, beta2, sb, eps, weight_decay, int(bias_correction), _ptr(nonfinite),
                      0 if refresh else 1, damping)
        self._check(self.lib.soap_step(self.handle, arr, n, byref(cfg), int(step), self._stream(stream)))

    def soap_muon_step(self, mats, step, *, lr=0.02, weight_decay=0.01, momentum=0.95, nesterov=True,
                       beta2=0.95, shampoo_beta=0.9, eps=1e-8, bias_correction=True, ns_steps=5,
                       coeffs=QUINTIC, ns_eps=1e-7, adjust_lr="match_rms_adamw", damping=0.0,
                       nonfinite=None, refresh=True, stream=None, reserve=True):
        """One SOAP-Muon step.  ``mats``: dicts with W, G, B (Muon momentum), V
        and optionally L, QL, R, QR (missing or None: identity basis)."""
        n = len(mats)
        arr = (SoapMuonMat * max(n, 1))()
        for i, d in enumerate(mats):
            for k in ("W", "G", "B", "V", "L", "QL", "R", "QR"):
                _check_f32(d.get(k), f"{k}[{i}]")
            _check_state_shapes(i, d, ("G", "B", "V"))
            W = d["W"]
            arr[i] = SoapMuonMat(W.shape[0], W.shape[1], _ptr(W), _ptr(d.get("G")), _ptr(d["B"]),
                                 _ptr(d["V"]), _ptr(d.get("L")), _ptr(d.get("QL")), _ptr(d.get("R")),
                                 _ptr(d.get("QR")))
        if reserve:
            need = c_size_t()
            self._check(self.lib.mo_soap_muon_workspace_bytes(self.handle, arr, n, byref(need)))
            if self.workspace is None or self.workspace.numel() < need.value:
                self.attach_workspace(need.value, stream)
        modes = {"match_rms_adamw": 0, "original": 1}
        cfg = SoapMuonCfg(lr, weight_decay, momentum, int(nesterov), beta2, shampoo_beta, eps,
                          int(bias_correction), ns_steps, coeffs[0], coeffs[1], coeffs[2], ns_eps,
                          modes[adjust_lr], damping, _ptr(nonfinite), 0 if refresh else 1)
        self._check(self.lib.soap_muon_step(self.handle, arr, n, byref(cfg), int(step),
                                            self._stream(stream)))

    # ------------------------------------------------------------ AdamW, clipping
    def _prepare(self, kind, make, array, tensors):
        h = c_void_p()
        self._check(make(self.handle, array, len(tensors), byref(h)))
        return TensorList(kind, self.lib, h, tensors, self.device)

    def _list(self, kind, mats):
        """mats as a TensorList of this kind."""
        if not isinstance(mats, TensorList):
            return {"adamw": self.adamw_tensors, "adamw8": self.adamw8_tensors,
                    "moments": self.adamw8_moments, "grads": self.clip_tensors}[kind](mats)
        if mats.kind != kind or mats.device != self.device:
            raise ValueError(f"a list for {kind!r} on cuda:{self.device} is needed, "
                             f"this one is for {mats.kind!r} on cuda:{mats.device}")
        return mats

    def _step_fields(self, i, d):
        """What both kinds of AdamW tensors share."""
        W, G, copy = d["W"], d.get("G"), d.get("copy")
        n = W.numel()
        wt = _type(W, "W", i, self.device, ("f32", "bf16"))
        gt = ct = _lib.F32
        if G is not None:
            gt = _type(G, "G", i, self.device, ("f32", "bf16", "f16"))
            _same_numel(G, "G", i, n)
        if copy is not None:
            ct = _type(copy, "copy", i, self.device, ("bf16", "f16"))
            _same_numel(copy, "copy", i, n)
        return n, W, G, copy, (wt, gt, ct, d.get("lr_scale", 1.0), d.get("weight_decay", 0.0))

    def adamw_tensors(self, mats):
        """The list for adamw_step: dicts with W, G (None: skipped), M, V (fp32)
        and optionally copy, lr_scale (1) and weight_decay (0)."""
        arr, keep = (AdamWTensor * max(len(mats), 1))(), []
        for i, d in enumerate(mats):
            M, V = d["M"], d["V"]
            n, W, G, copy, rest = self._step_fields(i, d)
            for t, nm in ((M, "M"), (V, "V")):
                _type(t, nm, i, self.device, ("f32",))
                _same_numel(t, nm, i, n)
            keep.append((W, G, M, V, copy))
            arr[i] = AdamWTensor(n, _addr(W), _addr(G), _addr(M), _addr(V), _addr(copy), *rest)
        return self._prepare("adamw", self.lib.mo_adamw_list, arr, keep)

    def _codes(self, i, d, n):
        codes = [d["M8"], d["V8"], d["MS"], d["VS"]]
        for t, nm, size in zip(codes, ("M8", "V8", "MS", "VS"), (n, n, -(-n // 256), -(-n // 256))):
            _type(t, nm, i, self.device, ("u8",))
            _same_numel(t, nm, i, size)
        return codes

    def adamw8_tensors(self, mats):
        """The list for adamw8_step: as adamw_tensors with the moments' codes
        M8, V8 (uint8, one for each element) and scales MS, VS (uint8, one for
        each 256 elements) in the place of M and V."""
        arr, keep = (AdamW8Tensor * max(len(mats), 1))(), []
        for i, d in enumerate(mats):
            n, W, G, copy, rest = self._step_fields(i, d)
            codes = self._codes(i, d, n)
            keep.append((W, G, copy, *codes))
            arr[i] = AdamW8Tensor(n, _addr(W), _addr(G), *map(_addr, codes), _addr(copy), *rest)
        return self._prepare("adamw8", self.lib.mo_adamw8_list, arr, keep)

    def adamw8_state(self, W):
        """Zero 8-bit moments for the parameter W: a dict of M8, V8, MS and VS."""
        import torch
        n = W.numel()
        sizes = dict(M8=n, V8=n, MS=-(-n // 256), VS=-(-n // 256))
        return {k: torch.zeros(s, dtype=torch.uint8, device=W.device) for k, s in sizes.items()}

    def adamw8_moments(self, mats):
        """The list for adamw8_pack and adamw8_unpack: dicts with M8, V8, MS, VS
        and the moments M, V, both fp32 or both bf16."""
        arr, keep = (AdamW8Moments * max(len(mats), 1))(), []
        for i, d in enumerate(mats):
            M, V = d["M"], d["V"]
            n = M.numel()
            types = [_type(t, nm, i, self.device, ("f32", "bf16")) for t, nm in ((M, "M"), (V, "V"))]
            _same_numel(V, "V", i, n)
            if types[0] != types[1]:
                raise ValueError(f"tensor {i}: M and V must have one dtype")
            codes = self._codes(i, d, n)
            keep.append((M, V, *codes))
            arr[i] = AdamW8Moments(n, *map(_addr, codes), _addr(M), _addr(V), types[0])
        return self._prepare("moments", self.lib.mo_moments_list, arr, keep)

    def clip_tensors(self, grads):
        """The list for clip_grads: gradients, or dicts with G and out (None:
        scaled in place); a gradient that is None is skipped."""
        arr, keep = (Grad * max(len(grads), 1))(), []
        types = ("f32", "bf16", "f16")
        for i, d in enumerate(grads):
            G, out = (d["G"], d.get("out")) if isinstance(d, dict) else (d, None)
            keep.append((G, out))
            if G is None:
                continue
            gt = ot = _type(G, "G", i, self.device, types)
            if out is not None:
                ot = _type(out, "out", i, self.device, types)
                _same_numel(out, "out", i, G.numel())
            arr[i] = Grad(G.numel(), _addr(G), _addr(out), gt, ot)
        return self._prepare("grads", self.lib.mo_grad_list, arr, keep)

    def _raw_stream(self, stream):
        return (self._torch.cuda.current_stream(self.device) if stream is None else stream).cuda_stream

    def _adamw(self, fn, mats, step, lr, beta1, beta2, eps, bias_correction, grad_scale, skip, stochastic, seed, stream):
        torch = self._torch
        step_dev = lr_dev = None
        if isinstance(step, torch.Tensor):
            step, step_dev = 1, _scalar(step, "step", self.device, torch.int64)
        if isinstance(lr, torch.Tensor):
            lr, lr_dev = 0.0, _scalar(lr, "lr", self.device, torch.float32)
        cfg = AdamWCfg(lr, beta1, beta2, eps, bool(bias_correction), stochastic, seed or 0, lr_dev, step_dev,
                       _scalar(grad_scale, "grad_scale", self.device, torch.float32),
                       _scalar(skip, "skip", self.device, torch.int32))
        self._check(fn(self.handle, mats.handle, cfg, int(step), self._raw_stream(stream)))

    def adamw_step(self, mats, step, *, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, bias_correction=True,
                   grad_scale=None, skip=None, seed=None, stream=None):
        """One AdamW step on a list of tensors (adamw_tensors, or what it takes).

        ``step`` and ``lr`` are numbers, or one-element int64 / fp32 CUDA tensors
        read when the kernel runs.  ``grad_scale`` (fp32) multiplies every
        gradient, a nonzero ``skip`` (int32) leaves everything as it is.  With a
        ``seed`` bf16 weights are rounded stochastically, else to nearest."""
        self._adamw(self.lib.adamw_step_list, self._list("adamw", mats), step, lr, beta1, beta2, eps,
                    bias_correction, grad_scale, skip, seed is not None, seed, stream)

    @staticmethod
    def _rounding(noise, seed, default):
        """The library's kind of rounding of an 8-bit call, and its seed."""
        if seed is _NOT_GIVEN:
            noise = default if noise is _NOT_GIVEN else noise
            return int(noise is not None), noise
        if noise is not _NOT_GIVEN:
            raise ValueError("noise and seed are two kinds of rounding: give one of them")
        return 2 * (seed is not None), seed

    def adamw8_step(self, mats, step, *, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, bias_correction=True,
                    grad_scale=None, skip=None, noise=_NOT_GIVEN, seed=_NOT_GIVEN, stream=None):
        """One AdamW step with both moments in 8 bits (adamw8_tensors, or what
        it takes).  ``noise`` (0) is the seed with which both moments and bf16
        weights are rounded stochastically; None rounds to nearest, which leaves moments
        that change by less than half a code step where they are: over more than
        a few steps the first no longer follows the gradient.

        ``seed`` in place of ``noise`` is an earlier form, for runs that have to
        keep its bits: the first moment is rounded to nearest and sticks to its code
        while the second decays, so that weights without gradient run away."""
        stochastic, seed = self._rounding(noise, seed, 0)
        if stochastic == 2 and not Context._warned:
            Context._warned = True
            warnings.warn("adamw8_step(seed=...) rounds the first moment to the nearest code, where it sticks: "
                          "train with noise=...", stacklevel=2)
        self._adamw(self.lib.adamw8_step_list, self._list("adamw8", mats), step, lr, beta1, beta2, eps,
                    bias_correction, grad_scale, skip, stochastic, seed, stream)

    def adamw8_pack(self, mats, *, noise=_NOT_GIVEN, seed=_NOT_GIVEN, step=0, stream=None):
        """Moments M, V to 8-bit codes (adamw8_moments, or what it takes), to
        nearest; with ``noise`` both are rounded stochastically, with ``seed`` V
        alone, with the bits of ``step``."""
        torch = self._torch
        stochastic, seed = self._rounding(noise, seed, None)
        mats = self._list("moments", mats)
        step_dev = None
        if isinstance(step, torch.Tensor):
            step, step_dev = 0, _scalar(step, "step", self.device, torch.int64)
        cfg = PackCfg(stochastic, seed or 0, int(step), step_dev)
        self._check(self.lib.adamw8_pack_list(self.handle, mats.handle, cfg, self._raw_stream(stream)))

    def adamw8_unpack(self, mats, *, stream=None):
        """The values that 8-bit codes stand for, written to M and V."""
        mats = self._list("moments", mats)
        self._check(self.lib.adamw8_unpack_list(self.handle, mats.handle, self._raw_stream(stream)))

    def clip_grads(self, grads, max_norm, *, apply=True, scale=None, nonfinite=None, stream=None, reserve=True):
        """Scales the gradients of a list (clip_tensors, or what it takes) so that
        their common 2-norm is at most ``max_norm``; returns (norm, factor) as
        fp32 device scalars.  ``apply=False`` computes these alone (adamw_step
        takes the factor as grad_scale).  ``scale`` (fp32 device scalar)
        multiplies the gradients first; ``nonfinite`` (int32 device scalar)
        receives 1 when the norm is not finite."""
        torch = self._torch
        grads = self._list("grads", grads)
        if reserve and (self._workspace is None or self._workspace.numel() < _lib.CLIP_WORKSPACE_BYTES):
            self.attach_workspace(_lib.CLIP_WORKSPACE_BYTES, stream)
        if stream is None:
            norm, factor = torch.empty(2, dtype=torch.float32, device=self._device).unbind()
        else:
            with torch.cuda.stream(stream):     # the scalars belong to the stream that writes them
                norm, factor = torch.empty(2, dtype=torch.float32, device=self._device).unbind()
        at = norm.data_ptr()
        cfg = ClipCfg(max_norm, bool(apply), _scalar(scale, "scale", self.device, torch.float32), at, at + 4,
                      _scalar(nonfinite, "nonfinite", self.device, torch.int32))
        self._check(self.lib.clip_grads_list(self.handle, grads.handle, cfg, self._raw_stream(stream)))
        return norm, factor

    def gemm_bf16(self, A, B, D, *, M, N, K, batch=1, a_mn=False, b_mn=False, sym=False,
                  alpha=1.0, beta=0.0, C=None, scale=None, alpha_pow=0, beta_pow=0,
                  lda=None, ldb=None, ldc=None, ldd=None, strideA=None, strideB=None,
                  strideC=None, strideD=None, band=0, stream=None):
        """Batched bf16 tensor-core GEMM with the fused epilogue (see mo.h)."""
        import torch

        def ld_of(t):
            return t.shape[-1]

        def stride_of(t):
            return t.shape[-1] * t.shape[-2] if t.dim() == 3 else 0

        d = GemmDesc()
        d.A, d.lda, d.strideA, d.a_mn = A.data_ptr(), lda or ld_of(A), strideA or stride_of(A), int(a_mn)
        d.B, d.ldb, d.strideB, d.b_mn = B.data_ptr(), ldb or ld_of(B), strideB or stride_of(B), int(b_mn)
        d.M, d.N, d.K, d.batch, d.sym = M, N, K, batch, int(sym)
        d.alpha, d.beta = alpha, beta
        d.scale = None if scale is None else scale.data_ptr()
        d.alpha_pow, d.beta_pow = alpha_pow, beta_pow
        if C is not None:
            d.C, d.ldc, d.strideC = C.data_ptr(), ldc or ld_of(C), strideC or stride_of(C)
            d.c_f32 = int(C.dtype == torch.float32)
        d.D, d.ldd, d.strideD = D.data_ptr(), ldd or ld_of(D), strideD or stride_of(D)
        d.d_f32 = int(D.dtype == torch.float32)
        d.band = band
        bf16, outs = (torch.bfloat16,), (torch.bfloat16, torch.float32)
        _check_extent(A, "A", K if a_mn else M, M if a_mn else K, d.lda, d.strideA, batch, bf16)
        _check_extent(B, "B", K if b_mn else N, N if b_mn else K, d.ldb, d.strideB, batch, bf16)
        _check_extent(D, "D", M, N, d.ldd, d.strideD, batch, outs)
        if C is not None:
            _check_extent(C, "C", M, N, d.ldc, d.strideC, batch, outs)
        if self.workspace is None:
            self.attach_workspace(4096, stream)
        self._check(self.lib.mo_gemm_bf16(self.handle, byref(d), self._stream(stream)))
