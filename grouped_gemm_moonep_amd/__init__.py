"""MoonEP hot path on AMD MI355X (gfx950): Python binding of libmoonep.so.

`Buffer` mirrors the MoonEP README's Buffer (MoonshotAI/MoonEP mirror,
"API guide"), for all R EP ranks of one GPU at once.  Each method is one call
of the C ABI of the same name (include/moonep.h) with torch tensors supplying
device memory and the current stream; nothing is computed in Python.

    buf = Buffer(R=8, S=4096, K=8, E=256, B=32, H=7168, Hp=2048, token_padding=128)
    plan = buf.plan(topk)                           # moonep_plan
    x_nvs, rw_nvs = buf.dispatch(plan, x, rw)       # moonep_dispatch
    buf.prefetch_weight(plan, home, pool)           # moonep_prefetch_weight
    buf.expert_ffn(plan, x_nvs, home, pool, z, y)   # moonep_expert_ffn
                                                    # (= expert_gateup + expert_down)
    out, rw_sk = buf.combine(plan, y, rw_nvs)       # moonep_combine

Around it, what a training step needs next (framework-side steps on the pages):
`Buffer.route` / `route_bwd` (the router's choice, its weights and their
gradient), `Buffer.combine_bwd` (the gradient of the weighted combine) and
`orthogonalize` (the Muon optimiser's direction of the weight gradients):

    topk, rw = buf.route(logits)                    # moonep_route
    dy, drw = buf.combine_bwd(plan, dout, y, rw_nvs)  # moonep_combine_bwd
    dlogits = buf.route_bwd(logits, topk, drw)      # moonep_route_bwd
    direction = orthogonalize(grad_home)            # moonep_orthogonalize

and what a block has around its experts: `shared_ffn` (the expert that every
token passes, added to combine's output), `block_norm` (the block's end and the
next one's start) and their gradients `shared_ffn_bwd` and `block_norm_bwd`:

    both = shared_ffn(u, (gate, up, down), add=out)          # moonep_shared_ffn
    h, u = block_norm(h, both, w_post=p, w_pre=n)            # moonep_block_norm
    dh, dy, dg, dp, dn = block_norm_bwd(h, dh, du, both, w_post=p, w_pre=n)
    du, dw = shared_ffn_bwd(u, dy, (gate, up, down))         # moonep_shared_ffn_bwd

`SymmetricBuffer` is the README's [E+B,H,H'] weight (or fp32 gradient) buffer
of one projection on virtual memory (moonep_symbuf_*): per-rank views whose
rows [0,E) map every rank's home chunk, with the *_views methods addressing
experts purely by row index.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _abi
from ._abi import MoonepError, lib  # noqa: F401

__all__ = ["Buffer", "Plan", "SymmetricBuffer", "MoonepError", "lib", "vmm_granularity",
           "orthogonalize", "orthogonalize_workspace", "block_norm", "block_norm_bwd",
           "block_norm_bwd_workspace", "shared_ffn", "shared_ffn_bwd", "shared_ffn_workspace",
           "shared_ffn_bwd_workspace"]


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev_ptr(t, dtype, shape, name, nullable=False):
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_FLOATS = {torch.float32: _abi.F32, torch.bfloat16: _abi.BF16}


def _float_type(t, name):
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32 or bfloat16, got {t.dtype}")
    return code


def _score(score):
    if score not in _abi.SCORES:
        raise ValueError(f"score: expected one of {sorted(_abi.SCORES)}, got {score!r}")
    return _abi.SCORES[score]


def _same_device(device, **tensors):
    """The calls below launch on `device`: every tensor has to be there."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name}: expected device {device}, got {t.device}")


def _apart(name, out, /, **inputs):
    """`out`, a tensor of the caller's, must not share memory with any of `inputs`."""
    o0 = out.data_ptr()
    o1 = o0 + out.nbytes
    for n, t in inputs.items():
        if t is not None:
            p = t.data_ptr()
            if p < o1 and o0 < p + t.nbytes:
                raise ValueError(f"{name} must not overlap {n}")


def _stream_of(i):
    return torch.cuda.current_stream(i).cuda_stream


# What torch.cuda's own functions call, a microsecond less each; torch does not promise them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(dev, name, *args):
    """The C call `name` on the current stream of `dev`, which is made current for it."""
    f, i = getattr(lib(), name), dev.index
    if i == _current_device():
        status = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(i))
    if status:
        _abi.check(status, name)


class Plan:
    """Device arrays of one plan (see moonep_plan_t)."""

    def __init__(self, cfg, device):
        self.arrays = {}
        self._store = []
        for i, name in enumerate(_abi.PLAN_ARRAYS):
            n = _abi.plan_len(cfg, i)
            # zero-length arrays (B = 0) still get a valid device pointer
            store = torch.empty(max(n, 1), dtype=torch.int32, device=device)
            self.arrays[name] = store[:n]
            self._store.append(store)
        self.struct = _abi.MoonepPlan(*[s.data_ptr() for s in self._store])

    def __getattr__(self, name):
        arrays = self.__dict__.get("arrays")
        if arrays is not None and name in arrays:
            return arrays[name]
        raise AttributeError(name)


class Buffer:
    """Handle of the MoonEP path for R ranks on the current device."""

    def __init__(self, R, S, K, E, B=None, H=7168, Hp=2048, token_padding=128, num_cus=0,
                 device="cuda"):
        if B is None:
            B = E // R
        self.R, self.S, self.K, self.E, self.B = R, S, K, E, B
        self.H, self.Hp, self.token_padding = H, Hp, token_padding
        self.device = torch.device(device)
        self.cfg = _abi.config(R, S, K, E, B, H, Hp, token_padding, num_cus)
        self.NvS = _abi.nvs(self.cfg)
        if self.NvS < 0:
            raise MoonepError(_abi.MOONEP_ERR_CONFIG, "Buffer")
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _abi.check(lib().moonep_create(ctypes.byref(self.cfg), ctypes.byref(self._h)),
                       "moonep_create")

    # -- lifecycle -----------------------------------------------------------
    def destroy(self):
        if self._h:
            _abi.check(lib().moonep_destroy(self._h), "moonep_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def new_plan(self):
        return Plan(self.cfg, self.device)

    # -- calls -----------------------------------------------------------------
    def plan(self, topk, tokens_per_expert=None, plan=None):
        plan = plan or self.new_plan()
        R, S, K, E = self.R, self.S, self.K, self.E
        p_topk = _dev_ptr(topk, torch.int32, (R, S, K), "topk")
        p_tpe = _dev_ptr(tokens_per_expert, torch.int32, (R, E), "tokens_per_expert", True)
        _abi.check(lib().moonep_plan(self._h, p_topk, p_tpe, ctypes.byref(plan.struct), _stream()),
                   "moonep_plan")
        return plan

    def plan_noalloc(self, topk, tokens_per_expert=None, plan=None):
        """moonep_plan_noalloc: the same plan as `plan`, computed without the
        handle's scratch and without allocating device memory (the library's
        fixed per-GPU scratch array; concurrent calls on one GPU race).  Only
        `plan=None` allocates here, in Python, for the plan arrays."""
        plan = plan or self.new_plan()
        R, S, K, E = self.R, self.S, self.K, self.E
        p_topk = _dev_ptr(topk, torch.int32, (R, S, K), "topk")
        p_tpe = _dev_ptr(tokens_per_expert, torch.int32, (R, E), "tokens_per_expert", True)
        _abi.check(lib().moonep_plan_noalloc(ctypes.byref(self.cfg), p_topk, p_tpe,
                                             ctypes.byref(plan.struct), _stream()),
                   "moonep_plan_noalloc")
        return plan

    def copy_rows(self, plan, src_nvs, dst_nvs=None):
        """The used slots of every rank from src_nvs to dst_nvs (moonep_copy_rows)."""
        R, NvS = self.R, self.NvS
        W = src_nvs.shape[-1]
        if dst_nvs is None:
            dst_nvs = torch.empty_like(src_nvs)
        args = (_dev_ptr(src_nvs, torch.bfloat16, (R, NvS, W), "src_nvs"), int(W),
                _dev_ptr(dst_nvs, torch.bfloat16, (R, NvS, W), "dst_nvs"))
        _abi.check(lib().moonep_copy_rows(self._h, ctypes.byref(plan.struct), *args, _stream()),
                   "moonep_copy_rows")
        return dst_nvs

    def _comm(self, W, device):
        """The communication buffer of the copy mode (zero_copy=False), one per
        row width, owned by this Buffer."""
        bufs = self.__dict__.setdefault("_comm_bufs", {})
        if W not in bufs:
            bufs[W] = torch.empty((self.R, self.NvS, W), dtype=torch.bfloat16, device=device)
        return bufs[W]

    def dispatch(self, plan, x, rw=None, x_nvs=None, rw_nvs=None, zero_copy=True):
        """zero_copy=False (the README's copy mode): dispatch into this Buffer's
        communication buffer, then copy the used slots into x_nvs."""
        if not zero_copy:
            comm, rw_nvs = self.dispatch(plan, x, rw, x_nvs=self._comm(x.shape[-1], x.device),
                                         rw_nvs=rw_nvs)
            return self.copy_rows(plan, comm, x_nvs), rw_nvs
        R, S, K, NvS = self.R, self.S, self.K, self.NvS
        W = x.shape[-1]
        if x_nvs is None:
            x_nvs = torch.empty((R, NvS, W), dtype=torch.bfloat16, device=x.device)
        if rw is not None and rw_nvs is None:
            rw_nvs = torch.empty((R, NvS), dtype=torch.float32, device=x.device)
        args = (_dev_ptr(x, torch.bfloat16, (R, S, W), "x"), int(W),
                _dev_ptr(rw, torch.float32, (R, S, K), "rw", True),
                _dev_ptr(x_nvs, torch.bfloat16, (R, NvS, W), "x_nvs"),
                _dev_ptr(rw_nvs, torch.float32, (R, NvS), "rw_nvs", True))
        _abi.check(lib().moonep_dispatch(self._h, ctypes.byref(plan.struct), *args, _stream()),
                   "moonep_dispatch")
        return x_nvs, rw_nvs

    def combine(self, plan, y_nvs, rw_nvs=None, out=None, rw_sk=None, gather_rw=True,
                zero_copy=True):
        """zero_copy=False (the README's copy mode): copy the used slots of
        y_nvs into this Buffer's communication buffer first, then combine."""
        if not zero_copy:
            comm = self.copy_rows(plan, y_nvs, self._comm(y_nvs.shape[-1], y_nvs.device))
            return self.combine(plan, comm, rw_nvs, out, rw_sk, gather_rw)
        R, S, K, NvS = self.R, self.S, self.K, self.NvS
        W = y_nvs.shape[-1]
        if out is None:
            out = torch.empty((R, S, W), dtype=torch.bfloat16, device=y_nvs.device)
        if rw_nvs is not None and rw_sk is None and gather_rw:
            rw_sk = torch.empty((R, S, K), dtype=torch.float32, device=y_nvs.device)
        args = (_dev_ptr(y_nvs, torch.bfloat16, (R, NvS, W), "y_nvs"), int(W),
                _dev_ptr(rw_nvs, torch.float32, (R, NvS), "rw_nvs", True),
                _dev_ptr(out, torch.bfloat16, (R, S, W), "out"),
                _dev_ptr(rw_sk, torch.float32, (R, S, K), "rw_sk", True))
        _abi.check(lib().moonep_combine(self._h, ctypes.byref(plan.struct), *args, _stream()),
                   "moonep_combine")
        return out, rw_sk

    def combine_bwd(self, plan, dout, y_nvs, rw_nvs, dy_nvs=None, drw=None, need_drw=True):
        """Gradient of the weighted combine: (dy_nvs, drw) from dout [R,S,W],
        the forward's y_nvs [R,NvS,W] and rw_nvs [R,NvS].  dy_nvs may be y_nvs
        (in place).  need_drw=False: the route weights need no gradient, drw is
        None and y_nvs may be None."""
        R, S, K, NvS = self.R, self.S, self.K, self.NvS
        W = dout.shape[-1]
        dev = dout.device
        if drw is not None and not need_drw:
            raise ValueError("drw given, but need_drw is False")
        args = (_dev_ptr(dout, torch.bfloat16, (R, S, W), "dout"), W,
                _dev_ptr(y_nvs, torch.bfloat16, (R, NvS, W), "y_nvs", not need_drw),
                _dev_ptr(rw_nvs, torch.float32, (R, NvS), "rw_nvs"))
        _same_device(dev, y_nvs=y_nvs, rw_nvs=rw_nvs, plan=plan.arrays["dest"])
        if dy_nvs is None:
            dy_nvs = torch.empty((R, NvS, W), dtype=torch.bfloat16, device=dev)
            p_dy = dy_nvs.data_ptr()
        else:
            p_dy = _dev_ptr(dy_nvs, torch.bfloat16, (R, NvS, W), "dy_nvs")
            _same_device(dev, dy_nvs=dy_nvs)
            _apart("dy_nvs", dy_nvs, dout=dout, rw_nvs=rw_nvs,
                   y_nvs=None if p_dy == args[2] else y_nvs)
        if drw is not None:
            p_drw = _dev_ptr(drw, torch.float32, (R, S, K), "drw")
            _same_device(dev, drw=drw)
            _apart("drw", drw, dout=dout, y_nvs=y_nvs, rw_nvs=rw_nvs, dy_nvs=dy_nvs)
        elif need_drw:
            drw = torch.empty(R, S, K, dtype=torch.float32, device=dev)
            p_drw = drw.data_ptr()
        else:
            p_drw = None
        _launch(dev, "moonep_combine_bwd", self._h, ctypes.byref(plan.struct), *args, p_dy, p_drw)
        return dy_nvs, drw

    def route(self, logits, bias=None, score="softmax", normalize=True, scale=1.0, topk=None,
              rw=None):
        """The router's choice: (topk [R,S,K] int32, rw [R,S,K] fp32) from logits
        [R,S,E] (float32 or bfloat16).  score: "softmax" or "sigmoid"; bias [E]
        fp32 (selection only): the choice goes by score + bias instead of the
        logit; normalize: the K weights are divided by their sum; scale
        multiplies them.  A logit of -inf closes its expert."""
        R, S, K, E = self.R, self.S, self.K, self.E
        dev = logits.device
        args = (_dev_ptr(logits, logits.dtype, (R, S, E), "logits"),
                _float_type(logits, "logits"),
                _dev_ptr(bias, torch.float32, (E,), "bias", True), _score(score),
                1 if normalize else 0, scale)
        if bias is not None and bias.device != dev:
            _same_device(dev, bias=bias)
        if topk is None:
            topk = torch.empty(R, S, K, dtype=torch.int32, device=dev)
        else:
            _dev_ptr(topk, torch.int32, (R, S, K), "topk")
            _same_device(dev, topk=topk)
            _apart("topk", topk, logits=logits, bias=bias, rw=rw)
        if rw is None:
            rw = torch.empty(R, S, K, dtype=torch.float32, device=dev)
        else:
            _dev_ptr(rw, torch.float32, (R, S, K), "rw")
            _same_device(dev, rw=rw)
            _apart("rw", rw, logits=logits, bias=bias)
        _launch(dev, "moonep_route", self._h, *args, topk.data_ptr(), rw.data_ptr())
        return topk, rw

    def route_bwd(self, logits, topk, drw, score="softmax", normalize=True, scale=1.0,
                  dlogits=None):
        """Gradient of route's weights: dlogits [R,S,E] in the logits' type from
        drw [R,S,K] fp32, for the topk and the form of the forward call (the
        selection bias takes no part).  dlogits may be logits (in place)."""
        R, S, K, E = self.R, self.S, self.K, self.E
        dev = logits.device
        args = (_dev_ptr(logits, logits.dtype, (R, S, E), "logits"),
                _float_type(logits, "logits"), _score(score), 1 if normalize else 0, scale,
                _dev_ptr(topk, torch.int32, (R, S, K), "topk"),
                _dev_ptr(drw, torch.float32, (R, S, K), "drw"))
        _same_device(dev, topk=topk, drw=drw)
        if dlogits is None:
            dlogits = torch.empty_like(logits)
        elif dlogits is not logits:
            p = _dev_ptr(dlogits, logits.dtype, (R, S, E), "dlogits")
            _same_device(dev, dlogits=dlogits)
            _apart("dlogits", dlogits, topk=topk, drw=drw,
                   logits=None if p == args[0] else logits)
        _launch(dev, "moonep_route_bwd", self._h, *args, dlogits.data_ptr())
        return dlogits

    def _weights(self, ts, pool, used=(0, 1, 2)):
        R, E, B, H, Hp = self.R, self.E, self.B, self.H, self.Hp
        if len(ts) != 3:
            raise ValueError("three projections (gate, up, down) expected")
        shape = (R, B, H, Hp) if pool else (E, H, Hp)
        for i, t in enumerate(ts):
            if t is None and (i not in used or (pool and B == 0)):
                continue
            _dev_ptr(t, torch.bfloat16, shape, f"{'pool' if pool else 'home'}[{i}]")
        return _abi.ptr3(ts)

    def prefetch_weight(self, plan, home, pool):
        _abi.check(lib().moonep_prefetch_weight(self._h, ctypes.byref(plan.struct),
                                                self._weights(home, False),
                                                self._weights(pool, True), _stream()),
                   "moonep_prefetch_weight")

    def expert_ffn(self, plan, x_nvs, home, pool, z_ws=None, y_nvs=None, rank=-1):
        R, NvS, H, Hp = self.R, self.NvS, self.H, self.Hp
        if z_ws is None:
            z_ws = torch.empty((R, NvS, Hp), dtype=torch.bfloat16, device=x_nvs.device)
        if y_nvs is None:
            y_nvs = torch.empty((R, NvS, H), dtype=torch.bfloat16, device=x_nvs.device)
        args = (int(rank), _dev_ptr(x_nvs, torch.bfloat16, (R, NvS, H), "x_nvs"),
                self._weights(home, False), self._weights(pool, True),
                _dev_ptr(z_ws, torch.bfloat16, (R, NvS, Hp), "z_ws"),
                _dev_ptr(y_nvs, torch.bfloat16, (R, NvS, H), "y_nvs"))
        _abi.check(lib().moonep_expert_ffn(self._h, ctypes.byref(plan.struct), *args, _stream()),
                   "moonep_expert_ffn")
        return z_ws, y_nvs

    def _views(self, views):
        R, E, B, H, Hp = self.R, self.E, self.B, self.H, self.Hp
        if len(views) != 3:
            raise ValueError("three projections (gate, up, down) expected")
        for i, t in enumerate(views):
            _dev_ptr(t, torch.bfloat16, (R, E + B, H, Hp), f"views[{i}]")
        return _abi.ptr3(views)

    def prefetch_weight_views(self, plan, views):
        """prefetch_weight over per-rank [E+B] views (views[p] [R,E+B,H,Hp])."""
        _abi.check(lib().moonep_prefetch_weight_views(self._h, ctypes.byref(plan.struct),
                                                      self._views(views), _stream()),
                   "moonep_prefetch_weight_views")

    def expert_ffn_views(self, plan, x_nvs, views, z_ws=None, y_nvs=None, rank=-1):
        """expert_ffn with experts located by row index in rank d's [E+B] view."""
        R, NvS, H, Hp = self.R, self.NvS, self.H, self.Hp
        if z_ws is None:
            z_ws = torch.empty((R, NvS, Hp), dtype=torch.bfloat16, device=x_nvs.device)
        if y_nvs is None:
            y_nvs = torch.empty((R, NvS, H), dtype=torch.bfloat16, device=x_nvs.device)
        args = (int(rank), _dev_ptr(x_nvs, torch.bfloat16, (R, NvS, H), "x_nvs"),
                self._views(views),
                _dev_ptr(z_ws, torch.bfloat16, (R, NvS, Hp), "z_ws"),
                _dev_ptr(y_nvs, torch.bfloat16, (R, NvS, H), "y_nvs"))
        _abi.check(lib().moonep_expert_ffn_views(self._h, ctypes.byref(plan.struct), *args,
                                                 _stream()), "moonep_expert_ffn_views")
        return z_ws, y_nvs

    def expert_gateup(self, plan, x_nvs, home, pool, z_nvs=None, rank=-1):
        R, NvS, H, Hp = self.R, self.NvS, self.H, self.Hp
        if z_nvs is None:
            z_nvs = torch.empty((R, NvS, Hp), dtype=torch.bfloat16, device=x_nvs.device)
        args = (int(rank), _dev_ptr(x_nvs, torch.bfloat16, (R, NvS, H), "x_nvs"),
                self._weights(home, False, (0, 1)), self._weights(pool, True, (0, 1)),
                _dev_ptr(z_nvs, torch.bfloat16, (R, NvS, Hp), "z_nvs"))
        _abi.check(lib().moonep_expert_gateup(self._h, ctypes.byref(plan.struct), *args,
                                              _stream()), "moonep_expert_gateup")
        return z_nvs

    def expert_down(self, plan, z_nvs, home, pool, y_nvs=None, rank=-1):
        R, NvS, H, Hp = self.R, self.NvS, self.H, self.Hp
        if y_nvs is None:
            y_nvs = torch.empty((R, NvS, H), dtype=torch.bfloat16, device=z_nvs.device)
        args = (int(rank), _dev_ptr(z_nvs, torch.bfloat16, (R, NvS, Hp), "z_nvs"),
                self._weights(home, False, (2,)), self._weights(pool, True, (2,)),
                _dev_ptr(y_nvs, torch.bfloat16, (R, NvS, H), "y_nvs"))
        _abi.check(lib().moonep_expert_down(self._h, ctypes.byref(plan.struct), *args,
                                            _stream()), "moonep_expert_down")
        return y_nvs

    def expert_ffn_bwd(self, plan, x_nvs, dy_nvs, home, pool, dz_ws=None, dg_nvs=None,
                       du_nvs=None, dx_nvs=None, rank=-1):
        """Backward of the grouped SwiGLU FFN: returns (dz_ws, dg_nvs, du_nvs,
        dx_nvs); dx_nvs may be dy_nvs or x_nvs (in place)."""
        R, NvS, H, Hp = self.R, self.NvS, self.H, self.Hp
        dev = x_nvs.device
        new = lambda W: torch.empty((R, NvS, W), dtype=torch.bfloat16, device=dev)
        dz_ws = new(Hp) if dz_ws is None else dz_ws
        dg_nvs = new(Hp) if dg_nvs is None else dg_nvs
        du_nvs = new(Hp) if du_nvs is None else du_nvs
        dx_nvs = new(H) if dx_nvs is None else dx_nvs
        args = (int(rank), _dev_ptr(x_nvs, torch.bfloat16, (R, NvS, H), "x_nvs"),
                _dev_ptr(dy_nvs, torch.bfloat16, (R, NvS, H), "dy_nvs"),
                self._weights(home, False), self._weights(pool, True),
                _dev_ptr(dz_ws, torch.bfloat16, (R, NvS, Hp), "dz_ws"),
                _dev_ptr(dg_nvs, torch.bfloat16, (R, NvS, Hp), "dg_nvs"),
                _dev_ptr(du_nvs, torch.bfloat16, (R, NvS, Hp), "du_nvs"),
                _dev_ptr(dx_nvs, torch.bfloat16, (R, NvS, H), "dx_nvs"))
        _abi.check(lib().moonep_expert_ffn_bwd(self._h, ctypes.byref(plan.struct), *args,
                                               _stream()), "moonep_expert_ffn_bwd")
        return dz_ws, dg_nvs, du_nvs, dx_nvs

    def expert_ffn_bwd_views(self, plan, x_nvs, dy_nvs, views, dz_ws=None, dg_nvs=None,
                             du_nvs=None, dx_nvs=None, rank=-1):
        """expert_ffn_bwd with experts located by row index in rank d's [E+B] view."""
        R, NvS, H, Hp = self.R, self.NvS, self.H, self.Hp
        dev = x_nvs.device
        new = lambda W: torch.empty((R, NvS, W), dtype=torch.bfloat16, device=dev)
        dz_ws = new(Hp) if dz_ws is None else dz_ws
        dg_nvs = new(Hp) if dg_nvs is None else dg_nvs
        du_nvs = new(Hp) if du_nvs is None else du_nvs
        dx_nvs = new(H) if dx_nvs is None else dx_nvs
        args = (int(rank), _dev_ptr(x_nvs, torch.bfloat16, (R, NvS, H), "x_nvs"),
                _dev_ptr(dy_nvs, torch.bfloat16, (R, NvS, H), "dy_nvs"),
                self._views(views),
                _dev_ptr(dz_ws, torch.bfloat16, (R, NvS, Hp), "dz_ws"),
                _dev_ptr(dg_nvs, torch.bfloat16, (R, NvS, Hp), "dg_nvs"),
                _dev_ptr(du_nvs, torch.bfloat16, (R, NvS, Hp), "du_nvs"),
                _dev_ptr(dx_nvs, torch.bfloat16, (R, NvS, H), "dx_nvs"))
        _abi.check(lib().moonep_expert_ffn_bwd_views(self._h, ctypes.byref(plan.struct), *args,
                                                     _stream()), "moonep_expert_ffn_bwd_views")
        return dz_ws, dg_nvs, du_nvs, dx_nvs

    def expert_wgrad(self, plan, a_nvs, b_nvs, grad_home, reduce_buf, rank=-1):
        R, NvS, E, B, H, Hp = self.R, self.NvS, self.E, self.B, self.H, self.Hp
        args = (int(rank), _dev_ptr(a_nvs, torch.bfloat16, (R, NvS, H), "a_nvs"),
                _dev_ptr(b_nvs, torch.bfloat16, (R, NvS, Hp), "b_nvs"),
                _dev_ptr(grad_home, torch.float32, (E, H, Hp), "grad_home"),
                _dev_ptr(reduce_buf, torch.float32, (R, B, H, Hp), "reduce_buf"))
        _abi.check(lib().moonep_expert_wgrad(self._h, ctypes.byref(plan.struct), *args, _stream()),
                   "moonep_expert_wgrad")

    def reduce_grad(self, plan, grad_home, reduce_buf):
        R, E, B, H, Hp = self.R, self.E, self.B, self.H, self.Hp
        for i in range(3):
            _dev_ptr(grad_home[i], torch.float32, (E, H, Hp), f"grad_home[{i}]")
            _dev_ptr(reduce_buf[i], torch.float32, (R, B, H, Hp), f"reduce_buf[{i}]")
        _abi.check(lib().moonep_reduce_grad(self._h, ctypes.byref(plan.struct),
                                            _abi.ptr3(grad_home), _abi.ptr3(reduce_buf),
                                            _stream()),
                   "moonep_reduce_grad")

    def read_stats(self, plan):
        import numpy as np
        out = np.zeros(_abi.STAT_FIXED + 2 * self.R, dtype=np.int32)
        _abi.check(lib().moonep_read_stats(self._h, ctypes.byref(plan.struct),
                                           out.ctypes.data_as(ctypes.c_void_p), _stream()),
                   "moonep_read_stats")
        return out


def vmm_granularity():
    """Minimum virtual-memory allocation granularity of the current device, bytes."""
    g = ctypes.c_int64()
    _abi.check(lib().moonep_vmm_granularity(ctypes.byref(g)), "moonep_vmm_granularity")
    return int(g.value)


MUON_COEFFS = (3.4445, -4.7750, 2.0315)


def orthogonalize_workspace(n, rows, cols, device="cuda"):
    """Workspace tensor of `orthogonalize` for n matrices of rows x cols."""
    nbytes = int(lib().moonep_orthogonalize_ws(n, rows, cols))
    if nbytes < 0:
        raise MoonepError(_abi.MOONEP_ERR_CONFIG, "moonep_orthogonalize_ws")
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _refused_steps(flat, eps):
    """What moonep_orthogonalize refuses of the steps (a, b, c) and eps, or None."""
    args = (ctypes.c_float * (3 * len(flat)))(*[v for c in flat for v in c])
    # of no matrices it looks at nothing else
    if not lib().moonep_orthogonalize(None, _abi.F32, 0, 1, 1, args, len(flat), eps, None, None, 0,
                                      None):
        return None
    if not 1 <= len(flat) <= _abi.ORTHO_MAX_STEPS:
        return f"{len(flat)} steps, 1 to {_abi.ORTHO_MAX_STEPS} are taken"
    if not eps > 0:
        return f"eps {eps}, it has to be positive"
    if not all(math.isfinite(v) for c in flat for v in c) or not all(c[0] > 0 for c in flat):
        return "coefficients that are not finite, or an a that is not positive"
    gain = math.prod(c[0] for c in flat)
    if gain > _abi.ORTHO_MAX_GAIN:
        return (f"{len(flat)} steps whose a multiply to {gain:.5g}, at most {_abi.ORTHO_MAX_GAIN}: "
                "they scale the rounding up (take fewer)")
    return ("coefficients that can take a singular value past 1.99, or 1 + (b A + c A A) / a or "
            "the product of those past 3.99")


def orthogonalize(g, steps=5, coeffs=MUON_COEFFS, eps=1e-7, out=None, ws=None):
    """Newton-Schulz directions of weight gradients (moonep_orthogonalize): g
    [n,rows,cols] or [rows,cols], float32 (such as grad_home [E,H,Hp]) or
    bfloat16, each matrix on its own, to bfloat16 of the same shape.  coeffs:
    one (a, b, c) for every step, or a sequence of `steps` of them; the a may
    multiply to 2048 (six of the default), for they scale rounding up.  ws: a
    workspace of orthogonalize_workspace(n, rows, cols); without one it is
    allocated per call."""
    if g.dim() not in (2, 3):
        raise ValueError(f"g: expected [n,rows,cols] or [rows,cols], got {tuple(g.shape)}")
    n, rows, cols = (1, *g.shape) if g.dim() == 2 else g.shape
    dt = _float_type(g, "g")
    nested = len(coeffs) == 0 or hasattr(coeffs[0], "__len__")
    flat = [tuple(c) for c in coeffs] if nested else [tuple(coeffs)] * steps
    if len(flat) != steps or any(len(c) != 3 for c in flat):
        raise ValueError("coeffs: expected (a, b, c) or one (a, b, c) per step")
    dev = g.device
    args = (_dev_ptr(g, g.dtype, g.shape, "g"), dt, n, rows, cols,
            (ctypes.c_float * (3 * steps))(*[v for c in flat for v in c]), steps, eps)
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=dev)
    else:
        _dev_ptr(out, torch.bfloat16, g.shape, "out")
        _same_device(dev, out=out)
        _apart("out", out, g=g, ws=ws)
    if ws is None:
        ws = orthogonalize_workspace(n, rows, cols, device=dev)
    else:
        _dev_ptr(ws, torch.uint8, ws.shape, "ws")
        _same_device(dev, ws=ws)
        _apart("ws", ws, g=g)
    try:
        _launch(dev, "moonep_orthogonalize", *args, out.data_ptr(), ws.data_ptr(), ws.numel())
    except MoonepError as e:
        why = _refused_steps(flat, eps) if e.status == _abi.MOONEP_ERR_ARG else None
        if why is None:
            raise
        raise MoonepError(e.status, f"moonep_orthogonalize: {why}") from None
    return out


def _rows(t, dtype, shape, dev, name):
    """Pointer of an input of this type and shape on the device `dev`, checked at the least cost."""
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    p = _dev_ptr(t, dtype, shape, name)
    _same_device(dev, **{name: t})
    return p


def _maybe(t, dtype, shape, dev, name):
    return None if t is None else _rows(t, dtype, shape, dev, name)


def _int32(n):
    """A size for a 32-bit argument; one that does not fit is refused as the library refuses -1."""
    return n if n < 1 << 31 else -1


def _workspace(name, nbytes, device):
    if nbytes < 0:
        raise MoonepError(_abi.MOONEP_ERR_CONFIG, name)
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _disjoint(outs, ins, instead=()):
    """Names what overlaps after the library has refused it: every tensor of `outs` has to lie apart
    from the inputs and the other outputs; `instead`: pairs (output, input) that may start alike."""
    done = {}
    for name, t in outs.items():
        if t is not None:
            free = {n for o, n in instead if o == name and ins[n] is not None and
                    ins[n].data_ptr() == t.data_ptr()}
            _apart(name, t, **{n: i for n, i in ins.items() if n not in free}, **done)
            done[name] = t


def _ffn_inputs(x, weights, act):
    """What shared_ffn and its backward check alike: (T, H, Hp, activation, weights' pointers)."""
    if act not in _abi.ACTS:
        raise ValueError(f"act: expected one of {sorted(_abi.ACTS)}, got {act!r}")
    if len(weights) != 3 or weights[0].dim() != 2:
        raise ValueError("three projections (gate, up, down) [H,Hp] expected")
    shape = weights[0].shape
    H, Hp = shape
    if x.dim() == 0:
        raise ValueError("x: expected [...,H], got a scalar")
    _dev_ptr(x, torch.bfloat16, (*x.shape[:-1], H), "x")
    dev = x.device
    w = _abi.PTR3(_rows(weights[0], torch.bfloat16, shape, dev, "gate"),
                  _rows(weights[1], torch.bfloat16, shape, dev, "up"),
                  _rows(weights[2], torch.bfloat16, shape, dev, "down"))
    return x.numel() // H if H else 0, _int32(H), _int32(Hp), _abi.ACTS[act], w


def shared_ffn_workspace(T, H, Hp, device="cuda"):
    """Workspace tensor of `shared_ffn` for T tokens."""
    return _workspace("moonep_shared_ffn_ws",
                      lib().moonep_shared_ffn_ws(T, _int32(H), _int32(Hp)), device)


def shared_ffn_bwd_workspace(T, H, Hp, device="cuda"):
    """Workspace tensor of `shared_ffn_bwd` for T tokens."""
    return _workspace("moonep_shared_ffn_bwd_ws",
                      lib().moonep_shared_ffn_bwd_ws(T, _int32(H), _int32(Hp)), device)


def shared_ffn(x, weights, act="silu", add=None, out=None, ws=None):
    """The shared expert (moonep_shared_ffn): (f(x Wg) * (x Wu)) Wd^T (+ add) for
    x [...,H] bfloat16 and weights = (gate, up, down), each [H,Hp] bfloat16 as the
    experts' are.  act: "silu" or "gelu_tanh"; add [...,H] bfloat16, such as
    combine's output, is added before the only rounding.  out may be add.  ws: a
    workspace of shared_ffn_workspace(T, H, Hp); without one it is allocated per
    call."""
    T, H, Hp, kind, w = _ffn_inputs(x, weights, act)
    dev = x.device
    p_add = _maybe(add, torch.bfloat16, x.shape, dev, "add")
    if ws is None:
        ws = shared_ffn_workspace(T, H, Hp, device=dev)
        p_ws = ws.data_ptr()
    else:
        p_ws = _rows(ws, torch.uint8, ws.shape, dev, "ws")
    if out is None:
        out = torch.empty_like(x)
        p = out.data_ptr()
    else:
        p = _rows(out, torch.bfloat16, x.shape, dev, "out")
    try:
        _launch(dev, "moonep_shared_ffn", x.data_ptr(), w, kind, p_add, T, H, Hp, p, p_ws,
                ws.numel())
    except MoonepError:
        _disjoint(dict(out=out, ws=ws), dict(x=x, gate=weights[0], up=weights[1], down=weights[2],
                                             add=add), [("out", "add")])
        raise
    return out


def shared_ffn_bwd(x, dy, weights, act="silu", need_dx=True, need_dw=True, dx=None, dw=None,
                   ws=None):
    """Gradients of shared_ffn (moonep_shared_ffn_bwd): (dx, (dgate, dup, ddown))
    from dy [...,H] bfloat16 (which is add's gradient too).  dw: three tensors
    [H,Hp], all bfloat16 (written) or all float32 (added to, like expert_wgrad's
    grad_home); without it they are bfloat16 and new.  need_dx / need_dw = False
    leave one out (None).  ws: a workspace of shared_ffn_bwd_workspace(T, H, Hp);
    without one it is allocated per call."""
    T, H, Hp, kind, w = _ffn_inputs(x, weights, act)
    dev = x.device
    p_dy = _rows(dy, torch.bfloat16, x.shape, dev, "dy")
    if (dx is not None and not need_dx) or (dw is not None and not need_dw):
        raise ValueError("dx or dw given, but need_dx or need_dw is False")
    if ws is None:
        ws = shared_ffn_bwd_workspace(T, H, Hp, device=dev)
        p_ws = ws.data_ptr()
    else:
        p_ws = _rows(ws, torch.uint8, ws.shape, dev, "ws")
    p_dx = None
    if dx is not None:
        p_dx = _rows(dx, torch.bfloat16, x.shape, dev, "dx")
    elif need_dx:
        dx = torch.empty_like(x)
        p_dx = dx.data_ptr()
    code, p_dw = _abi.BF16, None
    if dw is not None:
        if len(dw) != 3:
            raise ValueError("three gradients (gate, up, down) expected")
        code = _float_type(dw[0], "dw[0]")
        for i, t in enumerate(dw):
            _rows(t, dw[0].dtype, (H, Hp), dev, f"dw[{i}]")
        p_dw = _abi.ptr3(dw)
    elif need_dw:
        dw = tuple([torch.empty_like(t) for t in weights])
        p_dw = _abi.PTR3(dw[0].data_ptr(), dw[1].data_ptr(), dw[2].data_ptr())
    try:
        _launch(dev, "moonep_shared_ffn_bwd", x.data_ptr(), p_dy, w, kind, T, H, Hp, p_dx, p_dw,
                code, p_ws, ws.numel())
    except MoonepError:
        _disjoint({"dx": dx, "ws": ws, **{f"dw[{i}]": t for i, t in enumerate(dw or ())}},
                  dict(x=x, dy=dy, gate=weights[0], up=weights[1], down=weights[2]))
        raise
    return dx, dw


def _norm_inputs(h, y, y2, gate, w_post, w_pre):
    """What block_norm and its backward check alike: the C call's arguments (h, dtype), (y, y2,
    gate, kind, w_post, w_pre) and (T, W)."""
    shape, dev = h.shape, h.device
    if len(shape) == 0:
        raise ValueError("h: expected [...,W], got a scalar")
    W = shape[-1]
    p_h, dt = _dev_ptr(h, h.dtype, shape, "h"), _float_type(h, "h")
    p_gate, kind = None, _abi.GATE_NONE
    if gate is not None:
        if gate.dtype is torch.bfloat16:
            p_gate, kind = _rows(gate, torch.bfloat16, shape, dev, "gate"), _abi.GATE_FULL
        elif gate.shape == (W,):
            p_gate, kind = _rows(gate, torch.float32, (W,), dev, "gate"), _abi.GATE_CHANNEL
        else:
            token = (*shape[:-1], 1)
            if gate.dtype is torch.float32 and gate.shape != token:
                raise ValueError(f"gate: expected shape {(W,)} or {token} in float32 or "
                                 f"{tuple(shape)} in bfloat16, got {tuple(gate.shape)}")
            p_gate, kind = _rows(gate, torch.float32, token, dev, "gate"), _abi.GATE_TOKEN
    if y is None:
        for name, t in (("y2", y2), ("gate", gate), ("w_post", w_post)):
            if t is not None:
                raise ValueError(f"{name} given, but y is None")
        if w_pre is None:
            raise ValueError("one of y and w_pre is needed")
    return ((p_h, dt),
            (_maybe(y, torch.bfloat16, shape, dev, "y"),
             _maybe(y2, torch.bfloat16, shape, dev, "y2"), p_gate, kind,
             _maybe(w_post, torch.float32, (W,), dev, "w_post"),
             _maybe(w_pre, torch.float32, (W,), dev, "w_pre")),
            (math.prod(shape[:-1]), _int32(W)))


def block_norm(h, y=None, y2=None, gate=None, w_post=None, w_pre=None, scale=1.0, eps=1e-6,
               h_out=None, u=None):
    """A block's end and the next one's start in one pass (moonep_block_norm):

        h_out = h + scale * gate * norm(y + y2) * w_post
        u     = norm(h_out) * w_pre,   norm(v) = v / sqrt(mean(v^2) + eps)

    h [...,W] float32 or bfloat16 (the residual stream); y, y2 [...,W] bfloat16
    (the block's outputs: combine's, shared_ffn's); w_post, w_pre [W] float32,
    either may be None (no norm there); gate None, [W] or [...,1] float32, or
    [...,W] bfloat16.  Returns (h_out in the stream's type, u in bfloat16 or
    None).  Without y the stream is only normalised and h_out is h.  h_out may
    be h (in place), u may be y or y2."""
    a0, a1, a2 = _norm_inputs(h, y, y2, gate, w_post, w_pre)
    shape, dev = h.shape, h.device
    p_h = p_u = None
    if y is None:
        if h_out is not None and h_out is not h:
            raise ValueError("h_out given, but y is None: the stream stays as it is")
        h_out = h
    elif h_out is None:
        h_out = torch.empty_like(h)
        p_h = h_out.data_ptr()
    else:
        p_h = _rows(h_out, h.dtype, shape, dev, "h_out")
    if w_pre is None:
        if u is not None:
            raise ValueError("u given, but w_pre is None")
    elif u is None:
        u = torch.empty_like(h, dtype=torch.bfloat16) if y is None else torch.empty_like(y)
        p_u = u.data_ptr()
    else:
        p_u = _rows(u, torch.bfloat16, shape, dev, "u")
    try:
        _launch(dev, "moonep_block_norm", *a0, *a1, scale, eps, *a2, p_h, p_u)
    except MoonepError:
        _disjoint(dict(h_out=None if y is None else h_out, u=u),
                  dict(h=h, y=y, y2=y2, gate=gate, w_post=w_post, w_pre=w_pre),
                  [("h_out", "h"), ("u", "y"), ("u", "y2")])
        raise
    return h_out, u


def block_norm_bwd_workspace(T, W, device="cuda"):
    """Workspace tensor of `block_norm_bwd` for T rows of W elements."""
    return _workspace("moonep_block_norm_bwd_ws", lib().moonep_block_norm_bwd_ws(T, _int32(W)),
                      device)


def block_norm_bwd(h, dh, du=None, y=None, y2=None, gate=None, w_post=None, w_pre=None, scale=1.0,
                   eps=1e-6, need_dw=True, dres=None, dy=None, ws=None):
    """Gradients of block_norm (moonep_block_norm_bwd): h is the stream behind
    the block (block_norm's h_out), dh its gradient from later blocks in the
    stream's type (or None), du that of u in bfloat16 (with w_pre); the other
    arguments as in the forward.  Returns (dres, dy, dgate, dw_post, dw_pre):
    dres for the stream before the block (its type), dy for y and for y2 alike
    (bfloat16), dgate in the gate's shape and type, the weights' in float32; None
    where there is no such input.  need_dw=False leaves dgate, dw_post and dw_pre
    out.  dres may be dh, dy may be y, y2 or du.  ws: a workspace of
    block_norm_bwd_workspace(T, W); without one it is allocated per call."""
    a0, a1, a2 = _norm_inputs(h, y, y2, gate, w_post, w_pre)
    shape, dev = h.shape, h.device
    if dh is None and du is None:
        raise ValueError("one of dh and du is needed")
    if (du is None) != (w_pre is None):
        raise ValueError("du and w_pre go together")
    p_dh = _maybe(dh, h.dtype, shape, dev, "dh")
    p_du = _maybe(du, torch.bfloat16, shape, dev, "du")
    if dres is None:
        dres = torch.empty_like(h)
        p_dres = dres.data_ptr()
    else:
        p_dres = _rows(dres, h.dtype, shape, dev, "dres")
    p_dy = None
    if y is None:
        if dy is not None:
            raise ValueError("dy given, but y is None")
    elif dy is None:
        dy = torch.empty_like(y)
        p_dy = dy.data_ptr()
    else:
        p_dy = _rows(dy, torch.bfloat16, shape, dev, "dy")
    dgate = dw_post = dw_pre = p_dgate = p_dpost = p_dpre = None
    if need_dw:
        if gate is not None:
            dgate = torch.empty_like(gate)
            p_dgate = dgate.data_ptr()
        if w_post is not None:
            dw_post = torch.empty_like(w_post)
            p_dpost = dw_post.data_ptr()
        if w_pre is not None:
            dw_pre = torch.empty_like(w_pre)
            p_dpre = dw_pre.data_ptr()
    p_ws = None
    if ws is not None:
        p_ws = _rows(ws, torch.uint8, ws.shape, dev, "ws")
    elif p_dpost or p_dpre or (p_dgate and a1[3] == _abi.GATE_CHANNEL):
        ws = block_norm_bwd_workspace(*a2, device=dev)
        p_ws = ws.data_ptr()
    try:
        _launch(dev, "moonep_block_norm_bwd", *a0, p_dh, p_du, *a1, scale, eps, *a2, p_dres, p_dy,
                p_dgate, p_dpost, p_dpre, p_ws, 0 if ws is None else ws.numel())
    except MoonepError:
        _disjoint(dict(ws=ws, dres=dres, dy=dy),
                  dict(h=h, dh=dh, du=du, y=y, y2=y2, gate=gate, w_post=w_post, w_pre=w_pre),
                  [("dres", "dh"), ("dy", "du"), ("dy", "y"), ("dy", "y2")])
        raise
    return dres, dy, dgate, dw_post, dw_pre


class SymmetricBuffer:
    """One projection's [E+B,H,H'] buffer for the R ranks of `buf`, built on
    virtual memory by the library (moonep_symbuf_create): bf16 weights (README
    "Weight buffer") or fp32 gradients ("Gradient buffer").

    views [R,E+B,H,Hp]: rank d's contiguous [E+B] range; rows [0,E) map the R
                        home chunks, rows [E,E+B) rank d's own slot chunk
    home  [E,H,Hp]:     the home chunks (home[p] / grad_home of the other calls)
    slots [R,B,H,Hp]:   the slot chunks (pool[p] / the [R,B] reduce view)

    The three tensors alias the same physical memory.  They do not own it:
    drop them before destroy().  `slots_from`: another SymmetricBuffer whose
    slot chunks this one maps (one prefetch pool shared by every layer)."""

    def __init__(self, buf, dtype=torch.bfloat16, slots_from=None):
        elem = {torch.bfloat16: 2, torch.float32: 4}.get(dtype)
        if elem is None:
            raise TypeError("SymmetricBuffer holds bf16 weights or fp32 gradients")
        self._b = ctypes.c_void_p()
        dev = buf.device if buf.device.index is not None else \
            torch.device("cuda", torch.cuda.current_device())
        share = slots_from._b if slots_from is not None else None
        with torch.cuda.device(dev):
            _abi.check(lib().moonep_symbuf_create(buf._h, elem, share, ctypes.byref(self._b)),
                       "moonep_symbuf_create")
        info = _abi.MoonepSymbufInfo()
        _abi.check(lib().moonep_symbuf_info(self._b, ctypes.byref(info)), "moonep_symbuf_info")
        self.row_bytes = int(info.row_bytes)
        self.physical_bytes = int(info.physical_bytes)
        self.granularity = int(info.granularity)
        R, E, B, H, Hp = buf.R, buf.E, buf.B, buf.H, buf.Hp
        self.views = _abi.device_tensor(info.views, (R, E + B, H, Hp), dtype, dev.index)
        self.home = _abi.device_tensor(info.home, (E, H, Hp), dtype, dev.index)
        self.slots = (_abi.device_tensor(info.slots, (R, B, H, Hp), dtype, dev.index) if B
                      else torch.empty((R, 0, H, Hp), dtype=dtype, device=dev))

    def destroy(self):
        if self._b:
            self.views = self.home = self.slots = None
            _abi.check(lib().moonep_symbuf_destroy(self._b), "moonep_symbuf_destroy")
            self._b = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


# fail at import time, loudly, when the native library is missing
lib()
