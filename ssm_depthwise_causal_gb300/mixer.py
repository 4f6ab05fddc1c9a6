"""The rest of an SSM mixer around the packed convolution, over the C ABI of
``include/ccc.h``: the selective scan (``ccc_scan_fwd`` / ``ccc_scan_bwd``),
the one-launch decode step (``ccc_ssm_update``) and the gated RMS norm
(``ccc_gated_norm_fwd`` / ``ccc_gated_norm_bwd``).

As in the package's other entry points, every function marshals torch tensors
into pointers, sizes and strides and calls the library on the current stream;
outputs and workspaces are created when they are not given.  ``stream=s`` (a
stream or its handle) is the call under ``with torch.cuda.stream(s)``: what it
makes belongs to that stream, and what it is given has to be ready there.
"""
from __future__ import annotations

import functools
import struct
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import CCCError, _act_code, _lib, _on_current_device, _pool_args, _stream, _under_stream

__all__ = ["ScanGrads", "SelectiveScanFn", "GatedRMSNormFn", "ccc_scan_workspace_size", "ccc_gated_norm_workspace_size",
           "selective_scan_fn", "selective_scan_bwd", "selective_scan", "ssm_update", "gated_rms_norm_fn",
           "gated_rms_norm_bwd", "gated_rms_norm", "ccc_wait_status", "given_up_waits", "set_wait_limit"]


class ScanGrads(NamedTuple):
    """Gradients of selective_scan_bwd: dx, ddt, dB, dC in the inputs' types and
    shapes; dA, dD, ddt_bias [H] and d_initial [N, H, P, N_state] in FP32 (None
    for what was not there or not asked for)."""
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    d_initial: Optional[torch.Tensor]


@functools.lru_cache(maxsize=256)  # (a function of the sizes alone)
def ccc_scan_workspace_size(rows, n_seqs, heads, head_size, groups, state_size, for_bwd) -> int:
    return int(_lib.lib().ccc_scan_workspace_size(rows, n_seqs, heads, head_size, groups, state_size, int(bool(for_bwd))))


@functools.lru_cache(maxsize=256)
def ccc_gated_norm_workspace_size(rows, width, group_size) -> int:
    return int(_lib.lib().ccc_gated_norm_workspace_size(rows, width, group_size))


# The arguments of a call as one array of 64-bit integers (the _v entry points
# of include/ccc.h): packing them costs a fraction of converting each one.
_PACK = {n: struct.Struct(f"{n}q").pack for n in (14, 21, 33, 38, 42)}

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_CODE = {torch.float32: 0, torch.bfloat16: 1}


def _code(t, name="weight/bias") -> int:
    c = _CODE.get(t.dtype)
    if c is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return c


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


def _rows3s(t, name):
    """Row stride and sizes of BF16 [rows, heads or groups, size] with contiguous heads."""
    if t.dim() != 3 or t.dtype is not _BF16:
        raise ValueError(f"{name} must be BF16 [rows, heads or groups, size]")
    s, (n, a, b) = t.stride(), t.shape
    if (s[2] != 1 and b > 1) or (a > 1 and s[1] != b):
        raise ValueError(f"{name} must be [rows, heads or groups, size] with contiguous heads")
    return s[0] if n > 1 else max(s[0], a * b), (n, a, b)


def _rows3(t, name, sizes, what) -> int:
    """The row stride alone, of a tensor that has to have these sizes."""
    stride, have = _rows3s(t, name)
    if have != sizes:
        raise ValueError(what)
    return stride


def _rows2s(t, name):
    """Row stride and sizes of BF16 [rows, width] with contiguous columns."""
    if t.dim() != 2 or t.dtype is not _BF16:
        raise ValueError(f"{name} must be BF16 [rows, width]")
    s, (n, w) = t.stride(), t.shape
    if s[1] != 1 and w > 1:
        raise ValueError(f"{name} must be [rows, width] with contiguous columns")
    return s[0] if n > 1 else max(s[0], w), (n, w)


def _rows2(t, name, sizes, what) -> int:
    """The row stride alone, of a tensor that has to have these sizes."""
    stride, have = _rows2s(t, name)
    if have != sizes:
        raise ValueError(what)
    return stride


def _steps(dt, rows, H) -> int:
    """Row stride of dt [rows, H]."""
    if dt.shape != (rows, H):
        raise ValueError("dt must be [rows, H]")
    s = dt.stride()
    if s[1] != 1 and H > 1:
        raise ValueError("dt must be [rows, H] with contiguous heads")
    return s[0] if rows > 1 else max(s[0], H)


def _parameters(A, D, dt_bias, H) -> int:
    """The FP32-or-BF16 code that A, D and dt_bias [H] share."""
    kind = A.dtype
    for t in (A, D, dt_bias):
        if t is not None and (t.dtype is not kind or t.dim() != 1 or t.numel() != H or not t.is_contiguous()):
            raise ValueError("A, D and dt_bias must be contiguous [H] tensors of one type")
    return _code(A, "A, D and dt_bias")


# The library gets bare pointers: a tensor of another type or layout or of fewer elements would be read as something else.
def _ints(t, name, need) -> None:
    if t is not None and (t.dtype is not _I32 or t.numel() < need or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous int32 of {need} elements, got {t.dtype} {tuple(t.shape)}")


def _flags(t, name, need) -> None:
    if t is not None and (t.dtype not in (torch.bool, torch.uint8) or t.numel() < need or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous bool or uint8 of {need} elements, got {t.dtype} {tuple(t.shape)}")


class _Batch:
    """Packed inputs of the scan; [B, T, ...] input becomes B sequences of T tokens."""

    __slots__ = ("batch", "x", "dt", "B", "C", "cu", "rows", "H", "P", "G", "N", "seqs", "args")

    def __init__(self, x, dt, A, B, C, cu_seqlens, D, dt_bias, dt_softplus):
        self.batch = None
        if x.dim() == 4:
            if cu_seqlens is not None:
                raise ValueError("cu_seqlens is for packed [rows, H, P] input, not [B, T, H, P]")
            b, t = x.shape[:2]
            self.batch = (b, t)
            cu_seqlens = torch.arange(b + 1, dtype=torch.int32, device=x.device) * t
            x, dt, B, C = (self.flat(v) for v in (x, dt, B, C))
        if cu_seqlens is None:
            cu_seqlens = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=x.device)
        self.x, self.dt, self.B, self.C, self.cu = x, dt, B, C, cu_seqlens
        (xs, x_sizes), (bs, b_sizes), (cs, c_sizes) = _rows3s(x, "x"), _rows3s(B, "B"), _rows3s(C, "C")
        rows, H, P = self.rows, self.H, self.P = x_sizes
        _, G, N = b_sizes
        self.G, self.N = G, N
        if b_sizes[0] != rows or c_sizes != b_sizes:
            raise ValueError("x [rows, H, P], B and C [rows, G, N] do not match")
        self.seqs = cu_seqlens.numel() - 1
        _ints(cu_seqlens, "cu_seqlens", 1)
        self.args = (x.data_ptr(), rows, H, P, xs, dt.data_ptr(), _code(dt, "dt"), _steps(dt, rows, H), 1 if dt_softplus else 0,
                     A.data_ptr(), _at(D), _at(dt_bias), _parameters(A, D, dt_bias, H), B.data_ptr(), bs, C.data_ptr(), cs, G, N)

    def flat(self, t):
        """An input packed; a copy where batch and time do not follow each other in memory."""
        return t if self.batch is None else t.reshape(self.batch[0] * self.batch[1], *t.shape[2:])

    def place(self, t, sizes, name):
        """What is written, packed: the caller's memory, or new (t is None)."""
        if t is None:
            return self.x.new_empty(sizes)
        if self.batch is None:
            return t
        try:
            return t.view(self.batch[0] * self.batch[1], *t.shape[2:])
        except RuntimeError:
            raise ValueError(f"{name} {tuple(t.shape)} with strides {t.stride()} is written in place: batch and time must follow "
                             "each other in memory (a view as [B T, ...])") from None

    def unflat(self, t):
        return t if self.batch is None else t.view(*self.batch, *t.shape[1:])

    def workspace(self, given, for_bwd):
        if given is not None:
            return given
        need = ccc_scan_workspace_size(self.rows, self.seqs, self.H, self.P, self.G, self.N, for_bwd)
        return self.x.new_empty(need, dtype=torch.uint8) if need else None

    def states(self, t, name):
        if t is not None and (t.shape != (self.seqs, self.H, self.P, self.N) or t.dtype != _F32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous FP32 [N, H, P, N_state]")
        return t


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def selective_scan_fn(x, dt, A, B, C, ssm_state=None, cu_seqlens=None, cache_indices=None, has_initial_state=None, *,
                      D=None, dt_bias=None, dt_softplus=False, initial_state=None, final_state=None, out=None,
                      workspace=None, stream=None) -> torch.Tensor:
    """Selective scan forward (include/ccc.h, ccc_scan_fwd): y, shaped as x.

    ``x`` [rows, H, P], ``dt`` [rows, H], ``B`` and ``C`` [rows, G, N] are
    packed by ``cu_seqlens`` (or [B, T, ...]), and may be column slices of one
    buffer; rows past cu_seqlens[-1] of a y made here are not written.
    ``ssm_state`` is the FP32 slot pool [slots, H, P, N], updated in
    place (a pool with draft positions is passed as ``pool[:, 0]``); without
    one, ``initial_state`` / ``final_state`` are [N, H, P, N_state]."""
    if stream is not None:
        return _under_stream(stream, selective_scan_fn, locals())
    b = _Batch(x, dt, A, B, C, cu_seqlens, D, dt_bias, dt_softplus)
    H, P, N = b.H, b.P, b.N
    slots, st_slot = 0, 0
    if ssm_state is not None:
        slots = ssm_state.shape[0]
        if ssm_state.dtype != _F32 or ssm_state.shape[1:] != (H, P, N) or not (slots == 0 or ssm_state[0].is_contiguous()):
            raise ValueError("ssm_state must be FP32 [slots, H, P, N] with contiguous slots")
        st_slot = ssm_state.stride(0) if slots > 1 else H * P * N
    _ints(cache_indices, "cache_indices", b.seqs)
    _flags(has_initial_state, "has_initial_state", b.seqs)
    o = b.place(out, (b.rows, H, P), "out")
    os = H * P if out is None else _rows3(o, "out", (b.rows, H, P), "out must match x")
    b.states(initial_state, "initial_state")
    b.states(final_state, "final_state")
    workspace = b.workspace(workspace, 0)
    _on_current_device(b.x, b.dt, A, b.B, b.C, b.cu, D, dt_bias, ssm_state, cache_indices, has_initial_state, initial_state, final_state,
                       o, workspace)
    rc = _lib.lib().ccc_scan_fwd_v(_PACK[33](
        *b.args, _at(ssm_state), slots, st_slot, _at(initial_state), _at(final_state), b.cu.data_ptr(), b.seqs, _at(cache_indices),
        _at(has_initial_state), o.data_ptr(), os, _at(workspace), _bytes(workspace), _stream(None)))
    if rc != 0:
        raise CCCError(rc, "ccc_scan_fwd")
    return b.unflat(o) if out is None else out


def selective_scan_bwd(x, dt, A, B, C, dy, cu_seqlens=None, *, D=None, dt_bias=None, dt_softplus=False, initial_state=None,
                       cache_indices=None, d_final_state=None, want_d_initial=False, carry_empty=False, dx=None, dB=None,
                       dC=None, workspace=None, stream=None) -> ScanGrads:
    """Selective scan backward (include/ccc.h, ccc_scan_bwd).  ``dx``, ``dB``
    and ``dC`` may be given, also as column slices of one buffer (the dy of
    ccc_bwd); rows past cu_seqlens[-1] of what is made here are not written.
    ``d_initial`` is the gradient through a sequence's tokens; ``carry_empty``
    adds that of an empty sequence, whose final state is its initial one (its
    d_final_state as it is): pass it where fragments are chained, as the
    autograd wrapper does."""
    if stream is not None:
        return _under_stream(stream, selective_scan_bwd, locals())
    b = _Batch(x, dt, A, B, C, cu_seqlens, D, dt_bias, dt_softplus)
    _ints(cache_indices, "cache_indices", b.seqs)
    wide, narrow, new = (b.rows, b.H, b.P), (b.rows, b.G, b.N), b.x.new_empty
    dy2, dx2, dB2, dC2 = b.flat(dy), b.place(dx, wide, "dx"), b.place(dB, narrow, "dB"), b.place(dC, narrow, "dC")
    match = "dy and dx must match x, dB and dC must match B"
    strides = [_rows3(dy2, "dy", wide, match), _rows3(dx2, "dx", wide, match), _rows3(dB2, "dB", narrow, match), _rows3(dC2, "dC", narrow, match)]
    ddt = new((b.rows, b.H), dtype=b.dt.dtype)
    dA = new(b.H, dtype=_F32)
    dD = new(b.H, dtype=_F32) if D is not None else None
    dbias = new(b.H, dtype=_F32) if dt_bias is not None else None
    d_init = new((b.seqs, b.H, b.P, b.N), dtype=_F32) if want_d_initial else None
    b.states(initial_state, "initial_state")
    b.states(d_final_state, "d_final_state")
    workspace = b.workspace(workspace, 1)
    _on_current_device(b.x, b.dt, A, b.B, b.C, b.cu, D, dt_bias, initial_state, cache_indices, dy2, d_final_state, dx2, dB2, dC2, workspace)
    rc = _lib.lib().ccc_scan_bwd_ex_v(_PACK[42](
        *b.args, _at(initial_state), b.cu.data_ptr(), b.seqs, _at(cache_indices), dy2.data_ptr(), strides[0], _at(d_final_state),
        dx2.data_ptr(), strides[1], ddt.data_ptr(), b.H, dB2.data_ptr(), strides[2], dC2.data_ptr(), strides[3], dA.data_ptr(), _at(dD),
        _at(dbias), _at(d_init), _at(workspace), _bytes(workspace), _lib.OPT_CARRY_EMPTY if carry_empty else 0, _stream(None)))
    if rc != 0:
        raise CCCError(rc, "ccc_scan_bwd")
    return ScanGrads(b.unflat(dx2) if dx is None else dx, b.unflat(ddt), dA, b.unflat(dB2) if dB is None else dB,
                     b.unflat(dC2) if dC is None else dC, dD, dbias, d_init)


class SelectiveScanFn(torch.autograd.Function):
    """Autograd wrapper: (y, final_state) of selective_scan_fn; the backward
    recomputes the states, so nothing of the forward is kept but its inputs.
    A second derivative is refused."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, dt_bias, initial_state, cu_seqlens, cache_indices, dt_softplus):
        seqs = x.shape[0] if x.dim() == 4 else 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        final = torch.empty((seqs, *x.shape[-2:], B.shape[-1]), dtype=torch.float32, device=x.device)
        # rows past cu_seqlens[-1] are not written by the kernel: start from 0
        y = selective_scan_fn(x, dt, A, B, C, None, cu_seqlens, cache_indices, D=D, dt_bias=dt_bias, dt_softplus=dt_softplus,
                              initial_state=initial_state, final_state=final, out=torch.zeros(x.shape, dtype=x.dtype, device=x.device))
        ctx.save_for_backward(x, dt, A, B, C, D, dt_bias, initial_state, cu_seqlens, cache_indices)
        ctx.dt_softplus = dt_softplus
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, d_final):
        x, dt, A, B, C, D, dt_bias, initial, cu, cache = ctx.saved_tensors
        made = [torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (x, B, C)]
        g = selective_scan_bwd(x, dt, A, B, C, dy.contiguous(), cu, D=D, dt_bias=dt_bias, dt_softplus=ctx.dt_softplus,
                               initial_state=initial, cache_indices=cache, d_final_state=d_final.contiguous(),
                               want_d_initial=initial is not None, carry_empty=True, dx=made[0], dB=made[1], dC=made[2])
        ddt = g.ddt
        if cu is not None:  # as above, for the rows past the last sequence
            ddt = torch.where(torch.arange(dt.shape[0], device=dt.device)[:, None] < cu[-1], ddt, torch.zeros_like(ddt))

        def like(d, p):
            return None if p is None else d.to(p.dtype)
        return g.dx, ddt, like(g.dA, A), g.dB, g.dC, like(g.dD, D), like(g.ddt_bias, dt_bias), g.d_initial, None, None, None


def selective_scan(x, dt, A, B, C, cu_seqlens=None, *, D=None, dt_bias=None, dt_softplus=False, initial_state=None,
                   cache_indices=None):
    """Differentiable selective scan: ``(y, final_state)`` (see SelectiveScanFn)."""
    return SelectiveScanFn.apply(x, dt, A, B, C, D, dt_bias, initial_state, cu_seqlens, cache_indices, dt_softplus)


def ssm_update(xBC, weight, conv_state, dt, A, ssm_state, cache_indices, *, n_groups, cu_seqlens=None, num_accepted=None,
               bias=None, activation="silu", D=None, dt_bias=None, dt_softplus=False, out=None, stream=None) -> torch.Tensor:
    """One decode step of the mixer (include/ccc.h, ccc_ssm_update): y
    [rows, H, P] (or [B, k, H, P]) of the new tokens ``xBC`` [rows, C] with
    ``cu_seqlens`` ([B, C]: one token a request; [B, k, C]: k of them), with
    both pools updated in place.  ``ssm_state`` is [slots, H, P, N] for one
    token a request, or [slots, positions, H, P, N] to keep the states after a
    request's first ``positions`` tokens (of which num_accepted then names one)."""
    if stream is not None:
        return _under_stream(stream, ssm_update, locals())
    lead = None
    if xBC.dim() == 3:
        lead = xBC.shape[:2]
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens is for packed [rows, C] input, not [B, k, C]")
        cu_seqlens = torch.arange(lead[0] + 1, dtype=torch.int32, device=xBC.device) * lead[1]
        xBC, dt = xBC.reshape(-1, xBC.shape[-1]), dt.reshape(-1, dt.shape[-1])
    elif cu_seqlens is None:
        cu_seqlens = torch.arange(xBC.shape[0] + 1, dtype=torch.int32, device=xBC.device)
    xs, (rows, channels) = _rows2s(xBC, "xBC")
    seqs = cu_seqlens.numel() - 1
    _ints(cu_seqlens, "cu_seqlens", 1)
    _ints(cache_indices, "cache_indices", seqs)
    if num_accepted is not None:
        _ints(num_accepted, "num_accepted", seqs)
    if ssm_state.dtype != _F32 or ssm_state.dim() not in (4, 5):
        raise ValueError("ssm_state must be FP32 [slots, H, P, N] or [slots, positions, H, P, N]")
    G = int(n_groups)
    s = ssm_state.stride()
    if ssm_state.dim() == 4:
        if rows > seqs:
            raise ValueError(f"{rows} tokens of {seqs} requests: ssm_state [slots, H, P, N] has room for the state after one token; pass "
                             "[slots, positions, H, P, N]")
        slots, H, P, N = ssm_state.shape
        held, hpn = 1, H * P * N
        st_pos = hpn
    else:
        slots, held, H, P, N = ssm_state.shape
        hpn = H * P * N
        st_pos = s[1] if held > 1 else hpn
    if s[-3:] != (P * N, N, 1) and slots and held and not ssm_state[(0,) * (ssm_state.dim() - 3)].is_contiguous():
        raise ValueError("ssm_state must hold each [H, P, N] contiguously")
    st_slot = s[0] if slots > 1 else held * st_pos
    if channels != H * P + 2 * G * N or weight.dim() != 2 or weight.shape[0] != channels:
        raise ValueError("xBC [rows, H P + 2 G N] and weight [C, W] do not match ssm_state and n_groups")
    if not weight.is_contiguous() or (bias is not None and (bias.numel() != channels or not bias.is_contiguous())):
        raise ValueError("weight [C, W] and bias [C] must be contiguous")
    c_slots, L, st = _pool_args(conv_state, channels)
    if c_slots != slots:
        raise ValueError("conv_state and ssm_state must have the same slots")
    if out is None:
        y, os = xBC.new_empty((rows, H, P)), H * P
    else:
        y = out.view(rows, H, P) if lead else out
        os = _rows3(y, "out", (rows, H, P), "out must be [rows, H, P]")
    _on_current_device(xBC, weight, bias, conv_state, dt, A, D, dt_bias, ssm_state, cu_seqlens, cache_indices, num_accepted, y)
    rc = _lib.lib().ccc_ssm_update_v(_PACK[38](
        xBC.data_ptr(), rows, H, P, G, N, xs, weight.data_ptr(), _code(weight), weight.shape[1], _at(bias), -1 if bias is None else _code(bias),
        _act_code(activation), _at(conv_state), slots, L, st[0], st[1], st[2], dt.data_ptr(), _code(dt, "dt"), _steps(dt, rows, H),
        1 if dt_softplus else 0, A.data_ptr(), _at(D), _at(dt_bias), _parameters(A, D, dt_bias, H), ssm_state.data_ptr(), held, st_slot, st_pos,
        cu_seqlens.data_ptr(), seqs, _at(cache_indices), _at(num_accepted), y.data_ptr(), os, _stream(None)))
    if rc != 0:
        raise CCCError(rc, "ccc_ssm_update")
    if out is not None:
        return out
    return y.view(*lead, H, P) if lead else y


@functools.lru_cache(maxsize=64)
def _float_bits(v):
    return struct.unpack("i", struct.pack("f", v))[0]


def _flat2(t):
    return t if t.dim() == 2 else t.reshape(-1, t.shape[-1])


def _norm_args(y, z, weight, group_size, eps, norm_before_gate):
    """The arguments that both directions begin with, and y's sizes."""
    what = "y and z [rows, width] and weight [width] do not match"
    ys, sizes = _rows2s(y, "y")
    zs = _rows2(z, "z", sizes, what)
    rows, width = sizes
    if weight.dim() != 1 or weight.numel() != width or not weight.is_contiguous():
        raise ValueError(what)
    return (y.data_ptr(), rows, width, ys, z.data_ptr(), zs, weight.data_ptr(), _code(weight), int(group_size or width), _float_bits(eps),
            1 if norm_before_gate else 0), sizes


def gated_rms_norm_fn(y, z, weight, *, eps=1e-5, group_size=None, norm_before_gate=False, out=None, stream=None) -> torch.Tensor:
    """Gated RMS norm (include/ccc.h, ccc_gated_norm_fwd) of y by the gate z,
    both BF16 [..., width]; ``group_size`` defaults to the whole width."""
    if stream is not None:
        return _under_stream(stream, gated_rms_norm_fn, locals())
    y2, z2 = _flat2(y), _flat2(z)
    args, sizes = _norm_args(y2, z2, weight, group_size, eps, norm_before_gate)
    if out is None:
        o, os = y2.new_empty(sizes), sizes[1]
    else:
        o = out if out.dim() == 2 else out.view(sizes)
        os = _rows2(o, "out", sizes, "out must match y")
    _on_current_device(y2, z2, weight, o)
    rc = _lib.lib().ccc_gated_norm_fwd_v(_PACK[14](*args, o.data_ptr(), os, _stream(None)))
    if rc != 0:
        raise CCCError(rc, "ccc_gated_norm_fwd")
    return out if out is not None else o if y2 is y else o.view(y.shape)


def gated_rms_norm_bwd(y, z, weight, dout, *, eps=1e-5, group_size=None, norm_before_gate=False, dy=None, dz=None,
                       workspace=None, stream=None):
    """(dy, dz, dweight) of gated_rms_norm_fn; dweight is FP32 [width]."""
    if stream is not None:
        return _under_stream(stream, gated_rms_norm_bwd, locals())
    y2, z2, g2 = _flat2(y), _flat2(z), _flat2(dout)
    args, sizes = _norm_args(y2, z2, weight, group_size, eps, norm_before_gate)
    gs = _rows2(g2, "dout", sizes, "dout must match y")
    a = y2.new_empty(sizes) if dy is None else dy.view(sizes)
    b = y2.new_empty(sizes) if dz is None else dz.view(sizes)
    strides = _rows2(a, "dy", sizes, "dy must match y"), _rows2(b, "dz", sizes, "dz must match y")
    dw = y2.new_empty(sizes[1], dtype=_F32)
    need = ccc_gated_norm_workspace_size(*sizes, args[8])
    if workspace is None and need:
        workspace = y2.new_empty(need, dtype=torch.uint8)
    _on_current_device(y2, z2, weight, g2, a, b, workspace)
    rc = _lib.lib().ccc_gated_norm_bwd_v(_PACK[21](*args, g2.data_ptr(), gs, a.data_ptr(), strides[0], b.data_ptr(), strides[1], dw.data_ptr(),
                                                   _at(workspace), _bytes(workspace), _stream(None)))
    if rc != 0:
        raise CCCError(rc, "ccc_gated_norm_bwd")
    return (a.view(y.shape) if dy is None else dy), (b.view(y.shape) if dz is None else dz), dw


class GatedRMSNormFn(torch.autograd.Function):
    """Autograd wrapper: recomputes from y and z, keeps nothing else.  A second
    derivative is refused."""

    @staticmethod
    def forward(ctx, y, z, weight, eps, group_size, norm_before_gate):
        ctx.save_for_backward(y, z, weight)
        ctx.kind = dict(eps=eps, group_size=group_size, norm_before_gate=norm_before_gate)
        return gated_rms_norm_fn(y, z, weight, **ctx.kind)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, z, weight = ctx.saved_tensors
        dy, dz, dw = gated_rms_norm_bwd(y, z, weight, dout.contiguous(), **ctx.kind)
        return dy, dz, dw.to(weight.dtype), None, None, None


def gated_rms_norm(y, z, weight, *, eps=1e-5, group_size=None, norm_before_gate=False) -> torch.Tensor:
    """Differentiable gated RMS norm (see GatedRMSNormFn)."""
    return GatedRMSNormFn.apply(y, z, weight, eps, group_size, norm_before_gate)


def ccc_wait_status(status=None, stream=None) -> torch.Tensor:
    """How many CTAs have given up a bounded wait on the current device (include/ccc.h, ccc_wait_status): an int32 tensor whose
    first element receives the count once the stream gets there (no synchronization here).  Anything but 0: results of the
    scans and decode steps since it was 0 are undefined."""
    if status is None:
        make = functools.partial(torch.empty, 1, dtype=torch.int32, device="cuda")
        status = make() if stream is None else _under_stream(stream, make, {})
    if status.dtype is not torch.int32 or status.numel() < 1 or not status.is_contiguous():
        raise ValueError("status must be a contiguous int32 tensor")
    _on_current_device(status)
    rc = _lib.lib().ccc_wait_status(status.data_ptr(), _stream(stream))
    if rc != 0:
        raise CCCError(rc, "ccc_wait_status")
    return status


def given_up_waits() -> int:
    """ccc_wait_status, then a host read (synchronizes the current stream): 0 unless a scan or decode step on this device gave
    a wait up."""
    return int(ccc_wait_status()[0].item()) & 0xffffffff


def set_wait_limit(clocks=None) -> None:
    """How many SM clocks a wait inside a scan or decode step lasts at most, from the next launch on (ccc_set_wait_limit);
    None: the default, about half a second."""
    rc = _lib.lib().ccc_set_wait_limit(_lib.WAIT_LIMIT_DEFAULT if clocks is None else int(clocks))
    if rc != 0:
        raise CCCError(rc, "ccc_set_wait_limit")
