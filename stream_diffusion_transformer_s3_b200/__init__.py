"""B200-native hot path of the Z-Image-Turbo single-stream DiT (S3-DiT).

The compute lives in ``libzdit.so`` (hand-written sm_100a CUDA, C ABI declared in
``include/zdit.h``).  This module is the thin ctypes binding: it marshals torch
tensors (device memory, streams) into the C structs and calls the library under the
same names.  There is no fallback: if the library is missing or the device is not a
B200, calls raise.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from dataclasses import dataclass, field

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libzdit.so")
_lib = None

STATUS = {0: "ZDIT_OK", -1: "ZDIT_ERR_INVALID_ARG", -2: "ZDIT_ERR_SHAPE", -3: "ZDIT_ERR_ALIGNMENT",
          -4: "ZDIT_ERR_WORKSPACE", -5: "ZDIT_ERR_UNSUPPORTED", -6: "ZDIT_ERR_CUDA",
          -7: "ZDIT_ERR_DEVICE_TIMEOUT"}

F_ADALN, F_SANDWICH_NORM, F_QK_NORM, F_TANH_GATE = 1, 2, 4, 8
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_NTK, ROPE_SCALE_YARN = 0, 1, 2, 3
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU_TANH, ACT_GELU = 0, 1, 2, 3


class ZditError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where} failed: {STATUS.get(code, code)}")
        self.code = code


# ----------------------------------------------------------------------- C structs
class BlockCfg(C.Structure):
    _fields_ = [("dim", C.c_int32), ("n_heads", C.c_int32), ("head_dim", C.c_int32),
                ("ffn_hidden", C.c_int32), ("temb_dim", C.c_int32), ("rope_axes", C.c_int32 * 3),
                ("norm_eps", C.c_float), ("rope_theta", C.c_float), ("flags", C.c_uint32)]


class BlockWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "w_ada", "b_ada", "w_qkv", "w_out", "w_gate_up", "w_down", "n_attn", "n_attn_post",
        "n_ffn", "n_ffn_post", "n_q", "n_k")]


class Varlen(C.Structure):
    _fields_ = [("batch", C.c_int32), ("cu_seqlens_dev", C.c_void_p),
                ("cu_seqlens_host", C.POINTER(C.c_int32))]


class StackCfg(C.Structure):
    _fields_ = [("block", BlockCfg), ("n_noise_refiner", C.c_int32), ("n_context_refiner", C.c_int32),
                ("n_main", C.c_int32), ("patch_dim", C.c_int32), ("cap_dim", C.c_int32),
                ("t_scale", C.c_float), ("final_eps", C.c_float)]


class StackWeights(C.Structure):
    _fields_ = [("blocks", C.POINTER(BlockWeights))] + [(n, C.c_void_p) for n in (
        "w_x", "b_x", "w_capnorm", "w_cap", "b_cap", "pad_vec", "w_t1", "b_t1", "w_t2", "b_t2",
        "w_fada", "b_fada", "w_final", "b_final")]


class StackInputs(C.Structure):
    _fields_ = [("batch", C.c_int32), ("grid_h", C.c_int32), ("grid_w", C.c_int32),
                ("n_cap", C.POINTER(C.c_int32)), ("n_valid", C.POINTER(C.c_int32)),
                ("patches", C.c_void_p), ("cap_feats", C.c_void_p), ("t", C.POINTER(C.c_float)),
                ("shared_patches", C.c_int32)]


class SampleCfg(C.Structure):
    _fields_ = [("n_steps", C.c_int32), ("guidance", C.c_float), ("cache_context", C.c_int32),
                ("dedup_noise", C.c_int32), ("use_graph", C.c_int32)]


class ProfileEntry(C.Structure):
    _fields_ = [("name", C.c_char * 40), ("launches", C.c_int32), ("total_ms", C.c_double),
                ("flops", C.c_double), ("bytes", C.c_double)]


class RopeScaling(C.Structure):
    """Frequency scaling of zdit_rope_table_scaled: RopeScaling(kind, factor, original_len,
    beta_fast, beta_slow, magnitude); the trailing values default to those of no scaling."""
    _fields_ = [("kind", C.c_int32), ("factor", C.c_float), ("original_len", C.c_float),
                ("beta_fast", C.c_float), ("beta_slow", C.c_float), ("magnitude", C.c_float)]

    def __init__(self, kind=ROPE_SCALE_NONE, factor=1.0, original_len=1.0, beta_fast=32.0, beta_slow=1.0,
                 magnitude=1.0):
        super().__init__(kind, factor, original_len, beta_fast, beta_slow, magnitude)


class Heads(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("row_stride", C.c_int64), ("head_stride", C.c_int64)]


class QkNormRopeArgs(C.Structure):
    _fields_ = [("T", C.c_int64), ("n_q", C.c_int32), ("n_k", C.c_int32), ("head_dim", C.c_int32),
                ("in_dtype", C.c_int32), ("out_dtype", C.c_int32), ("q", Heads), ("k", Heads),
                ("q_out", Heads), ("k_out", Heads), ("w_q", C.c_void_p), ("w_k", C.c_void_p),
                ("eps", C.c_float), ("cos", C.c_void_p), ("sin", C.c_void_p), ("rotary_dim", C.c_int32),
                ("layout", C.c_int32)]


class PromptAttentionArgs(C.Structure):
    _fields_ = [("batch", C.c_int32), ("q_len", C.POINTER(C.c_int32)), ("kv_len", C.POINTER(C.c_int32)),
                ("kv_start", C.POINTER(C.c_int32)), ("n_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("causal", C.c_int32), ("scale", C.c_float), ("q", Heads),
                ("k", Heads), ("v", Heads), ("o", Heads)]


class LinearArgs(C.Structure):
    _fields_ = [("M", C.c_int64), ("N", C.c_int64), ("K", C.c_int64), ("a", C.c_void_p), ("lda", C.c_int64),
                ("w", C.c_void_p), ("ldw", C.c_int64), ("bias", C.c_void_p), ("act", C.c_int32),
                ("residual", C.c_void_p), ("ld_residual", C.c_int64), ("residual_dtype", C.c_int32),
                ("out", C.c_void_p), ("ld_out", C.c_int64), ("out_dtype", C.c_int32)]


_SIGS = {
    "zdit_profile_begin": (C.c_int, [C.c_int32]),
    "zdit_profile_end": (C.c_int, [C.POINTER(ProfileEntry), C.c_int32, C.POINTER(C.c_int32)]),
    "zdit_launch_count": (C.c_int64, []),
    "zdit_version": (C.c_int32, []),
    "zdit_status_string": (C.c_char_p, [C.c_int]),
    "zdit_block_workspace_bytes": (C.c_size_t, [C.POINTER(BlockCfg), C.c_int64, C.c_int32]),
    "zdit_block_forward": (C.c_int, [C.POINTER(BlockCfg), C.POINTER(BlockWeights), C.POINTER(Varlen),
                                     C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                     C.c_size_t, C.c_void_p]),
    "zdit_block_forward_static": (C.c_int, [C.POINTER(BlockCfg), C.POINTER(BlockWeights), C.POINTER(Varlen),
                                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "zdit_stack_workspace_bytes": (C.c_size_t, [C.POINTER(StackCfg), C.POINTER(StackInputs)]),
    "zdit_stack_forward": (C.c_int, [C.POINTER(StackCfg), C.POINTER(StackWeights), C.POINTER(StackInputs),
                                     C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "zdit_sample_workspace_bytes": (C.c_size_t, [C.POINTER(StackCfg), C.POINTER(StackInputs)]),
    "zdit_sample": (C.c_int, [C.POINTER(StackCfg), C.POINTER(StackWeights), C.POINTER(StackInputs),
                              C.POINTER(SampleCfg), C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "zdit_euler_cfg_step": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_float,
                                      C.c_float, C.c_float, C.c_void_p]),
    "zdit_sigma_schedule": (C.c_int, [C.c_int32, C.POINTER(C.c_float)]),
    "zdit_rope_table": (C.c_int, [C.c_void_p, C.c_int64, C.c_int32, C.POINTER(C.c_int32), C.c_float,
                                  C.c_void_p, C.c_void_p, C.c_void_p]),
    "zdit_joint_attention": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_void_p,
                                       C.c_int32, C.c_void_p, C.c_int32, C.POINTER(Varlen), C.c_int32,
                                       C.c_int32, C.c_void_p]),
    "zdit_adaln_project": (C.c_int, [C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.POINTER(C.c_void_p),
                                     C.c_int32, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p]),
    "zdit_gemm_bf16": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_int64,
                                 C.c_int64, C.c_void_p, C.c_void_p]),
    "zdit_rope_table_scaled": (C.c_int, [C.c_void_p, C.c_int64, C.c_int32, C.c_float, C.POINTER(RopeScaling),
                                         C.c_void_p, C.c_void_p, C.c_void_p]),
    "zdit_qk_norm_rope": (C.c_int, [C.POINTER(QkNormRopeArgs), C.c_void_p]),
    "zdit_prompt_attention_workspace_bytes": (C.c_size_t, [C.POINTER(PromptAttentionArgs)]),
    "zdit_prompt_attention": (C.c_int, [C.POINTER(PromptAttentionArgs), C.c_void_p, C.c_size_t, C.c_void_p]),
    "zdit_linear": (C.c_int, [C.POINTER(LinearArgs), C.c_void_p]),
    "zdit_patchify": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p]),
    "zdit_unpatchify": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p]),
    "zdit_device_status": (C.c_int, [C.c_void_p]),
    "zdit_selftest_wait_timeout": (C.c_int, [C.c_void_p, C.c_void_p]),
}


def lib():
    """Load libzdit.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libzdit.so not built ({LIB_PATH}); run "
                               "`python -m stream_diffusion_transformer_s3_b200.build`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(code: int, where: str):
    if code != 0:
        raise ZditError(code, where)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


_torch = None


def _th():
    """torch, imported on the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _stream(stream=None):
    if stream is not None:
        return C.c_void_p(stream.cuda_stream)
    T = _th()
    raw = getattr(T._C, "_cuda_getCurrentRawStream", None)
    if raw is not None and T.cuda.is_initialized():
        # the current stream's handle without building a Stream object (0.1 instead of 3 us)
        return C.c_void_p(raw(T.cuda.current_device()))
    return C.c_void_p(T.cuda.current_stream().cuda_stream)


# ---------------------------------------------------------------- python-side config
@dataclass
class Dims:
    dim: int = 3840
    n_heads: int = 30
    head_dim: int = 128
    ffn_hidden: int = 10240
    temb_dim: int = 256
    rope_axes: tuple = (32, 48, 48)
    norm_eps: float = 1e-5
    rope_theta: float = 10000.0

    def cfg(self, flags: int) -> BlockCfg:
        c = BlockCfg()
        c.dim, c.n_heads, c.head_dim = self.dim, self.n_heads, self.head_dim
        c.ffn_hidden, c.temb_dim = self.ffn_hidden, self.temb_dim
        for i in range(3):
            c.rope_axes[i] = self.rope_axes[i]
        c.norm_eps, c.rope_theta, c.flags = self.norm_eps, self.rope_theta, flags
        return c


def flags_of(adaln=True, sandwich=True, qk_norm=False, tanh_gate=False) -> int:
    return (F_ADALN if adaln else 0) | (F_SANDWICH_NORM if sandwich else 0) | \
        (F_QK_NORM if qk_norm else 0) | (F_TANH_GATE if tanh_gate else 0)


class DeviceVarlen:
    """cu_seqlens on host and device, kept alive with the struct that points at them."""

    def __init__(self, cu_seqlens, device="cuda"):
        import torch
        cu = [int(v) for v in cu_seqlens]
        self.host = (C.c_int32 * len(cu))(*cu)
        self.dev = torch.tensor(cu, dtype=torch.int32, device=device)
        self.struct = Varlen(len(cu) - 1, C.c_void_p(self.dev.data_ptr()), self.host)
        self.total = cu[-1]


def interleave_gate_up(w1, w3):
    """[F, D] gate and up weights -> [2F, D] with 128-row blocks alternating
    (the w_gate_up layout declared in zdit.h).  Works on numpy arrays and tensors."""
    F = w1.shape[0]
    assert F % 128 == 0 and w3.shape == w1.shape
    if hasattr(w1, "reshape") and hasattr(w1, "dim"):  # torch
        import torch
        return torch.stack([w1.reshape(F // 128, 128, -1), w3.reshape(F // 128, 128, -1)], 1).reshape(2 * F, -1)
    import numpy as np
    return np.stack([w1.reshape(F // 128, 128, -1), w3.reshape(F // 128, 128, -1)], 1).reshape(2 * F, -1)


class DeviceBlock:
    """One block's weights in device memory (bf16 GEMM weights, fp32 norms/biases)."""

    def __init__(self, w: dict, device="cuda"):
        import torch
        bf = lambda a: torch.as_tensor(a, dtype=torch.float32).to(device=device, dtype=torch.bfloat16).contiguous()
        f32 = lambda a: torch.as_tensor(a, dtype=torch.float32).to(device).contiguous()
        self.t = {
            "w_qkv": bf(w["w_qkv"]), "w_out": bf(w["w_out"]),
            "w_gate_up": bf(interleave_gate_up(w["w1"], w["w3"])), "w_down": bf(w["w2"]),
        }
        for n in ("n_attn", "n_attn_post", "n_ffn", "n_ffn_post", "n_q", "n_k", "b_ada"):
            if n in w:
                self.t[n] = f32(w[n])
        if "w_ada" in w:
            self.t["w_ada"] = bf(w["w_ada"])
        self.struct = BlockWeights(**{n: (C.c_void_p(v.data_ptr())) for n, v in self.t.items()})

    @classmethod
    def from_tensors(cls, tensors: dict):
        self = cls.__new__(cls)
        self.t = dict(tensors)
        self.struct = BlockWeights(**{n: (C.c_void_p(v.data_ptr())) for n, v in self.t.items()})
        return self


# ------------------------------------------------------------------------ wrappers
def block_workspace_bytes(dims: Dims, flags: int, total_tokens: int, batch: int) -> int:
    c = dims.cfg(flags)
    return int(lib().zdit_block_workspace_bytes(C.byref(c), total_tokens, batch))


def zdit_block_forward(dims: Dims, flags: int, weights: DeviceBlock, varlen: DeviceVarlen, x, temb,
                       rope_cos, rope_sin, workspace, stream=None):
    c = dims.cfg(flags)
    code = lib().zdit_block_forward(C.byref(c), C.byref(weights.struct), C.byref(varlen.struct), _ptr(x),
                                    _ptr(temb), _ptr(rope_cos), _ptr(rope_sin), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check(code, "zdit_block_forward")


def zdit_block_forward_static(dims: Dims, flags: int, weights: DeviceBlock, varlen: DeviceVarlen, x, temb,
                              rope_cos, rope_sin, stream=None):
    """zdit_block_forward with the library's static 40 MiB scratch as workspace: for
    callers that cannot allocate device memory.  Calls must not overlap on the GPU."""
    c = dims.cfg(flags)
    code = lib().zdit_block_forward_static(C.byref(c), C.byref(weights.struct), C.byref(varlen.struct), _ptr(x),
                                           _ptr(temb), _ptr(rope_cos), _ptr(rope_sin), _stream(stream))
    _check(code, "zdit_block_forward_static")


def zdit_rope_table(pos, rope_axes, theta, cos_out, sin_out, head_dim=128, stream=None):
    axes = (C.c_int32 * 3)(*rope_axes)
    _check(lib().zdit_rope_table(_ptr(pos), pos.shape[0], head_dim, axes, theta, _ptr(cos_out),
                                 _ptr(sin_out), _stream(stream)), "zdit_rope_table")


def zdit_joint_attention(q, k, v, o, varlen: DeviceVarlen, n_heads, head_dim=128, stream=None):
    _check(lib().zdit_joint_attention(_ptr(q), q.stride(0), _ptr(k), k.stride(0), _ptr(v), v.stride(0),
                                      _ptr(o), o.stride(0), C.byref(varlen.struct), n_heads, head_dim,
                                      _stream(stream)), "zdit_joint_attention")


def zdit_gemm_bf16(A, B, Cout, bias=None, stream=None):
    M, K = A.shape
    N = B.shape[0]
    _check(lib().zdit_gemm_bf16(_ptr(A), _ptr(B), _ptr(Cout), M, N, K, Cout.stride(0), _ptr(bias),
                                _stream(stream)), "zdit_gemm_bf16")


def zdit_adaln_project(w_ada, b_ada, out, temb, stream=None):
    """out[i] [B, rows] = temb [B, E] . w_ada[i]^T [E, rows] + b_ada[i] for every i, one launch
    (lists of device tensors: w_ada bf16 [rows, E], b_ada fp32 [rows] or None, out fp32 [B, rows])."""
    n = len(w_ada)
    rows, E = w_ada[0].shape
    ws = (C.c_void_p * n)(*[t.data_ptr() for t in w_ada])
    bs = (C.c_void_p * n)(*[(b.data_ptr() if b is not None else None) for b in b_ada])
    os_ = (C.c_void_p * n)(*[t.data_ptr() for t in out])
    _check(lib().zdit_adaln_project(ws, bs, os_, n, _ptr(temb), temb.shape[0], E, rows, _stream(stream)),
           "zdit_adaln_project")


def zdit_euler_cfg_step(x, v_pos, v_neg, g, sigma_cur, sigma_next, stream=None):
    _check(lib().zdit_euler_cfg_step(_ptr(x), _ptr(v_pos), _ptr(v_neg), x.numel(), g, sigma_cur,
                                     sigma_next, _stream(stream)), "zdit_euler_cfg_step")


def zdit_sigma_schedule(n_steps: int):
    buf = (C.c_float * (n_steps + 1))()
    _check(lib().zdit_sigma_schedule(n_steps, buf), "zdit_sigma_schedule")
    return list(buf)


def zdit_patchify(latent, tokens, stream=None):
    Cc, H2, W2 = latent.shape
    _check(lib().zdit_patchify(_ptr(latent), _ptr(tokens), Cc, H2, W2, _stream(stream)), "zdit_patchify")


def zdit_unpatchify(tokens, latent, stream=None):
    Cc, H2, W2 = latent.shape
    _check(lib().zdit_unpatchify(_ptr(tokens), _ptr(latent), Cc, H2, W2, _stream(stream)), "zdit_unpatchify")


def zdit_selftest_wait_timeout(result_dev, stream=None):
    _check(lib().zdit_selftest_wait_timeout(_ptr(result_dev), _stream(stream)), "zdit_selftest_wait_timeout")


def zdit_device_status(stream=None):
    return int(lib().zdit_device_status(_stream(stream)))


# ------------------------------------------------------------------------ prompt operators
# These take torch tensors of any strides the C calls allow.  What the C structs cannot
# carry (element types, shapes, the device) is checked here.
def _packer(cls, fmt):
    """Builds a `cls` from its values in one step (field-wise construction of nested
    structures costs more than the launch of a small kernel)."""
    s = struct.Struct(fmt)
    assert s.size == C.sizeof(cls), (cls, s.size, C.sizeof(cls))
    pack, make = s.pack, cls.from_buffer_copy
    return lambda *v: make(pack(*v))


_NO_HEADS = (0, 0, 0)
_qk_args = _packer(QkNormRopeArgs, "@q5i4xPqqPqqPqqPqqPPf4xPPii")
_attn_args = _packer(PromptAttentionArgs, "@i4xPPP4if4xPqqPqqPqqPqq")
_linear_args = _packer(LinearArgs, "@qqqPqPqPi4xPqi4xPqi4x")


# (These run on every call of kernels that take a few us, so they read each property of a
# tensor once and format messages only on failure.)
def _dtype_code(t, where):
    T = _th()
    dt = t.dtype
    if dt is T.bfloat16:
        return 0
    if dt is T.float32:
        return 1
    raise ValueError(f"{where}: {dt} is neither bfloat16 nor float32")


def _launch_stream(where, stream, *tensors):
    """Handle of the stream to launch on; the tensors must be on the current device."""
    T = _th()
    dev = T.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: tensor on {t.device}, current device is cuda:{dev}")
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(T._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else T.cuda.current_stream().cuda_stream


def _f32(where, name, t, *shape):
    """Address of a contiguous fp32 tensor of that shape, 0 of None."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not _th().float32 or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous float32 {list(shape)}")
    return t.data_ptr()


def _heads(where, name, t, shape):
    """Heads fields (address, row stride, head stride) of a tensor of that [rows, heads,
    head_dim] shape whose last axis is contiguous."""
    if len(shape) != 3 or t.shape != shape:
        raise ValueError(f"{where}: {name} has shape {list(t.shape)}, expected [rows, heads, head_dim] = {list(shape)}")
    rs, hs, es = t.stride()
    if es != 1 and shape[2] > 1:
        raise ValueError(f"{where}: {name}'s last axis must be contiguous")
    return t.data_ptr(), rs, hs


def zdit_rope_table_scaled(pos, rotary_dim, theta, cos_out, sin_out, scaling: RopeScaling = None, stream=None):
    """cos / sin [T, rotary_dim / 2] (fp32) of one int32 position per token."""
    w = "zdit_rope_table_scaled"
    if pos.dtype is not _th().int32 or pos.dim() != 1 or not pos.is_contiguous():
        raise ValueError(f"{w}: pos must be a contiguous int32 vector")
    T = pos.shape[0]
    pc, ps = _f32(w, "cos_out", cos_out, T, rotary_dim // 2), _f32(w, "sin_out", sin_out, T, rotary_dim // 2)
    s = _launch_stream(w, stream, pos, cos_out, sin_out)
    if T == 0:
        return
    _check(lib().zdit_rope_table_scaled(pos.data_ptr(), T, rotary_dim, theta,
                                        C.byref(scaling) if scaling is not None else None, pc, ps, s), w)


def zdit_qk_norm_rope(q, k, q_out, k_out, w_q, w_k, cos, sin, rotary_dim, layout=ROPE_HALF, eps=1e-6, stream=None):
    """Per-head RMSNorm (w_q / w_k fp32 [head_dim], None: no norm) and rotation of q [T, n_q,
    head_dim] and k [T, n_k, head_dim] (k and k_out may be None) into q_out, k_out (which may
    be q and k themselves)."""
    w = "zdit_qk_norm_rope"
    shape = q.shape
    hq, hqo = _heads(w, "q", q, shape), _heads(w, "q_out", q_out, shape)
    T, n_q, hd = shape
    if (k is None) != (k_out is None):
        raise ValueError(f"{w}: k and k_out go together")
    n_k, hk, hko = 0, _NO_HEADS, _NO_HEADS
    if k is not None:
        kshape = k.shape
        if k.dtype is not q.dtype or k_out.dtype is not q_out.dtype or kshape[0] != T or kshape[2] != hd:
            raise ValueError(f"{w}: k must have q's type, rows and head_dim, and k_out q_out's type")
        n_k = kshape[1]
        hk, hko = _heads(w, "k", k, kshape), _heads(w, "k_out", k_out, kshape)
    pq, pk = _f32(w, "w_q", w_q, hd), _f32(w, "w_k", w_k, hd)
    pc, ps = 0, 0
    if rotary_dim:
        if cos is None or sin is None:
            raise ValueError(f"{w}: a rotation needs cos and sin")
        pc, ps = _f32(w, "cos", cos, T, rotary_dim // 2), _f32(w, "sin", sin, T, rotary_dim // 2)
    a = _qk_args(T, n_q, n_k, hd, _dtype_code(q, w), _dtype_code(q_out, w), *hq, *hk, *hqo, *hko, pq, pk, eps, pc, ps,
                 rotary_dim, layout)
    s = _launch_stream(w, stream, q, k, q_out, k_out, w_q, w_k, cos, sin)
    if T == 0:
        return
    _check(lib().zdit_qk_norm_rope(C.byref(a), s), w)


class PromptBatch:
    """Lengths of the packed sequences of zdit_prompt_attention (host arrays, kept alive):
    q_len new rows each; kv_len keys each (None: q_len); kv_start first key row of each
    (None: packed one after the other).  Other lengths need another batch: the rows that a
    call's tensors must have are counted here, once."""

    def __init__(self, q_len, kv_len=None, kv_start=None):
        def whole(v):
            if v is None:
                return None
            v = tuple(int(x) for x in v)
            if any(not -2**31 <= x < 2**31 for x in v):  # (ctypes would keep the low 32 bits)
                raise ValueError("PromptBatch: lengths and first rows must fit 32 bits")
            return v

        q_len, kv_len, kv_start = whole(q_len), whole(kv_len), whole(kv_start)
        n = len(q_len)
        if any(v is not None and len(v) != n for v in (kv_len, kv_start)):
            raise ValueError("PromptBatch: q_len, kv_len and kv_start must have one entry per sequence")
        lens = q_len if kv_len is None else kv_len
        ends = [sum(lens)] if kv_start is None else [s + m for s, m in zip(kv_start, lens)]
        arrays = tuple(None if v is None else (C.c_int32 * n)(*v) for v in (q_len, kv_len, kv_start))
        self.__dict__.update(batch=n, q_len=q_len, kv_len=kv_len, kv_start=kv_start, q_rows=sum(q_len),
                             kv_rows=max(ends, default=0), _arrays=arrays,
                             _addr=tuple(0 if v is None else C.addressof(v) for v in arrays))

    def __setattr__(self, name, value):
        raise AttributeError(f"PromptBatch: {name} cannot be set, make another batch")

    def __reduce__(self):  # copies make arrays of their own
        return PromptBatch, (self.q_len, self.kv_len, self.kv_start)

    def args(self, n_heads, n_kv_heads, head_dim, causal, scale, heads=_NO_HEADS * 4):
        return _attn_args(self.batch, *self._addr, n_heads, n_kv_heads, head_dim, 1 if causal else 0, scale, *heads)


def prompt_attention_workspace_bytes(batch: PromptBatch, n_heads, n_kv_heads, head_dim, causal=True) -> int:
    a = batch.args(n_heads, n_kv_heads, head_dim, causal, 0.0)
    return int(lib().zdit_prompt_attention_workspace_bytes(C.byref(a)))


def zdit_prompt_attention(q, k, v, o, batch: PromptBatch, workspace=None, causal=True, scale=0.0, stream=None):
    """Attention of packed prompts: q, o [rows, n_heads, head_dim], k, v [rows, n_kv_heads,
    head_dim], bf16, any row and head strides.  workspace: a contiguous uint8 tensor of
    prompt_attention_workspace_bytes (None when that is 0)."""
    w = "zdit_prompt_attention"
    bf = _th().bfloat16
    if not (q.dtype is bf and k.dtype is bf and v.dtype is bf and o.dtype is bf):
        raise ValueError(f"{w}: q, k, v and o must be bfloat16")
    qs, ks, os_ = q.shape, k.shape, o.shape
    hq, ho = _heads(w, "q", q, qs), _heads(w, "o", o, os_)
    hk, hv = _heads(w, "k", k, ks), _heads(w, "v", v, ks)
    (R, H, hd), (S, Hkv, khd), (Ro, Ho, ohd) = qs, ks, os_
    if Ho != H or not hd == khd == ohd:
        raise ValueError(f"{w}: o must have q's heads, and all the same head_dim")
    if R < batch.q_rows or Ro < batch.q_rows or S < batch.kv_rows:
        raise ValueError(f"{w}: the batch needs {batch.q_rows} rows of q and o and {batch.kv_rows} of k and v")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"{w}: workspace must be contiguous")
    s = _launch_stream(w, stream, q, k, v, o, workspace)
    a = batch.args(H, Hkv, hd, causal, scale, hq + hk + hv + ho)
    pw, nw = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check(lib().zdit_prompt_attention(C.byref(a), pw, nw, s), w)


def zdit_linear(a, w, out, bias=None, act=ACT_NONE, residual=None, stream=None):
    """out [M, N] = residual + act(a [M, K] . w [N, K]^T + bias): a and w bf16, bias fp32,
    residual and out fp32 or bf16; residual may be out."""
    n = "zdit_linear"
    bf = _th().bfloat16
    (M, K), (N, Kw) = a.shape, w.shape
    if a.dtype is not bf or w.dtype is not bf or Kw != K:
        raise ValueError(f"{n}: a [M, K] and w [N, K] must be bfloat16 matrices with the same K")
    (lda, ea), (ldw, ew), (ldo, eo) = a.stride(), w.stride(), out.stride()
    if (ea != 1 or ew != 1) and K > 1:
        raise ValueError(f"{n}: rows of a and w must be contiguous")
    if out.shape != (M, N) or (eo != 1 and N > 1):
        raise ValueError(f"{n}: out must be [{M}, {N}] with contiguous rows")
    pr, ldr, dr = 0, 0, 0
    if residual is not None:
        (ldr, er), pr, dr = residual.stride(), residual.data_ptr(), _dtype_code(residual, n)
        if residual.shape != (M, N) or (er != 1 and N > 1):
            raise ValueError(f"{n}: residual must be [{M}, {N}] with contiguous rows")
    g = _linear_args(M, N, K, a.data_ptr(), lda, w.data_ptr(), ldw, _f32(n, "bias", bias, N), act, pr, ldr, dr,
                     out.data_ptr(), ldo, _dtype_code(out, n))
    s = _launch_stream(n, stream, a, w, out, bias, residual)
    if M == 0:
        return
    _check(lib().zdit_linear(C.byref(g), s), n)


# ------------------------------------------------------------------------ stack
class DeviceStack:
    """All stack weights in device memory plus the C structs that point at them."""

    def __init__(self, W: dict, dims: Dims, n_noise: int, n_context: int, n_main: int,
                 patch_dim=64, cap_dim=2560, flags: int = F_ADALN | F_SANDWICH_NORM,
                 t_scale=1000.0, final_eps=1e-6, device="cuda", blocks=None):
        import torch
        bf = lambda a: torch.as_tensor(a, dtype=torch.float32).to(device=device, dtype=torch.bfloat16).contiguous()
        f32 = lambda a: torch.as_tensor(a, dtype=torch.float32).to(device).contiguous()
        self.dims, self.flags = dims, flags
        self.blocks = blocks if blocks is not None else [DeviceBlock(w, device) for w in W["blocks"]]
        assert len(self.blocks) == n_noise + n_context + n_main
        self.t = {}
        for n in ("w_x", "w_cap", "w_t1", "w_t2", "w_fada", "w_final"):
            self.t[n] = W[n] if hasattr(W[n], "data_ptr") else bf(W[n])
        for n in ("b_x", "w_capnorm", "b_cap", "pad_vec", "b_t1", "b_t2", "b_fada", "b_final"):
            self.t[n] = W[n] if hasattr(W[n], "data_ptr") else f32(W[n])
        self._barr = (BlockWeights * len(self.blocks))(*[b.struct for b in self.blocks])
        self.wstruct = StackWeights(C.cast(self._barr, C.POINTER(BlockWeights)),
                                    **{n: C.c_void_p(v.data_ptr()) for n, v in self.t.items()})
        self.cfg = StackCfg(dims.cfg(flags), n_noise, n_context, n_main, patch_dim, cap_dim, t_scale, final_eps)


class StackCall:
    """Inputs of one zdit_stack_forward call (host arrays kept alive)."""

    def __init__(self, grid, n_caps, n_valids, t, patches, cap_feats, shared_patches=False):
        B = len(n_caps)
        self.n_cap = (C.c_int32 * B)(*[int(v) for v in n_caps])
        self.n_valid = (C.c_int32 * B)(*[int(v) for v in n_valids])
        self.t = (C.c_float * B)(*[float(v) for v in t])
        self.patches, self.cap_feats = patches, cap_feats
        self.struct = StackInputs(B, int(grid[0]), int(grid[1]), self.n_cap, self.n_valid,
                                  C.c_void_p(patches.data_ptr()),
                                  C.c_void_p(cap_feats.data_ptr()) if cap_feats is not None else None,
                                  self.t, 1 if shared_patches else 0)

    def set_t(self, t):
        for i, v in enumerate(t):
            self.t[i] = float(v)


def stack_workspace_bytes(stack: DeviceStack, call: StackCall) -> int:
    return int(lib().zdit_stack_workspace_bytes(C.byref(stack.cfg), C.byref(call.struct)))


def zdit_stack_forward(stack: DeviceStack, call: StackCall, out, workspace, stream=None):
    _check(lib().zdit_stack_forward(C.byref(stack.cfg), C.byref(stack.wstruct), C.byref(call.struct),
                                    _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "zdit_stack_forward")


def zdit_profile_begin(max_records: int = 65536):
    _check(lib().zdit_profile_begin(max_records), "zdit_profile_begin")


def zdit_profile_end() -> dict:
    """{kernel kind: {launches, total_ms, flops, bytes}} of the launches recorded
    since zdit_profile_begin."""
    buf = (ProfileEntry * 32)()
    n = C.c_int32(0)
    _check(lib().zdit_profile_end(buf, 32, C.byref(n)), "zdit_profile_end")
    return {buf[i].name.decode(): {"launches": buf[i].launches, "total_ms": buf[i].total_ms,
                                   "flops": buf[i].flops, "bytes": buf[i].bytes} for i in range(n.value)}


def zdit_launch_count() -> int:
    return int(lib().zdit_launch_count())


def sample_workspace_bytes(stack: DeviceStack, call: StackCall) -> int:
    return int(lib().zdit_sample_workspace_bytes(C.byref(stack.cfg), C.byref(call.struct)))


def zdit_sample(stack: DeviceStack, call: StackCall, latent, workspace, n_steps=8, guidance=1.0,
                cache_context=True, dedup_noise=False, use_graph=False, stream=None):
    """In-place 8-step negated-CFG FlowMatchEuler sampling of `latent` [C, 2h, 2w].
    use_graph: capture the launch sequence as one CUDA graph and replay it on later calls
    with the same arguments."""
    sc = SampleCfg(n_steps, guidance, 1 if cache_context else 0, 1 if dedup_noise else 0, 1 if use_graph else 0)
    _check(lib().zdit_sample(C.byref(stack.cfg), C.byref(stack.wstruct), C.byref(call.struct), C.byref(sc),
                             _ptr(latent), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(stream)), "zdit_sample")
