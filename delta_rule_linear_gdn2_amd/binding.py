"""ctypes binding of ``libgdn2.so`` (the C ABI declared in include/gdn2.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or cannot bind to the
HIP runtime torch uses, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# GDN2_LIBRARY names another build of the library to load (the sanitizer
# check loads a build whose host code carries AddressSanitizer).
LIB_PATH = os.environ.get("GDN2_LIBRARY") or os.path.join(PKG, "libgdn2.so")

GDN2_OK = 0
STATUS_NAMES = {
    0: "GDN2_OK", 1: "GDN2_ERR_NULL_POINTER", 2: "GDN2_ERR_BAD_SHAPE", 3: "GDN2_ERR_UNSUPPORTED",
    4: "GDN2_ERR_BAD_DTYPE", 5: "GDN2_ERR_MISALIGNED", 6: "GDN2_ERR_ALIAS", 7: "GDN2_ERR_WORKSPACE",
    8: "GDN2_ERR_HIP",
}
DTYPE_F32 = 0
DTYPE_BF16 = 1

EXPORTS = ("gdn2_block_norm_bwd", "gdn2_block_norm_bwd_workspace_bytes", "gdn2_block_norm_fwd",
           "gdn2_chunk_bwd", "gdn2_chunk_bwd_noalloc", "gdn2_chunk_bwd_noalloc_max_workspace_bytes",
           "gdn2_chunk_bwd_workspace_bytes", "gdn2_chunk_fwd", "gdn2_chunk_fwd_gates",
           "gdn2_chunk_fwd_workspace_bytes", "gdn2_dropout",
           "gdn2_linear_attn_bwd", "gdn2_linear_attn_bwd_workspace_bytes", "gdn2_linear_attn_fwd",
           "gdn2_linear_attn_fwd_workspace_bytes", "gdn2_linear_attn_step",
           "gdn2_mixer_epilogue", "gdn2_mixer_epilogue_bwd", "gdn2_mixer_epilogue_bwd_workspace_bytes",
           "gdn2_mixer_prologue", "gdn2_mixer_prologue_bwd", "gdn2_mixer_prologue_bwd_workspace_bytes",
           "gdn2_mixer_prologue_bwd_zeroed",
           "gdn2_qk_norm_rope", "gdn2_qk_norm_rope_bwd", "gdn2_qk_norm_rope_bwd_workspace_bytes",
           "gdn2_recurrent_fwd", "gdn2_recurrent_step",
           "gdn2_recurrent_step_gates", "gdn2_status_string", "gdn2_version")

# gdn2_gate_flags: layout of the gates (b, w, alpha), OR-ed together
GATES_FULL, GATES_SCALAR_ERASE, GATES_SCALAR_WRITE, GATES_TIED, GATES_SCALAR_DECAY = 0, 1, 2, 4, 8
GATES_KDA = GATES_SCALAR_ERASE | GATES_TIED
GATES_GDN = GATES_KDA | GATES_SCALAR_DECAY
VALID_GATES = (0, 1, 2, 3, 5, 8, 9, 10, 11, 13)


class Gdn2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {status_string(status)}")


_LIB = None


def _hip_runtimes_loaded() -> set[str]:
    paths = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                if "libamdhip64" in line:
                    paths.add(os.path.realpath(line.split()[-1]))
    except OSError:
        pass
    return paths


def load(path: str = LIB_PATH):
    """Load ``libgdn2.so`` (after torch, so it binds to torch's HIP runtime)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    import torch  # noqa: F401  -- loads torch's libamdhip64 first (same SONAME)

    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; build it with `python -m delta_rule_linear_gdn2_amd.build` "
            "(the GDN-2 ops have no non-HIP implementation)")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.gdn2_chunk_fwd.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, Z, P]
    lib.gdn2_chunk_fwd.restype = ctypes.c_int
    lib.gdn2_chunk_fwd_gates.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, Z, P]
    lib.gdn2_chunk_fwd_gates.restype = ctypes.c_int
    lib.gdn2_chunk_fwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.gdn2_chunk_fwd_workspace_bytes.restype = Z
    lib.gdn2_recurrent_step.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P]
    lib.gdn2_recurrent_step.restype = ctypes.c_int
    lib.gdn2_recurrent_step_gates.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, P]
    lib.gdn2_recurrent_step_gates.restype = ctypes.c_int
    lib.gdn2_recurrent_fwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
    lib.gdn2_recurrent_fwd.restype = ctypes.c_int
    lib.gdn2_chunk_bwd.argtypes = [P] * 17 + [I, I, I, I, I, I, I, P, Z, P]
    lib.gdn2_chunk_bwd.restype = ctypes.c_int
    lib.gdn2_chunk_bwd_noalloc.argtypes = [P] * 17 + [I, I, I, I, I, I, I, P]
    lib.gdn2_chunk_bwd_noalloc.restype = ctypes.c_int
    lib.gdn2_chunk_bwd_noalloc_max_workspace_bytes.argtypes = []
    lib.gdn2_chunk_bwd_noalloc_max_workspace_bytes.restype = Z
    lib.gdn2_chunk_bwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.gdn2_chunk_bwd_workspace_bytes.restype = Z
    F = ctypes.c_float
    lib.gdn2_mixer_prologue.argtypes = [P] * 16 + [I] * 7 + [F, F, I, P]
    lib.gdn2_mixer_prologue.restype = ctypes.c_int
    lib.gdn2_mixer_epilogue.argtypes = [P, P, P, P, ctypes.c_int64, I, F, I, I, P]
    lib.gdn2_mixer_epilogue.restype = ctypes.c_int
    L, D, U = ctypes.c_int64, ctypes.c_double, ctypes.c_uint64
    lib.gdn2_block_norm_fwd.argtypes = [P] * 7 + [L, I, F, F, I, I, D, U, U, P, I, I, P]
    lib.gdn2_block_norm_fwd.restype = ctypes.c_int
    lib.gdn2_block_norm_bwd.argtypes = [P] * 12 + [L, I, F, F, I, I, D, U, U, P, I, I, P, Z, P]
    lib.gdn2_block_norm_bwd.restype = ctypes.c_int
    lib.gdn2_block_norm_bwd_workspace_bytes.argtypes = [L, I]
    lib.gdn2_block_norm_bwd_workspace_bytes.restype = Z
    lib.gdn2_dropout.argtypes = [P, P, L, L, D, U, U, P, I, P]
    lib.gdn2_dropout.restype = ctypes.c_int
    lib.gdn2_mixer_epilogue_bwd.argtypes = [P] * 7 + [L, I, F, I, I, P, Z, P]
    lib.gdn2_mixer_epilogue_bwd.restype = ctypes.c_int
    lib.gdn2_mixer_epilogue_bwd_workspace_bytes.argtypes = [L, I]
    lib.gdn2_mixer_epilogue_bwd_workspace_bytes.restype = Z
    for f in (lib.gdn2_mixer_prologue_bwd, lib.gdn2_mixer_prologue_bwd_zeroed):
        f.argtypes = [P] * 25 + [I] * 7 + [F, F, I, P, Z, P]
        f.restype = ctypes.c_int
    lib.gdn2_mixer_prologue_bwd_workspace_bytes.argtypes = [I] * 6
    lib.gdn2_mixer_prologue_bwd_workspace_bytes.restype = Z
    lib.gdn2_linear_attn_fwd.argtypes = [P] * 8 + [I] * 8 + [P, Z, P]
    lib.gdn2_linear_attn_fwd.restype = ctypes.c_int
    lib.gdn2_linear_attn_bwd.argtypes = [P] * 12 + [I] * 8 + [P, Z, P]
    lib.gdn2_linear_attn_bwd.restype = ctypes.c_int
    for f in (lib.gdn2_linear_attn_fwd_workspace_bytes, lib.gdn2_linear_attn_bwd_workspace_bytes):
        f.argtypes = [I] * 7
        f.restype = Z
    lib.gdn2_linear_attn_step.argtypes = [P] * 6 + [I] * 5 + [P]
    lib.gdn2_linear_attn_step.restype = ctypes.c_int
    lib.gdn2_qk_norm_rope.argtypes = [P] * 8 + [I] * 7 + [F, F, I, P]
    lib.gdn2_qk_norm_rope.restype = ctypes.c_int
    lib.gdn2_qk_norm_rope_bwd.argtypes = [P] * 12 + [I] * 7 + [F, F, I, P, Z, P]
    lib.gdn2_qk_norm_rope_bwd.restype = ctypes.c_int
    lib.gdn2_qk_norm_rope_bwd_workspace_bytes.argtypes = [I] * 5
    lib.gdn2_qk_norm_rope_bwd_workspace_bytes.restype = Z
    lib.gdn2_status_string.argtypes = [ctypes.c_int]
    lib.gdn2_status_string.restype = ctypes.c_char_p
    lib.gdn2_version.argtypes = []
    lib.gdn2_version.restype = ctypes.c_int32
    runtimes = _hip_runtimes_loaded()
    if len(runtimes) > 1:
        raise RuntimeError(f"two HIP runtimes are mapped in this process: {sorted(runtimes)}")
    _LIB = lib
    return lib


def status_string(status: int) -> str:
    return load().gdn2_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt) -> int:
    import torch

    if dt == torch.bfloat16:
        return DTYPE_BF16
    if dt == torch.float32:
        return DTYPE_F32
    raise TypeError(f"unsupported dtype {dt} (float32 or bfloat16)")


def _check(name, t, shape, dtype, device):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {shape}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def gdn2_chunk_fwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code) -> int:
    return int(load().gdn2_chunk_fwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code))


def _gate_widths(gates, dk, dv):
    """Trailing sizes of (b, w, alpha) for a gate layout (w None: not used)."""
    if gates not in VALID_GATES:
        raise ValueError(f"gates must be one of {VALID_GATES} (got {gates})")
    bw = () if gates & GATES_SCALAR_ERASE else (dk,)
    ww = None if gates & GATES_TIED else () if gates & GATES_SCALAR_WRITE else (dv,)
    aw = () if gates & GATES_SCALAR_DECAY else (dk,)
    return bw, ww, aw


def _chunk_fwd(q, k, v, alpha, b, w, gates, initial_state, output_final_state, final_state, out,
               cu_seqlens, stream, segmented=True):
    import torch

    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    N = B if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    bw, ww, aw = _gate_widths(gates, dk, dv)
    for name, t, width in (("q", q, dk), ("k", k, dk), ("v", v, dv)):
        _check(name, t, (B, T, H, width), dt, dev)
    _check("b", b, (B, T, H) + bw, dt, dev)
    if ww is not None:
        _check("w", w, (B, T, H) + ww, dt, dev)
    else:
        w = None
    _check("alpha", alpha, (B, T, H) + aw, torch.float32, dev)
    if initial_state is not None:
        _check("initial_state", initial_state, (N, H, dk, dv), torch.float32, dev)
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    else:
        _check("out", out, (B, T, H, dv), dt, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    elif final_state is not None:
        _check("final_state", final_state, (N, H, dk, dv), torch.float32, dev)
    ws_bytes = gdn2_chunk_fwd_workspace_bytes(B, T, H, dk, dv, N if cu_seqlens is not None else 0, code)
    if not segmented:
        ws_bytes = 0
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(initial_state), _ptr(final_state),
            _ptr(out), _ptr(cu_seqlens), B, T, H, dk, dv, N, code)
    tail = (_ptr(ws), ws_bytes, _stream(stream))
    if gates == GATES_FULL:
        rc, name = lib.gdn2_chunk_fwd(*args, *tail), "gdn2_chunk_fwd"
    else:
        rc, name = lib.gdn2_chunk_fwd_gates(*args, gates, *tail), "gdn2_chunk_fwd_gates"
    if rc != GDN2_OK:
        raise Gdn2Error(rc, name)
    return out, final_state


def gdn2_chunk_fwd(q, k, v, alpha, b, w, initial_state=None, *, output_final_state=True,
                   final_state=None, out=None, cu_seqlens=None, stream=None, segmented=True):
    """Chunkwise GDN-2 forward.  Returns ``(o, final_state)`` (final_state may be None).

    q, k, b: [B, T, H, dk]; v, w: [B, T, H, dv] (float32 or bfloat16, all the
    same); alpha: [B, T, H, dk] float32; initial_state: [N, H, dk, dv] float32
    or None; cu_seqlens: int32 [N + 1] on the device or None (then B must be 1).
    ``final_state`` may be passed (e.g. the initial_state tensor itself for an
    in-place update); otherwise it is allocated when ``output_final_state``.
    The workspace gdn2_chunk_fwd_workspace_bytes asks for is allocated, which
    selects the segmented path for few-chain shapes; ``segmented=False``
    passes none (the single pass).
    """
    return _chunk_fwd(q, k, v, alpha, b, w, GATES_FULL, initial_state, output_final_state, final_state, out,
                      cu_seqlens, stream, segmented)


def gdn2_chunk_fwd_gates(q, k, v, alpha, b, w, gates, initial_state=None, *, output_final_state=True,
                         final_state=None, out=None, cu_seqlens=None, stream=None, segmented=True):
    """gdn2_chunk_fwd with a gate layout, an OR of the GATES_* flags:
    SCALAR_ERASE takes b as [B, T, H]; SCALAR_WRITE takes w as [B, T, H];
    TIED (with SCALAR_ERASE) uses b as the write gate too (w ignored, may be
    None); SCALAR_DECAY takes alpha as [B, T, H] float32.  GATES_FULL is
    gdn2_chunk_fwd; GATES_KDA and GATES_GDN are the two reductions."""
    return _chunk_fwd(q, k, v, alpha, b, w, gates, initial_state, output_final_state, final_state, out,
                      cu_seqlens, stream, segmented)


def _recurrent_step(q, k, v, alpha, b, w, gates, state, out, stream):
    import torch

    lib = load()
    N, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    bw, ww, aw = _gate_widths(gates, dk, dv)
    for name, t, width in (("q", q, dk), ("k", k, dk), ("v", v, dv)):
        _check(name, t, (N, H, width), dt, dev)
    _check("b", b, (N, H) + bw, dt, dev)
    if ww is not None:
        _check("w", w, (N, H) + ww, dt, dev)
    else:
        w = None
    _check("alpha", alpha, (N, H) + aw, torch.float32, dev)
    _check("state", state, (N, H, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty((N, H, dv), dtype=dt, device=dev)
    else:
        _check("out", out, (N, H, dv), dt, dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(state), _ptr(out), N, H, dk, dv, code)
    if gates == GATES_FULL:
        rc, name = lib.gdn2_recurrent_step(*args, _stream(stream)), "gdn2_recurrent_step"
    else:
        rc, name = lib.gdn2_recurrent_step_gates(*args, gates, _stream(stream)), "gdn2_recurrent_step_gates"
    if rc != GDN2_OK:
        raise Gdn2Error(rc, name)
    return out


def gdn2_recurrent_step(q, k, v, alpha, b, w, state, *, out=None, stream=None):
    """One fused recurrent (decode) step; updates ``state`` in place, returns o.

    q, k, b: [N, H, dk]; v, w: [N, H, dv]; alpha: [N, H, dk] float32;
    state: [N, H, dk, dv] float32.
    """
    return _recurrent_step(q, k, v, alpha, b, w, GATES_FULL, state, out, stream)


def gdn2_recurrent_step_gates(q, k, v, alpha, b, w, gates, state, *, out=None, stream=None):
    """gdn2_recurrent_step with a gate layout (see gdn2_chunk_fwd_gates); a
    scalar gate is [N, H]."""
    return _recurrent_step(q, k, v, alpha, b, w, gates, state, out, stream)


def gdn2_recurrent_fwd(q, k, v, alpha, b, w, state, *, gates=GATES_FULL, out=None, stream=None):
    """The fused recurrent form over T tokens per sequence in one call; updates
    ``state`` in place and returns o.

    q, k, b: [N, T, H, dk]; v, w: [N, T, H, dv]; alpha: [N, T, H, dk] float32
    (scalar gates [N, T, H] as the ``gates`` layout says); state:
    [N, H, dk, dv] float32.
    """
    import torch

    lib = load()
    N, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    bw, ww, aw = _gate_widths(gates, dk, dv)
    for name, t, width in (("q", q, dk), ("k", k, dk), ("v", v, dv)):
        _check(name, t, (N, T, H, width), dt, dev)
    _check("b", b, (N, T, H) + bw, dt, dev)
    if ww is not None:
        _check("w", w, (N, T, H) + ww, dt, dev)
    else:
        w = None
    _check("alpha", alpha, (N, T, H) + aw, torch.float32, dev)
    _check("state", state, (N, H, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty((N, T, H, dv), dtype=dt, device=dev)
    else:
        _check("out", out, (N, T, H, dv), dt, dev)
    rc = lib.gdn2_recurrent_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(state), _ptr(out),
                                N, T, H, dk, dv, code, gates, _stream(stream))
    if rc != GDN2_OK:
        raise Gdn2Error(rc, "gdn2_recurrent_fwd")
    return out


def gdn2_chunk_bwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code) -> int:
    return int(load().gdn2_chunk_bwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code))


def gdn2_chunk_bwd(q, k, v, alpha, b, w, d_o, initial_state=None, d_final_state=None, *, cu_seqlens=None,
                   output_d_initial_state=True, d_initial_state=None, workspace=None, stream=None):
    """Gradients of gdn2_chunk_fwd for the loss <d_o, o> + <d_final_state, S_final>.

    Inputs as for gdn2_chunk_fwd, plus d_o [B, T, H, dv] (input dtype) and
    d_final_state [N, H, dk, dv] float32 or None.  Returns a dict with dq, dk,
    db [B, T, H, dk] and dv, dw [B, T, H, dv] (input dtype), dalpha [B, T, H, dk]
    float32 and d_initial_state [N, H, dk, dv] float32 (None if not wanted).
    ``workspace`` (uint8 device tensor) is allocated when not given.
    """
    import torch

    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    N = B if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t, width in (("q", q, dk), ("k", k, dk), ("b", b, dk), ("v", v, dv), ("w", w, dv),
                           ("d_o", d_o, dv)):
        _check(name, t, (B, T, H, width), dt, dev)
    _check("alpha", alpha, (B, T, H, dk), torch.float32, dev)
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            _check(name, t, (N, H, dk, dv), torch.float32, dev)
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    out = {name: torch.empty((B, T, H, width), dtype=dt, device=dev)
           for name, width in (("dq", dk), ("dk", dk), ("db", dk), ("dv", dv), ("dw", dv))}
    out["dalpha"] = torch.empty((B, T, H, dk), dtype=torch.float32, device=dev)
    if d_initial_state is not None:
        _check("d_initial_state", d_initial_state, (N, H, dk, dv), torch.float32, dev)
    elif output_d_initial_state:
        d_initial_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    out["d_initial_state"] = d_initial_state
    ws_bytes = gdn2_chunk_bwd_workspace_bytes(B, T, H, dk, dv, N if cu_seqlens is not None else 0, code)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev) if ws_bytes else None
    elif workspace.numel() < ws_bytes:
        raise ValueError(f"workspace of {workspace.numel()} bytes < {ws_bytes}")
    rc = lib.gdn2_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(initial_state),
                            _ptr(d_o), _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                            _ptr(out["dalpha"]), _ptr(out["db"]), _ptr(out["dw"]), _ptr(d_initial_state),
                            _ptr(cu_seqlens), B, T, H, dk, dv, N, code, _ptr(workspace),
                            0 if workspace is None else workspace.numel(), _stream(stream))
    if rc != GDN2_OK:
        raise Gdn2Error(rc, "gdn2_chunk_bwd")
    return out


def gdn2_chunk_bwd_noalloc_max_workspace_bytes() -> int:
    return int(load().gdn2_chunk_bwd_noalloc_max_workspace_bytes())


def gdn2_chunk_bwd_noalloc(q, k, v, alpha, b, w, d_o, initial_state=None, d_final_state=None, *, out,
                           cu_seqlens=None, stream=None):
    """gdn2_chunk_bwd on the library's own workspace (the call allocates nothing).

    ``out``: dict of preallocated outputs dq, dk, db [B, T, H, dk] and dv, dw
    [B, T, H, dv] (input dtype), dalpha [B, T, H, dk] float32 and
    d_initial_state [N, H, dk, dv] float32 or None; filled in place and
    returned."""
    import torch

    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(dt)
    N = B if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t, width in (("q", q, dk), ("k", k, dk), ("b", b, dk), ("v", v, dv), ("w", w, dv),
                           ("d_o", d_o, dv), ("dq", out["dq"], dk), ("dk", out["dk"], dk), ("db", out["db"], dk),
                           ("dv", out["dv"], dv), ("dw", out["dw"], dv)):
        _check(name, t, (B, T, H, width), dt, dev)
    _check("alpha", alpha, (B, T, H, dk), torch.float32, dev)
    _check("dalpha", out["dalpha"], (B, T, H, dk), torch.float32, dev)
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state),
                    ("d_initial_state", out.get("d_initial_state"))):
        if t is not None:
            _check(name, t, (N, H, dk, dv), torch.float32, dev)
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    rc = lib.gdn2_chunk_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(b), _ptr(w), _ptr(initial_state),
                                    _ptr(d_o), _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]),
                                    _ptr(out["dv"]), _ptr(out["dalpha"]), _ptr(out["db"]), _ptr(out["dw"]),
                                    _ptr(out.get("d_initial_state")), _ptr(cu_seqlens), B, T, H, dk, dv, N, code,
                                    _stream(stream))
    if rc != GDN2_OK:
        raise Gdn2Error(rc, "gdn2_chunk_bwd_noalloc")
    return out


GATE_ACTS = {"sigmoid": 0, "silu": 1}


def gdn2_mixer_prologue(xq, xk, xv, conv_q, conv_k, conv_v, b_logit, w_logit, *, conv_state=None,
                        output_conv_state=True, conv_state_out=None, cu_seqlens=None, q_scale=1.0, eps_l2=1e-6,
                        stream=None):
    """q, k, v, b, w of the recurrence from the projection outputs (one pass).

    xq, xk, b_logit: [B, T, H, dk]; xv, w_logit: [B, T, H, dv] (float32 or
    bfloat16); conv_q, conv_k: [H * dk, K], conv_v: [H * dv, K] float32;
    conv_state: [N, H * (2 dk + dv), K - 1] float32 or None (zeros).  Returns
    dict(q, k, v, b, w, conv_state) with the final convolution state (None if
    not wanted; pass conv_state_out=conv_state for an in-place decode step).
    """
    import torch

    lib = load()
    B, T, H, dk = xq.shape
    dv = xv.shape[-1]
    K = conv_q.shape[-1]
    dev, dt = xq.device, xq.dtype
    code = _dtype_code(dt)
    N = B if cu_seqlens is None else int(cu_seqlens.shape[0]) - 1
    for name, t, width in (("xq", xq, dk), ("xk", xk, dk), ("b_logit", b_logit, dk), ("xv", xv, dv),
                           ("w_logit", w_logit, dv)):
        _check(name, t, (B, T, H, width), dt, dev)
    for name, t, width in (("conv_q", conv_q, dk), ("conv_k", conv_k, dk), ("conv_v", conv_v, dv)):
        _check(name, t, (H * width, K), torch.float32, dev)
    st_shape = (N, H * (2 * dk + dv), K - 1)
    if conv_state is not None:
        _check("conv_state", conv_state, st_shape, torch.float32, dev)
    if conv_state_out is not None:
        _check("conv_state_out", conv_state_out, st_shape, torch.float32, dev)
    elif output_conv_state:
        conv_state_out = torch.empty(st_shape, dtype=torch.float32, device=dev)
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    out = {name: torch.empty((B, T, H, width), dtype=dt, device=dev)
           for name, width in (("q", dk), ("k", dk), ("b", dk), ("v", dv), ("w", dv))}
    rc = lib.gdn2_mixer_prologue(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(conv_q), _ptr(conv_k), _ptr(conv_v),
                                 _ptr(b_logit), _ptr(w_logit), _ptr(conv_state), _ptr(conv_state_out),
                                 _ptr(out["q"]), _ptr(out["k"]), _ptr(out["v"]), _ptr(out["b"]), _ptr(out["w"]),
                                 _ptr(cu_seqlens), B, T, H, dk, dv, K, N, float(q_scale), float(eps_l2), code,
                                 _stream(stream))
    if rc != GDN2_OK:
        raise Gdn2Error(rc, "gdn2_mixer_prologue")
    out["conv_state"] = conv_state_out
    return out


def gdn2_mixer_epilogue(o, gate, weight, *, eps=1e-5, act="sigmoid", out=None, stream=None):
    """RMS-normalised o times weight times act(gate), over the last axis (dv).

    o, gate: [..., dv] (float32 or bfloat16, same shape); weight: [dv] float32;
    act: "sigmoid" or "silu"."""
    import torch

    lib = load()
    dv = o.shape[-1]
    dev, dt = o.device, o.dtype
    code = _dtype_code(dt)
    _check("gate", gate, tuple(o.shape), dt, dev)
    _check("weight", weight, (dv,), torch.float32, dev)
    if not o.is_contiguous():
        raise ValueError("o: must be contiguous")
    if out is None:
        out = torch.empty_like(o)
    else:
        _check("out", out, tuple(o.shape), dt, dev)
    if act not in GATE_ACTS:
        raise ValueError(f"act must be one of {tuple(GATE_ACTS)}")
    rows = o.numel() // dv
    rc = lib.gdn2_mixer_epilogue(_ptr(o), _ptr(gate), _ptr(weight), _ptr(out), rows, dv, float(eps),
                                 GATE_ACTS[act], code, _stream(stream))
    if rc != GDN2_OK:
        raise Gdn2Error(rc, "gdn2_mixer_epilogue")
    return out


# --- training operators ------------------------------------------------------

# A small call's time is this module's own: torch is imported once (at the first
# call, not with the package), sizes are asked of the library once per shape, and
# whatever can only raise comes after one comparison that says it need not.
torch = None
_CODES = {}


def _import_torch():
    global torch
    import torch as module

    load()
    _CODES.update({module.float32: DTYPE_F32, module.bfloat16: DTYPE_BF16})
    torch = module  # last: from here on calls take the rest as done


def _code(dt):
    return _CODES[dt] if dt in _CODES else _dtype_code(dt)  # the latter raises


def _on_stream(f):
    """Runs a call on ``stream`` (default: the current stream of its tensors'
    device), with that device current.  What the call allocates (outputs,
    workspace) belongs to that stream, and the caller's tensors are recorded on
    it: memory that one stream still uses is never handed to another."""

    signature = inspect.signature(f)
    name = next(iter(signature.parameters))

    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if torch is None:
            _import_torch()
        first = args[0] if args else kw.get(name)
        if first is None:
            return f(*args, **kw)  # raises
        if stream is not None:
            if stream.device != first.device:
                raise ValueError(f"stream: on {stream.device}, the tensors are on {first.device}")
            for t in (*args, *kw.values()):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
            with torch.cuda.stream(stream):
                return f(*args, **kw)
        index = first.get_device()
        if index >= 0 and index != torch.cuda.current_device():
            with torch.cuda.device(index):
                return f(*args, **kw)
        return f(*args, **kw)

    parameters = [*signature.parameters.values(), inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)]
    call.__signature__ = signature.replace(parameters=parameters)
    return call


def _run(name, index, *args):
    """Calls the C function on device ``index``'s current stream (its handle
    alone: building the stream object takes longer than all checks); raises
    what it refuses."""
    if index < 0:
        raise ValueError(f"{name}: tensors must be on a GPU")
    rc = getattr(_LIB, name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != GDN2_OK:
        raise Gdn2Error(rc, name)


def _expect(name, t, shape, dtype, index):
    """_check at a fifth of its time where nothing is wrong."""
    if not (t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous()):
        _check(name, t, tuple(shape), dtype, torch.device("cuda", index) if index >= 0 else torch.device("cpu"))


def _addr(t):
    return None if t is None else t.data_ptr()


def _buffer(name, t, like, shape, dtype, index):
    """The caller's output tensor, checked, or a new one like ``like`` (of that
    shape, type and device)."""
    if t is None:
        return torch.empty_like(like)
    _expect(name, t, shape, dtype, index)
    return t


def _workspace(t, nbytes, like):
    """The caller's workspace, checked, or a new one on ``like``'s device."""
    if not nbytes:
        return None, 0
    if t is None:
        return like.new_empty(nbytes, dtype=torch.uint8), nbytes
    dev = like.device
    if t.dtype != torch.uint8 or t.device != dev or not t.is_contiguous():
        raise ValueError(f"workspace: must be contiguous uint8 on {dev}")
    if t.numel() < nbytes:
        raise ValueError(f"workspace of {t.numel()} bytes < {nbytes}")
    return t, t.numel()


def _rows(name, t, shape):
    if not shape or shape[-1] < 1:
        raise ValueError(f"{name}: needs a last axis of at least one element (shape {tuple(shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.numel() // shape[-1]


def _random(seed, offset, offset_device, index):
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError(f"seed and offset must be in [0, 2^64) (got {seed}, {offset})")
    seed, offset = int(seed), int(offset)
    if offset_device is None:
        return seed, offset, None
    _expect("offset_device", offset_device, (1,), torch.int64, index)
    return seed, offset, offset_device.data_ptr()


GATE_LAYOUTS = {"none": 0, "channel": 1, "token": 2, "full": 3}
BLOCK_GATE_ACTS = {"sigmoid": 0, "silu": 1, "identity": 2}


def _block_inputs(x, u, gate, gate_layout, gate_act, weight_post, weight_pre):
    """Checks the inputs that the block norm's two directions share; returns
    their rows, shape and device index, and the codes of gate and activation."""
    shape, index = x.shape, x.get_device()
    rows = _rows("x", x, shape)
    if u is not None:
        _expect("u", u, shape, u.dtype, index)
    layout, act = GATE_LAYOUTS.get(gate_layout), BLOCK_GATE_ACTS.get(gate_act)
    if layout is None:
        raise ValueError(f"gate_layout must be one of {tuple(GATE_LAYOUTS)}")
    if act is None:
        raise ValueError(f"gate_act must be one of {tuple(BLOCK_GATE_ACTS)}")
    if gate is None:
        if layout:
            raise ValueError(f"gate_layout {gate_layout!r} needs a gate")
    elif layout == 1:
        _expect("gate", gate, shape[-1:], torch.float32, index)
    elif not layout:
        raise ValueError("a gate needs a gate_layout")
    elif u is not None:
        _expect("gate", gate, shape if layout == 3 else shape[:-1], u.dtype, index)
    if weight_post is not None:
        _expect("weight_post", weight_post, shape[-1:], torch.float32, index)
    if weight_pre is not None:
        _expect("weight_pre", weight_pre, shape[-1:], torch.float32, index)
    return rows, shape, index, layout, act


@_on_stream
def gdn2_block_norm_fwd(x, u=None, *, gate=None, gate_layout="none", gate_act="sigmoid", weight_post=None,
                        weight_pre=None, eps=1e-5, residual_scale=1.0, dropout_p=0.0, seed=0, offset=0,
                        offset_device=None, dtype=None, x_out=None, h=None):
    """The step from one block to the next: returns ``(x_out, h)``.

        n = u / rms(u) * weight_post                       (u itself without weight_post)
        x_out = x + residual_scale * dropout(act(gate) * n)
        h = x_out / rms(x_out) * weight_pre                (None without weight_pre)

    x: the residual stream, [..., D] float32 or bfloat16; u: the block's output,
    the same shape, or None (then h is the norm of x, and the returned x_out is
    x).  The stream is u's type, or float32 with bfloat16 blocks.  gate: None, or
    as gate_layout says: "channel" [D] float32, "token" [...] or "full" [..., D]
    of u's type; gate_act "sigmoid", "silu" or "identity".  weight_post,
    weight_pre: [D] float32 or None (no such norm).  dropout_p with seed, offset
    (integers in [0, 2^64)) and offset_device ([1] int64 on the device, added to
    offset; or None) as for gdn2_dropout.  dtype: h's type where u is None
    (default x's).  x_out may be x (in place); x_out and h are allocated when not
    given.
    """
    rows, shape, index, layout, act = _block_inputs(x, u, gate, gate_layout, gate_act, weight_post, weight_pre)
    rdt = x.dtype
    dt = u.dtype if u is not None else dtype or rdt
    if u is not None:
        if dtype is not None and dtype != dt:
            raise TypeError(f"dtype: h has u's type, {dt} (got {dtype})")
        x_out = _buffer("x_out", x_out, x, shape, rdt, index)
    elif x_out is not None:
        raise ValueError("x_out: there is none without u")
    if weight_pre is None:
        if h is not None:
            raise ValueError("h: there is none without weight_pre")
    elif u is not None:
        h = _buffer("h", h, u, shape, dt, index)
    elif h is None:
        h = x.new_empty(shape, dtype=dt)
    else:
        _expect("h", h, shape, dt, index)
    _run("gdn2_block_norm_fwd", index, x.data_ptr(), _addr(u), _addr(gate), _addr(weight_post), _addr(weight_pre),
         _addr(x_out), _addr(h), rows, shape[-1], eps, residual_scale, layout, act, dropout_p,
         *_random(seed, offset, offset_device, index), _code(dt), _code(rdt))
    return (x if u is None else x_out), h


@functools.lru_cache(maxsize=256)
def gdn2_block_norm_bwd_workspace_bytes(rows, D) -> int:
    return int(load().gdn2_block_norm_bwd_workspace_bytes(rows, D))


@_on_stream
def gdn2_block_norm_bwd(x_out, u, d_x_out, d_h, *, gate=None, gate_layout="none", gate_act="sigmoid", weight_post=None,
                        weight_pre=None, eps=1e-5, residual_scale=1.0, dropout_p=0.0, seed=0, offset=0,
                        offset_device=None, d_x=None, d_u=None, d_gate=None, want_d_gate=True, want_d_weights=True,
                        workspace=None):
    """Gradients of gdn2_block_norm_fwd for the loss <d_x_out, x_out> + <d_h, h>.

    x_out: the stream the forward call returned; u and the keyword arguments:
    the forward call's; d_x_out: like x_out, or None for zero; d_h: like h, None
    exactly when weight_pre is.  Returns dict(d_x, d_u, d_gate, d_weight_post,
    d_weight_pre), None in the place of what has no input or is not wanted.  d_x
    may be d_x_out (in place).  ``workspace`` (uint8) is allocated when not given.
    """
    rows, shape, index, layout, act = _block_inputs(x_out, u, gate, gate_layout, gate_act, weight_post, weight_pre)
    D, rdt = shape[-1], x_out.dtype
    dt = u.dtype if u is not None else d_h.dtype if d_h is not None else rdt
    code = _code(dt)
    if d_x_out is not None:
        _expect("d_x_out", d_x_out, shape, rdt, index)
    if (d_h is None) != (weight_pre is None):
        raise ValueError("d_h and weight_pre: both or neither")
    if d_h is not None:
        _expect("d_h", d_h, shape, dt, index)
    d_x = _buffer("d_x", d_x, x_out, shape, rdt, index)
    if u is not None:
        d_u = _buffer("d_u", d_u, u, shape, dt, index)
    elif d_u is not None:
        raise ValueError("d_u: there is none without u")
    if gate is not None and want_d_gate:
        d_gate = _buffer("d_gate", d_gate, gate, gate.shape, gate.dtype, index)
    elif d_gate is not None:
        raise ValueError("d_gate: there is none without a gate, or with want_d_gate=False")
    d_post = torch.empty_like(weight_post) if want_d_weights and weight_post is not None else None
    d_pre = torch.empty_like(weight_pre) if want_d_weights and weight_pre is not None else None
    sums = d_post is not None or d_pre is not None or (d_gate is not None and layout == 1)
    workspace, ws_bytes = _workspace(workspace, gdn2_block_norm_bwd_workspace_bytes(rows, D) if sums else 0, x_out)
    _run("gdn2_block_norm_bwd", index, x_out.data_ptr(), _addr(u), _addr(gate), _addr(weight_post), _addr(weight_pre),
         _addr(d_x_out), _addr(d_h), d_x.data_ptr(), _addr(d_u), _addr(d_gate), _addr(d_post), _addr(d_pre), rows, D,
         eps, residual_scale, layout, act, dropout_p, *_random(seed, offset, offset_device, index), code,
         _code(rdt), _addr(workspace), ws_bytes)
    return {"d_x": d_x, "d_u": d_u, "d_gate": d_gate, "d_weight_post": d_post, "d_weight_pre": d_pre}


@_on_stream
def gdn2_dropout(x, p, seed, offset=0, *, offset_device=None, out=None):
    """Counter-based dropout of x ([..., D] float32 or bfloat16): the mask comes
    from (seed, offset) and each element's position and is never stored; the
    gradient is the same call on the gradient.  p is rounded to a multiple of
    2^-16; kept elements are divided by 1 - p.  offset_device: [1] int64 on the
    device, added to offset when the kernel runs (replayed graphs), or None.
    ``out`` may be x (in place)."""
    shape, index, dt = x.shape, x.get_device(), x.dtype
    rows = _rows("x", x, shape)
    out = _buffer("out", out, x, shape, dt, index)
    _run("gdn2_dropout", index, x.data_ptr(), out.data_ptr(), rows, shape[-1], p,
         *_random(seed, offset, offset_device, index), _code(dt))
    return out


@functools.lru_cache(maxsize=256)
def gdn2_mixer_epilogue_bwd_workspace_bytes(rows, dv) -> int:
    return int(load().gdn2_mixer_epilogue_bwd_workspace_bytes(rows, dv))


@_on_stream
def gdn2_mixer_epilogue_bwd(o, gate, weight, d_y, *, eps=1e-5, act="sigmoid", want_d_weight=True, workspace=None):
    """Gradients of gdn2_mixer_epilogue for the loss <d_y, y>: dict(d_o, d_gate,
    d_weight), d_weight None when not wanted.  ``workspace`` (uint8) is
    allocated when not given."""
    shape, index, dt = o.shape, o.get_device(), o.dtype
    rows = _rows("o", o, shape)
    dv, code = shape[-1], _code(dt)
    _expect("gate", gate, shape, dt, index)
    _expect("weight", weight, shape[-1:], torch.float32, index)
    _expect("d_y", d_y, shape, dt, index)
    if act not in GATE_ACTS:
        raise ValueError(f"act must be one of {tuple(GATE_ACTS)}")
    d_o, d_gate = torch.empty_like(o), torch.empty_like(o)
    d_weight = torch.empty_like(weight) if want_d_weight else None
    workspace, ws_bytes = _workspace(workspace, gdn2_mixer_epilogue_bwd_workspace_bytes(rows, dv) if want_d_weight else 0,
                                     o)
    _run("gdn2_mixer_epilogue_bwd", index, o.data_ptr(), gate.data_ptr(), weight.data_ptr(), d_y.data_ptr(),
         d_o.data_ptr(), d_gate.data_ptr(), _addr(d_weight), rows, dv, eps, GATE_ACTS[act], code, _addr(workspace),
         ws_bytes)
    return {"d_o": d_o, "d_gate": d_gate, "d_weight": d_weight}


@functools.lru_cache(maxsize=256)
def gdn2_mixer_prologue_bwd_workspace_bytes(B, T, H, dk, dv, kernel_size) -> int:
    return int(load().gdn2_mixer_prologue_bwd_workspace_bytes(B, T, H, dk, dv, kernel_size))


@_on_stream
def gdn2_mixer_prologue_bwd(xq, xk, xv, conv_q, conv_k, conv_v, b_logit, w_logit, d_q, d_k, d_v, d_b, d_w, *,
                            conv_state=None, d_conv_state_out=None, output_d_conv_state=False, cu_seqlens=None,
                            q_scale=1.0, eps_l2=1e-6, want_d_conv=True, workspace=None):
    """Gradients of gdn2_mixer_prologue for the loss <d_q, q> + <d_k, k> + <d_v, v>
    + <d_b, b> + <d_w, w> + <d_conv_state_out, final convolution state>.

    The inputs are the forward call's (conv_state: its initial state or None);
    d_q, d_k, d_b: [B, T, H, dk] and d_v, d_w: [B, T, H, dv] of the inputs' type;
    d_conv_state_out: [N, H * (2 dk + dv), K - 1] float32 or None.  Returns
    dict(d_xq, d_xk, d_xv, d_conv_q, d_conv_k, d_conv_v, d_b_logit, d_w_logit,
    d_conv_state), None in the place of what is not wanted.  Packed input may be
    longer than its sequences: tokens that none of them owns are not read, and
    their gradients are zero.  ``workspace`` (uint8) is allocated when not given.
    """
    key, value, index, dt = xq.shape, xv.shape, xq.get_device(), xq.dtype
    if len(key) != 4 or len(value) != 4:
        raise ValueError(f"xq, xk, xv: [B, T, H, d] (got {tuple(key)}, {tuple(value)})")
    B, T, H, dk = key
    dv, K, code = value[3], conv_q.shape[-1], _code(dt)
    N = B if cu_seqlens is None else cu_seqlens.shape[0] - 1
    for want, tensors in ((key, (xq, xk, b_logit, d_q, d_k, d_b)), ((B, T, H, dv), (xv, w_logit, d_v, d_w))):
        for t in tensors:
            if not (t.shape == want and t.dtype is dt and t.get_device() == index and t.is_contiguous()):
                name = next(n for n, v in dict(xq=xq, xk=xk, b_logit=b_logit, d_q=d_q, d_k=d_k, d_b=d_b, xv=xv,
                                               w_logit=w_logit, d_v=d_v, d_w=d_w).items() if v is t)
                _expect(name, t, want, dt, index)
    for name, t, width in (("conv_q", conv_q, dk), ("conv_k", conv_k, dk), ("conv_v", conv_v, dv)):
        _expect(name, t, (H * width, K), torch.float32, index)
    st_shape = (N, H * (2 * dk + dv), K - 1)
    for name, t in (("conv_state", conv_state), ("d_conv_state_out", d_conv_state_out)):
        if t is not None:
            _expect(name, t, st_shape, torch.float32, index)
    if cu_seqlens is not None:
        _expect("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, index)
    new = torch.empty_like
    out = {"d_xq": new(xq), "d_xk": new(xk), "d_xv": new(xv),
           "d_conv_q": new(conv_q) if want_d_conv else None, "d_conv_k": new(conv_k) if want_d_conv else None,
           "d_conv_v": new(conv_v) if want_d_conv else None, "d_b_logit": new(b_logit), "d_w_logit": new(w_logit)}
    out["d_conv_state"] = conv_q.new_empty(st_shape) if output_d_conv_state else None
    need = gdn2_mixer_prologue_bwd_workspace_bytes(B, T, H, dk, dv, K) if want_d_conv else 0
    workspace, ws_bytes = _workspace(workspace, need, xq)
    _run("gdn2_mixer_prologue_bwd_zeroed", index, xq.data_ptr(), xk.data_ptr(), xv.data_ptr(), conv_q.data_ptr(),
         conv_k.data_ptr(), conv_v.data_ptr(), b_logit.data_ptr(), w_logit.data_ptr(), _addr(conv_state),
         d_q.data_ptr(), d_k.data_ptr(), d_v.data_ptr(), d_b.data_ptr(), d_w.data_ptr(), _addr(d_conv_state_out),
         *[_addr(t) for t in out.values()], _addr(cu_seqlens), B, T, H, dk, dv, K, N, q_scale, eps_l2, code,
         _addr(workspace), ws_bytes)
    return out


# --- linear attention with a fixed decay for each head -----------------------


def _four(name, t):
    if len(t.shape) != 4:
        raise ValueError(f"{name}: [B, T, H, d] (got {tuple(t.shape)})")
    return t.shape


def gdn2_linear_attn_fwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code) -> int:
    return int(load().gdn2_linear_attn_fwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code))


def gdn2_linear_attn_bwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code) -> int:
    return int(load().gdn2_linear_attn_bwd_workspace_bytes(B, T, H, dk, dv, num_seqs, dtype_code))


@functools.lru_cache(maxsize=512)
def _linear_workspace(name, device, *sizes):
    """The query's answer on a device: the plan goes by its compute units."""
    return int(getattr(_LIB, name)(*sizes))


@_on_stream
def gdn2_linear_attn_fwd(q, k, v, alpha, initial_state=None, *, output_final_state=True, final_state=None, out=None,
                         cu_seqlens=None, segmented=True, workspace=None):
    """Linear attention with a fixed decay for each head over whole sequences:
    S_t = alpha S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.  Returns ``(o, final_state)``
    (final_state None if not wanted).

    q, k: [B, T, H, dk]; v: [B, T, H, dv] (float32 or bfloat16, all the same);
    alpha: [H] float32, a constant of the layer; initial_state: [N, H, dk, dv]
    float32 or None; cu_seqlens: int32 [N + 1] on the device or None (then B must
    be 1).  ``final_state`` may be passed (the initial_state tensor itself for an
    in-place update).  Tokens that no packed sequence owns are not read: their
    rows are zero in a new output, and stay as they were in a given ``out``.
    ``segmented=False`` walks each sequence in one piece (no workspace);
    ``workspace`` (uint8, of at least gdn2_linear_attn_fwd_workspace_bytes of this
    call's sizes, which smaller calls may exceed) is allocated when not given.
    """
    B, T, H, dk = _four("q", q)
    dv, dt, index = _four("v", v)[3], q.dtype, q.get_device()
    code = _code(dt)
    N = B if cu_seqlens is None else cu_seqlens.shape[0] - 1
    _expect("q", q, q.shape, dt, index)
    _expect("k", k, q.shape, dt, index)
    _expect("v", v, (B, T, H, dv), dt, index)
    _expect("alpha", alpha, (H,), torch.float32, index)
    st_shape = (N, H, dk, dv)
    if initial_state is not None:
        _expect("initial_state", initial_state, st_shape, torch.float32, index)
    if cu_seqlens is not None:
        _expect("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, index)
    new = out is None
    out = _buffer("out", out, v, v.shape, dt, index)
    if final_state is not None:
        _expect("final_state", final_state, st_shape, torch.float32, index)
    elif output_final_state:
        final_state = alpha.new_empty(st_shape)
    packed = N if cu_seqlens is not None else 0
    need = _linear_workspace("gdn2_linear_attn_fwd_workspace_bytes", index, B, T, H, dk, dv, packed, code) if segmented else 0
    workspace, ws_bytes = _workspace(workspace, need, q)
    _run("gdn2_linear_attn_fwd", index, q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), _addr(initial_state),
         _addr(final_state), out.data_ptr(), _addr(cu_seqlens), B, T, H, dk, dv, packed, new, code, _addr(workspace),
         ws_bytes)
    return out, final_state


@_on_stream
def gdn2_linear_attn_bwd(q, k, v, alpha, d_o, *, initial_state=None, d_final_state=None, output_d_initial_state=False,
                         cu_seqlens=None, segmented=True, workspace=None):
    """Gradients of gdn2_linear_attn_fwd for the loss <d_o, o> + <d_final_state,
    final_state>: dict(dq, dk, dv, d_initial_state), the last None when not
    wanted.  The inputs are the forward call's; d_o: like its o; d_final_state:
    [N, H, dk, dv] float32 or None for zero.  alpha has no gradient.  Gradients
    of tokens that no packed sequence owns are zero.  ``segmented`` and
    ``workspace`` as in the forward call.
    """
    B, T, H, dk = _four("q", q)
    dv, dt, index = _four("v", v)[3], q.dtype, q.get_device()
    code = _code(dt)
    N = B if cu_seqlens is None else cu_seqlens.shape[0] - 1
    _expect("q", q, q.shape, dt, index)
    _expect("k", k, q.shape, dt, index)
    _expect("v", v, (B, T, H, dv), dt, index)
    _expect("d_o", d_o, v.shape, dt, index)
    _expect("alpha", alpha, (H,), torch.float32, index)
    st_shape = (N, H, dk, dv)
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            _expect(name, t, st_shape, torch.float32, index)
    if cu_seqlens is not None:
        _expect("cu_seqlens", cu_seqlens, (N + 1,), torch.int32, index)
    new = torch.empty_like
    out = {"dq": new(q), "dk": new(k), "dv": new(v),
           "d_initial_state": alpha.new_empty(st_shape) if output_d_initial_state else None}
    packed = N if cu_seqlens is not None else 0
    need = _linear_workspace("gdn2_linear_attn_bwd_workspace_bytes", index, B, T, H, dk, dv, packed, code) if segmented else 0
    workspace, ws_bytes = _workspace(workspace, need, q)
    _run("gdn2_linear_attn_bwd", index, q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), _addr(initial_state),
         d_o.data_ptr(), _addr(d_final_state), *[_addr(t) for t in out.values()], _addr(cu_seqlens), B, T, H, dk, dv,
         packed, True, code, _addr(workspace), ws_bytes)
    return out


@_on_stream
def gdn2_linear_attn_step(q, k, v, alpha, state, *, out=None):
    """One decode step of the same layer; updates ``state`` in place, returns o.

    q, k: [N, H, dk]; v: [N, H, dv]; alpha: [H] float32; state: [N, H, dk, dv]
    float32."""
    if len(q.shape) != 3 or len(v.shape) != 3:
        raise ValueError(f"q, v: [N, H, d] (got {tuple(q.shape)}, {tuple(v.shape)})")
    (N, H, dk), dv, dt, index = q.shape, v.shape[2], q.dtype, q.get_device()
    _expect("q", q, q.shape, dt, index)
    _expect("k", k, q.shape, dt, index)
    _expect("v", v, (N, H, dv), dt, index)
    _expect("alpha", alpha, (H,), torch.float32, index)
    _expect("state", state, (N, H, dk, dv), torch.float32, index)
    out = _buffer("out", out, v, v.shape, dt, index)
    _run("gdn2_linear_attn_step", index, q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), state.data_ptr(),
         out.data_ptr(), N, H, dk, dv, _code(dt))
    return out


def _qk_inputs(q, k, inv_freq, positions, weight_q, weight_k):
    """Checks what the two directions of the q, k norm and rotation share;
    returns its sizes, type and device index."""
    (B, T, Hq, d), dt, index = _four("q", q), q.dtype, q.get_device()
    Hk = _four("k", k)[2]
    _expect("q", q, q.shape, dt, index)
    _expect("k", k, (B, T, Hk, d), dt, index)
    if weight_q is not None:
        _expect("weight_q", weight_q, (d,), torch.float32, index)
    if weight_k is not None:
        _expect("weight_k", weight_k, (d,), torch.float32, index)
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _expect("inv_freq", inv_freq, (rot // 2,), torch.float32, index)
        if not rot:
            inv_freq = None
    if positions is not None:
        _expect("positions", positions, (B, T), torch.int32, index)
    return B, T, Hq, Hk, d, rot, _code(dt), index, _addr(inv_freq)


@_on_stream
def gdn2_qk_norm_rope(q, k, inv_freq=None, *, positions=None, weight_q=None, weight_k=None, q_scale=1.0, eps=1e-6,
                      interleaved=False, q_out=None, k_out=None):
    """Queries and keys normalised for each head and rotated by their position:
    returns ``(q_out, k_out)``.

        n = x / sqrt(mean(x^2) + eps) * weight         (over a head's d channels)
        y = scale * rotate(n, position)                (scale: q_scale for q, 1 for k)

    q: [B, T, Hq, d], k: [B, T, Hk, d] (float32 or bfloat16); weight_q, weight_k:
    [d] float32 or None (ones); inv_freq: [rot / 2] float32, the rotation's
    frequency for each pair, or None (no rotation); positions: [B, T] int32 or
    None (the token's index in its row).  Pairs are channels (i, i + rot / 2), or
    (2 i, 2 i + 1) with ``interleaved``; channels from rot on are not turned.
    q_out may be q and k_out may be k (in place); they are allocated when not
    given.
    """
    B, T, Hq, Hk, d, rot, code, index, freq = _qk_inputs(q, k, inv_freq, positions, weight_q, weight_k)
    q_out = _buffer("q_out", q_out, q, q.shape, q.dtype, index)
    k_out = _buffer("k_out", k_out, k, k.shape, k.dtype, index)
    _run("gdn2_qk_norm_rope", index, q.data_ptr(), k.data_ptr(), _addr(weight_q), _addr(weight_k), freq, _addr(positions),
         q_out.data_ptr(), k_out.data_ptr(), B, T, Hq, Hk, d, rot, interleaved, q_scale, eps, code)
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d) -> int:
    return int(load().gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d))


@_on_stream
def gdn2_qk_norm_rope_bwd(q, k, d_q_out, d_k_out, inv_freq=None, *, positions=None, weight_q=None, weight_k=None,
                          q_scale=1.0, eps=1e-6, interleaved=False, want_d_weights=True, workspace=None):
    """Gradients of gdn2_qk_norm_rope for the loss <d_q_out, q_out> + <d_k_out,
    k_out>: dict(d_q, d_k, d_weight_q, d_weight_k), None in the place of what has
    no weight or is not wanted.  q and k are the forward call's inputs (not its
    outputs).  ``workspace`` (uint8) is allocated when not given."""
    B, T, Hq, Hk, d, rot, code, index, freq = _qk_inputs(q, k, inv_freq, positions, weight_q, weight_k)
    _expect("d_q_out", d_q_out, q.shape, q.dtype, index)
    _expect("d_k_out", d_k_out, k.shape, k.dtype, index)
    d_q, d_k = torch.empty_like(q), torch.empty_like(k)
    dw_q = torch.empty_like(weight_q) if want_d_weights and weight_q is not None else None
    dw_k = torch.empty_like(weight_k) if want_d_weights and weight_k is not None else None
    need = gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d) if dw_q is not None or dw_k is not None else 0
    workspace, ws_bytes = _workspace(workspace, need, q)
    _run("gdn2_qk_norm_rope_bwd", index, q.data_ptr(), k.data_ptr(), _addr(weight_q), _addr(weight_k), freq,
         _addr(positions), d_q_out.data_ptr(), d_k_out.data_ptr(), d_q.data_ptr(), d_k.data_ptr(), _addr(dw_q),
         _addr(dw_k), B, T, Hq, Hk, d, rot, interleaved, q_scale, eps, code, _addr(workspace), ws_bytes)
    return {"d_q": d_q, "d_k": d_k, "d_weight_q": dw_q, "d_weight_k": dw_k}
