"""Thin ctypes binding over libdomino (declared in ``include/domino.h``).

Argument marshalling only: every step of the head runs in the library's CUDA kernels.  PyTorch
provides device memory and the current stream.  If ``libdomino.so`` is missing or cannot be
loaded, every call raises -- there is no CPU fallback.

Names follow the C ABI without the ``domino_`` prefix: ``draft_greedy``, ``teacher_forced``,
``accept_len``, ``top_logits``, ``beam_select``, ``distill``, ``workspace_bytes``,
``accept_workspace_bytes``, ``status_string``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdomino.so")

OK = 0
ERR_INVALID_ARGUMENT = -1
ERR_UNSUPPORTED = -2
ERR_CUDA = -3
ERR_WORKSPACE = -4
ERR_SCRATCH_LIMIT = -5
NOALLOC_SCRATCH_BYTES = 1024 * 1024
STATUS_DEVICE_TIMEOUT = 1
STATUS_BAD_TOKEN = 2

DTYPE_F32 = 0
DTYPE_BF16 = 1
_TORCH_DTYPE = {DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16}

EXPORTS = ("domino_workspace_bytes", "domino_draft_greedy", "domino_teacher_forced",
           "domino_accept_workspace_bytes", "domino_accept_len", "domino_status_string",
           "domino_abi_version", "domino_debug_set_spin_limit", "domino_launch_count",
           "domino_greedy_plan", "domino_teacher_forced_plan", "domino_draft_greedy_noalloc", "domino_debug_set_trace",
           "domino_embed_proj_bytes", "domino_project_embeddings", "domino_arena_bytes",
           "domino_pack_weights", "domino_set_l2_persistence", "domino_debug_gemm",
           "domino_debug_read_passes", "domino_teacher_forced_ex", "domino_accept_sample_workspace_bytes",
           "domino_accept_sample", "domino_top_logits", "domino_beam_workspace_bytes", "domino_beam_select",
           "domino_distill", "domino_distill_backward")


class DominoError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "L", "d", "Hs", "r", "V", "dtype")]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("embed", "W_ih", "W_hh", "b_ih", "b_hh", "W1", "W2", "embed_proj")]


class BeamArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "W_in", "W_out", "V")] + [("ld", ctypes.c_int64)] +
                [(n, ctypes.c_int32) for n in ("dtype", "eos", "Hs", "hist_len", "pos")] +
                [(n, ctypes.c_void_p) for n in ("logits", "scores", "finished", "states", "history", "scores_out",
                                                "parents_out", "tokens_out", "finished_out", "states_out",
                                                "history_out")])


class DistillArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("V", ctypes.c_int32), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("K", ctypes.c_int32), ("logits", ctypes.c_void_p), ("top_ids", ctypes.c_void_p),
                ("top_logits", ctypes.c_void_p), ("teacher_lse", ctypes.c_void_p), ("row_weights", ctypes.c_void_p),
                ("temperature", ctypes.c_float)]


_lib = None


def lib(path: str = LIB_PATH) -> ctypes.CDLL:
    """Open libdomino once; raise if it is absent (no fallback path exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libdomino not built ({path} missing): run python -m draft_block_causal_b200.build")
        L = ctypes.CDLL(path)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        L.domino_workspace_bytes.argtypes = [ctypes.POINTER(Shape)]
        L.domino_workspace_bytes.restype = sz
        L.domino_draft_greedy.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, vp, vp, vp, vp, vp,
                                          vp, sz, vp, vp]
        L.domino_draft_greedy.restype = ctypes.c_int
        L.domino_teacher_forced.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, vp, vp, vp, vp, vp,
                                            vp, sz, vp, vp]
        L.domino_teacher_forced.restype = ctypes.c_int
        L.domino_accept_workspace_bytes.argtypes = [i32, i32]
        L.domino_accept_workspace_bytes.restype = sz
        L.domino_accept_len.argtypes = [i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]
        L.domino_accept_len.restype = ctypes.c_int
        L.domino_status_string.argtypes = [ctypes.c_int]
        L.domino_status_string.restype = ctypes.c_char_p
        L.domino_abi_version.argtypes = []
        L.domino_abi_version.restype = i32
        L.domino_debug_set_spin_limit.argtypes = [ctypes.c_uint64]
        L.domino_debug_set_spin_limit.restype = ctypes.c_int
        L.domino_launch_count.argtypes = []
        L.domino_launch_count.restype = ctypes.c_uint64
        L.domino_draft_greedy_noalloc.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, vp, vp, vp,
                                                  vp, vp, vp, vp]
        L.domino_draft_greedy_noalloc.restype = ctypes.c_int
        L.domino_embed_proj_bytes.argtypes = [ctypes.POINTER(Shape)]
        L.domino_embed_proj_bytes.restype = sz
        L.domino_project_embeddings.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, vp, vp]
        L.domino_project_embeddings.restype = ctypes.c_int
        L.domino_debug_set_trace.argtypes = [vp, i32]
        L.domino_debug_set_trace.restype = ctypes.c_int
        L.domino_greedy_plan.argtypes = [ctypes.POINTER(Shape)]
        L.domino_greedy_plan.restype = ctypes.c_char_p
        L.domino_teacher_forced_plan.argtypes = [ctypes.POINTER(Shape)]
        L.domino_teacher_forced_plan.restype = ctypes.c_char_p
        L.domino_arena_bytes.argtypes = [ctypes.POINTER(Shape)]
        L.domino_arena_bytes.restype = sz
        L.domino_pack_weights.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, sz,
                                          ctypes.POINTER(Weights), vp]
        L.domino_pack_weights.restype = ctypes.c_int
        L.domino_set_l2_persistence.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, ctypes.c_float]
        L.domino_set_l2_persistence.restype = ctypes.c_int
        L.domino_debug_gemm.argtypes = [vp, vp, i32, i32, i32, i32, vp, ctypes.c_int64, i32, i32, i32, vp, vp]
        L.domino_debug_gemm.restype = ctypes.c_int
        L.domino_teacher_forced_ex.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(Weights), vp, vp, vp, vp, vp,
                                               i32, vp, vp, sz, vp, vp]
        L.domino_teacher_forced_ex.restype = ctypes.c_int
        L.domino_debug_read_passes.argtypes = [vp, sz, i32, vp]
        L.domino_debug_read_passes.restype = ctypes.c_int
        L.domino_accept_sample_workspace_bytes.argtypes = [i32, i32, i32]
        L.domino_accept_sample_workspace_bytes.restype = sz
        L.domino_accept_sample.argtypes = [i32, i32, i32, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, sz, vp, vp]
        L.domino_accept_sample.restype = ctypes.c_int
        L.domino_top_logits.argtypes = [i32, i32, ctypes.c_int64, i32, vp, i32, ctypes.c_float, vp, vp, vp, vp]
        L.domino_top_logits.restype = ctypes.c_int
        L.domino_beam_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.domino_beam_workspace_bytes.restype = sz
        L.domino_beam_select.argtypes = [ctypes.POINTER(BeamArgs), vp, sz, vp]
        L.domino_beam_select.restype = ctypes.c_int
        L.domino_distill.argtypes = [ctypes.POINTER(DistillArgs), vp, vp, vp, ctypes.c_int64, i32, vp, vp]
        L.domino_distill.restype = ctypes.c_int
        L.domino_distill_backward.argtypes = [ctypes.POINTER(DistillArgs), vp, vp, vp, ctypes.c_int64, i32, vp, vp]
        L.domino_distill_backward.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().domino_status_string(int(code)).decode()


def abi_version() -> int:
    return int(lib().domino_abi_version())


def launch_count() -> int:
    """Kernels the library has enqueued in this process so far."""
    return int(lib().domino_launch_count())


def greedy_plan(shape: Shape) -> str:
    """Which kernels draft_greedy runs for this shape."""
    return lib().domino_greedy_plan(ctypes.byref(shape)).decode()


def teacher_forced_plan(shape: Shape) -> str:
    """Which kernels teacher_forced runs for this shape (weights without the projection table)."""
    return lib().domino_teacher_forced_plan(ctypes.byref(shape)).decode()


def set_trace(buf) -> None:
    """Profiling hook: a CUDA int64 tensor receives SM-clock stamps of the fused kernel's phases
    (CTA 0); None turns it off.  Layout in include/domino.h (domino_debug_set_trace)."""
    if buf is None:
        _check(lib().domino_debug_set_trace(None, 0), "domino_debug_set_trace")
    else:
        _check(lib().domino_debug_set_trace(ctypes.c_void_p(buf.data_ptr()), buf.numel()), "domino_debug_set_trace")


def set_spin_limit(limit: int) -> None:
    """Test hook: iteration limit of the library's bounded device waits (0 = default)."""
    lib().domino_debug_set_spin_limit(int(limit))


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise DominoError(rc, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    """The caller's stream (default: the current stream of `device`), which must belong to `device`."""
    if device.type != "cuda":
        raise ValueError(f"the call's tensors must be on a CUDA device, not {device}")
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"stream is on {s.device}, the call's tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


def _launch(device, fn, *args):
    """Call a library entry point with `device` current: the library queries and launches on the
    current device, which must be the one that holds the call's memory."""
    if torch.cuda.current_device() == device.index:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _expect(t, name: str, shape, dtype, device) -> None:
    """The library sees only a pointer: check here that a tensor has the exact shape, dtype,
    contiguity and device the call reads or writes, so that no kernel touches memory outside it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.shape != shape:  # torch.Size compares equal to a tuple of ints
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(int(x) for x in shape)}")
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        dts = dtype if isinstance(dtype, tuple) else (dtype,)
        raise ValueError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dts)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _expect_out(t, name: str, shape, dtype, device) -> None:
    """_expect for a tensor that the call fills.  Autograd is told, as by torch's operations in place: a backward pass
    that has saved the tensor is then refused, where it would compute with what the call left there."""
    _expect(t, name, shape, dtype, device)
    torch._C._increment_version((t,))


def _expect_status(status, device) -> None:
    if status is not None:
        if not isinstance(status, torch.Tensor) or status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError("status must be an int32 tensor with at least one element")
        if status.device != device:
            raise ValueError(f"status is on {status.device}, expected {device}")


def _expect_workspace(ws, device) -> None:
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor (see alloc_workspace)")
    if ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, expected {device}")


@dataclass
class HeadWeights:
    """Device-resident head weights (all one storage type, fp32 or bf16).

    embed [V, d], W_ih [3Hs, d], W_hh [3Hs, Hs], b_ih [3Hs], b_hh [3Hs], W1 [r, d+Hs], W2 [V, r].
    """
    embed: torch.Tensor
    W_ih: torch.Tensor
    W_hh: torch.Tensor
    b_ih: torch.Tensor
    b_hh: torch.Tensor
    W1: torch.Tensor
    W2: torch.Tensor
    embed_proj: "torch.Tensor | None" = None  # [V, 3Hs] fp32 from project_embeddings, optional

    @property
    def dtype_code(self) -> int:
        if self.W2.dtype == torch.float32:
            return DTYPE_F32
        if self.W2.dtype == torch.bfloat16:
            return DTYPE_BF16
        raise TypeError(f"unsupported weight dtype {self.W2.dtype}")

    def dims(self):
        V, d = self.embed.shape
        Hs = self.W_hh.shape[1]
        r = self.W2.shape[1]
        return d, Hs, r, V

    def check(self) -> None:
        """Every weight has the shape the dimensions of embed, W_hh and W2 imply, the storage type
        of W2, and the device of W2."""
        d, Hs, r, V = self.dims()
        dev = self.W2.device
        want = {"embed": (V, d), "W_ih": (3 * Hs, d), "W_hh": (3 * Hs, Hs), "b_ih": (3 * Hs,), "b_hh": (3 * Hs,),
                "W1": (r, d + Hs), "W2": (V, r)}
        for n, shp in want.items():
            _expect(getattr(self, n), f"weight {n}", shp, self.W2.dtype, dev)
        if self.embed_proj is not None:
            _expect(self.embed_proj, "embed_proj", (V, 3 * Hs), torch.float32, dev)

    def __post_init__(self):
        self.check()
        object.__setattr__(self, "_checked", True)

    def __setattr__(self, name, value):
        # a replaced weight is checked against the others at once (every call relies on it); a
        # rejected one leaves the previous value in place
        old = self.__dict__.get(name)
        object.__setattr__(self, name, value)
        if self.__dict__.get("_checked"):
            try:
                self.check()
            except Exception:
                object.__setattr__(self, name, old)
                raise

    def c_struct(self) -> Weights:
        for n in ("embed", "W_ih", "W_hh", "b_ih", "b_hh", "W1", "W2"):
            if not getattr(self, n).is_cuda:
                raise ValueError(f"weight {n} must be a CUDA tensor")
        xp = self.embed_proj
        ptrs = [self.__dict__[n].data_ptr() for n in ("embed", "W_ih", "W_hh", "b_ih", "b_hh", "W1", "W2")]
        return Weights(*ptrs, xp.data_ptr() if xp is not None else None)


def _check_head_inputs(w: HeadWeights, base_logits, hidden, S0):
    """The inputs every head call reads; returns (B, L, device)."""
    d, Hs, r, V = w.dims()
    dev = w.W2.device
    if not isinstance(base_logits, torch.Tensor) or base_logits.dim() != 3:
        raise ValueError("base_logits must be a [B, L, V] tensor")
    B, L = int(base_logits.shape[0]), int(base_logits.shape[1])
    _expect(base_logits, "base_logits", (B, L, V), w.W2.dtype, dev)
    _expect(hidden, "hidden", (B, L, d), w.W2.dtype, dev)
    _expect(S0, "S0", (B, Hs), torch.float32, dev)
    return B, L, dev


def make_shape(w: HeadWeights, B: int, L: int) -> Shape:
    d, Hs, r, V = w.dims()
    return Shape(int(B), int(L), int(d), int(Hs), int(r), int(V), w.dtype_code)


def workspace_bytes(w: HeadWeights, B: int, L: int) -> int:
    n = int(lib().domino_workspace_bytes(ctypes.byref(make_shape(w, B, L))))
    if n == 0:
        raise DominoError(ERR_INVALID_ARGUMENT, "domino_workspace_bytes")
    return n


def project_embeddings(w: HeadWeights, out=None, status=None, stream=None) -> torch.Tensor:
    """The GRU input projection of every embedding row, [V, 3Hs] fp32 (domino_project_embeddings).
    Assign the result to ``w.embed_proj`` to have every entry point gather it per token."""
    d, Hs, r, V = w.dims()
    if out is None:
        out = torch.empty((V, 3 * Hs), dtype=torch.float32, device=w.W2.device)
    _expect(out, "out", (V, 3 * Hs), torch.float32, w.W2.device)
    _expect_status(status, w.W2.device)
    sh = make_shape(w, 1, 1)
    ws = w.c_struct()
    dev = w.W2.device
    rc = _launch(dev, lib().domino_project_embeddings, ctypes.byref(sh), ctypes.byref(ws), _ptr(out), _ptr(status),
                 _stream(stream, dev))
    _check(rc, "domino_project_embeddings")
    return out


def arena_bytes(w: HeadWeights) -> int:
    n = int(lib().domino_arena_bytes(ctypes.byref(make_shape(w, 1, 1))))
    if n == 0:
        raise DominoError(ERR_INVALID_ARGUMENT, "domino_arena_bytes")
    return n


def pack_weights(w: HeadWeights, stream=None) -> HeadWeights:
    """Copy W2, W1, W_hh, W_ih, b_ih, b_hh into one contiguous arena (domino_pack_weights) and return
    HeadWeights whose tensors are views of it (embed and embed_proj are shared with ``w``)."""
    nbytes = arena_bytes(w)
    arena = torch.empty(nbytes, dtype=torch.uint8, device=w.W2.device)
    sh = make_shape(w, 1, 1)
    src = w.c_struct()
    out = Weights()
    rc = _launch(w.W2.device, lib().domino_pack_weights, ctypes.byref(sh), ctypes.byref(src),
                 ctypes.c_void_p(arena.data_ptr()), nbytes, ctypes.byref(out), _stream(stream, w.W2.device))
    _check(rc, "domino_pack_weights")
    dt = w.W2.dtype
    es = torch.empty((), dtype=dt).element_size()

    def view(name):
        t = getattr(w, name)
        off = getattr(out, name) - arena.data_ptr()
        return arena[off:off + t.numel() * es].view(dt).view(t.shape)

    return HeadWeights(embed=w.embed, W_ih=view("W_ih"), W_hh=view("W_hh"), b_ih=view("b_ih"), b_hh=view("b_hh"),
                       W1=view("W1"), W2=view("W2"), embed_proj=w.embed_proj)


def set_l2_persistence(w: HeadWeights, stream, hit_ratio: float = 1.0) -> None:
    """Opt-in L2 residency of packed weights for kernels on ``stream`` (domino_set_l2_persistence);
    ``hit_ratio=0`` clears it and restores the context's persisting-L2 set-aside."""
    sh = make_shape(w, 1, 1)
    ws = w.c_struct()
    rc = _launch(w.W2.device, lib().domino_set_l2_persistence, ctypes.byref(sh), ctypes.byref(ws),
                 _stream(stream, w.W2.device), float(hit_ratio))
    _check(rc, "domino_set_l2_persistence")


def debug_gemm(A, B, out=None, trans=False, a_kwrap=0, bn=0, ks=0, status=None, stream=None) -> torch.Tensor:
    """The tensor-core GEMM engine on its own (domino_debug_gemm): fp32 A[:, k mod K'] . B^T for bf16
    A [M, K'] and B [N, K]; [M, N], or [N, M] when ``trans``.  bn/ks force a plan (0, 0: automatic)."""
    M, N, K = A.shape[0], B.shape[0], B.shape[1]
    _expect(A, "A", (M, int(a_kwrap) or K), torch.bfloat16, A.device)
    _expect(B, "B", (N, K), torch.bfloat16, A.device)
    if out is None:
        out = torch.empty((N, M) if trans else (M, N), dtype=torch.float32, device=A.device)
    _expect(out, "out", (N, M) if trans else (M, N), torch.float32, A.device)
    _expect_status(status, A.device)
    rc = _launch(A.device, lib().domino_debug_gemm, _ptr(A), _ptr(B), M, N, K, int(a_kwrap), _ptr(out), out.shape[1],
                 int(bool(trans)), int(bn), int(ks), _ptr(status), _stream(stream, A.device))
    _check(rc, "domino_debug_gemm")
    return out


def debug_read_passes(buf, passes: int, stream=None) -> None:
    """Re-read a device buffer `passes` times in one launch (domino_debug_read_passes)."""
    rc = _launch(buf.device, lib().domino_debug_read_passes, _ptr(buf), buf.numel() * buf.element_size(), int(passes),
                 _stream(stream, buf.device))
    _check(rc, "domino_debug_read_passes")


def accept_workspace_bytes(B: int, L: int) -> int:
    return int(lib().domino_accept_workspace_bytes(int(B), int(L)))


def alloc_workspace(nbytes: int, device=None) -> torch.Tensor:
    # torch's caching allocator hands out 512-byte aligned blocks
    return torch.empty(int(nbytes), dtype=torch.uint8, device=device or "cuda")


def _check_greedy_outputs(tokens_out, logits_out, states_out, B, L, Hs, V, dev) -> None:
    _expect_out(tokens_out, "tokens_out", (B, L), torch.int32, dev)
    if logits_out is not None:
        _expect_out(logits_out, "logits_out", (B, L, V), torch.float32, dev)
    if states_out is not None:
        _expect_out(states_out, "states_out", (B, L, Hs), torch.float32, dev)


def draft_greedy(w: HeadWeights, base_logits, hidden, S0, tokens_out=None, logits_out=None, states_out=None,
                 workspace=None, status=None, stream=None):
    """Greedy drafting (``domino_draft_greedy``); returns (tokens, logits or None, states or None).

    base_logits [B, L, V] and hidden [B, L, d] in the weights' storage type, S0 [B, Hs] fp32.
    Pass ``logits_out=True`` / ``states_out=True`` to have them allocated, or tensors to fill.
    """
    B, L, dev = _check_head_inputs(w, base_logits, hidden, S0)
    d, Hs, r, V = w.dims()
    if tokens_out is None:
        tokens_out = torch.empty((B, L), dtype=torch.int32, device=dev)
    if logits_out is True:
        logits_out = torch.empty((B, L, V), dtype=torch.float32, device=dev)
    if states_out is True:
        states_out = torch.empty((B, L, Hs), dtype=torch.float32, device=dev)
    if logits_out is False:
        logits_out = None
    if states_out is False:
        states_out = None
    _check_greedy_outputs(tokens_out, logits_out, states_out, B, L, Hs, V, dev)
    _expect_status(status, dev)
    sh = make_shape(w, B, L)
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(w, B, L), dev)
    _expect_workspace(workspace, dev)
    ws = w.c_struct()
    rc = _launch(dev, lib().domino_draft_greedy, ctypes.byref(sh), ctypes.byref(ws), _ptr(base_logits), _ptr(hidden),
                 _ptr(S0), _ptr(tokens_out), _ptr(logits_out), _ptr(states_out), _ptr(workspace), workspace.numel(),
                 _ptr(status), _stream(stream, dev))
    _check(rc, "domino_draft_greedy")
    return tokens_out, logits_out, states_out


def draft_greedy_noalloc(w: HeadWeights, base_logits, hidden, S0, tokens_out=None, logits_out=None,
                         states_out=None, status=None, stream=None):
    """Greedy drafting with no workspace (``domino_draft_greedy_noalloc``).

    For callers that cannot allocate device memory at call time: the scratch is a fixed array
    inside the library (NOALLOC_SCRATCH_BYTES per device).  Calls that overlap on the GPU share
    that array and race -- keep them on one stream.  Pass preallocated output tensors to keep the
    whole call free of allocations; ``logits_out=True`` / ``states_out=True`` allocate them here.
    """
    B, L, dev = _check_head_inputs(w, base_logits, hidden, S0)
    d, Hs, r, V = w.dims()
    if tokens_out is None:
        tokens_out = torch.empty((B, L), dtype=torch.int32, device=dev)
    if logits_out is True:
        logits_out = torch.empty((B, L, V), dtype=torch.float32, device=dev)
    if states_out is True:
        states_out = torch.empty((B, L, Hs), dtype=torch.float32, device=dev)
    logits_out = None if logits_out is False else logits_out
    states_out = None if states_out is False else states_out
    _check_greedy_outputs(tokens_out, logits_out, states_out, B, L, Hs, V, dev)
    _expect_status(status, dev)
    sh = make_shape(w, B, L)
    ws = w.c_struct()
    rc = _launch(dev, lib().domino_draft_greedy_noalloc, ctypes.byref(sh), ctypes.byref(ws), _ptr(base_logits),
                 _ptr(hidden), _ptr(S0), _ptr(tokens_out), _ptr(logits_out), _ptr(states_out), _ptr(status),
                 _stream(stream, dev))
    _check(rc, "domino_draft_greedy_noalloc")
    return tokens_out, logits_out, states_out


def teacher_forced(w: HeadWeights, base_logits, hidden, S0, tokens, logits_out=None, states_out=None,
                   workspace=None, status=None, stream=None, logits_dtype=torch.float32):
    """Teacher-forced logits (``domino_teacher_forced``, or ``domino_teacher_forced_ex`` for bf16
    logits: ``logits_dtype=torch.bfloat16``); returns (logits, states or None)."""
    B, L, dev = _check_head_inputs(w, base_logits, hidden, S0)
    d, Hs, r, V = w.dims()
    _expect(tokens, "tokens", (B, L), torch.int32, dev)
    if logits_out is None:
        logits_out = torch.empty((B, L, V), dtype=logits_dtype, device=dev)
    _expect_out(logits_out, "logits_out", (B, L, V), (torch.float32, torch.bfloat16), dev)
    if states_out is True:
        states_out = torch.empty((B, L, Hs), dtype=torch.float32, device=dev)
    if states_out is False:
        states_out = None
    if states_out is not None:
        _expect_out(states_out, "states_out", (B, L, Hs), torch.float32, dev)
    _expect_status(status, dev)
    sh = make_shape(w, B, L)
    if workspace is None:
        workspace = alloc_workspace(workspace_bytes(w, B, L), dev)
    _expect_workspace(workspace, dev)
    ws = w.c_struct()
    if logits_out.dtype == torch.float32:
        rc = _launch(dev, lib().domino_teacher_forced, ctypes.byref(sh), ctypes.byref(ws), _ptr(base_logits),
                     _ptr(hidden), _ptr(S0), _ptr(tokens), _ptr(logits_out), _ptr(states_out), _ptr(workspace),
                     workspace.numel(), _ptr(status), _stream(stream, dev))
        _check(rc, "domino_teacher_forced")
    else:
        rc = _launch(dev, lib().domino_teacher_forced_ex, ctypes.byref(sh), ctypes.byref(ws), _ptr(base_logits),
                     _ptr(hidden), _ptr(S0), _ptr(tokens), _ptr(logits_out), DTYPE_BF16, _ptr(states_out),
                     _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream, dev))
        _check(rc, "domino_teacher_forced_ex")
    return logits_out, states_out


def accept_len(draft_tokens, target_logits, accept_out=None, workspace=None, status=None, stream=None):
    """Greedy accept length per row (``domino_accept_len``)."""
    if not isinstance(target_logits, torch.Tensor) or target_logits.dim() != 3:
        raise ValueError("target_logits must be a [B, L, V] tensor")
    B, L, V = (int(x) for x in target_logits.shape)
    dev = target_logits.device
    _expect(target_logits, "target_logits", (B, L, V), torch.float32, dev)
    _expect(draft_tokens, "draft_tokens", (B, L), torch.int32, dev)
    if accept_out is None:
        accept_out = torch.empty((B,), dtype=torch.int32, device=dev)
    _expect(accept_out, "accept_out", (B,), torch.int32, dev)
    _expect_status(status, dev)
    if workspace is None:
        workspace = alloc_workspace(accept_workspace_bytes(B, L), dev)
    _expect_workspace(workspace, dev)
    rc = _launch(dev, lib().domino_accept_len, B, L, V, _ptr(draft_tokens), _ptr(target_logits), _ptr(accept_out),
                 _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream, dev))
    _check(rc, "domino_accept_len")
    return accept_out


def accept_sample(draft_tokens, target_logits, temperature: float, uniforms, draft_logits=None, accept_out=None,
                  next_out=None, workspace=None, status=None, stream=None):
    """Sampled verification (``domino_accept_sample``): returns (accept lengths [B], replacement
    tokens [B], -1 where every position was accepted).  ``draft_logits`` None means a greedy draft
    (one-hot draft distribution); ``uniforms`` [B, L + 1] fp32 are the caller's random draws."""
    if not isinstance(target_logits, torch.Tensor) or target_logits.dim() != 3:
        raise ValueError("target_logits must be a [B, L, V] tensor")
    B, L, V = (int(x) for x in target_logits.shape)
    dev = target_logits.device
    _expect(target_logits, "target_logits", (B, L, V), torch.float32, dev)
    if draft_logits is not None:
        _expect(draft_logits, "draft_logits", (B, L, V), torch.float32, dev)
    _expect(draft_tokens, "draft_tokens", (B, L), torch.int32, dev)
    _expect(uniforms, "uniforms", (B, L + 1), torch.float32, dev)
    if accept_out is None:
        accept_out = torch.empty((B,), dtype=torch.int32, device=dev)
    if next_out is None:
        next_out = torch.empty((B,), dtype=torch.int32, device=dev)
    _expect(accept_out, "accept_out", (B,), torch.int32, dev)
    _expect(next_out, "next_out", (B,), torch.int32, dev)
    _expect_status(status, dev)
    if workspace is None:
        n = int(lib().domino_accept_sample_workspace_bytes(B, L, V))
        if n == 0:
            raise DominoError(ERR_INVALID_ARGUMENT, "domino_accept_sample_workspace_bytes")
        workspace = alloc_workspace(n, dev)
    _expect_workspace(workspace, dev)
    rc = _launch(dev, lib().domino_accept_sample, B, L, V, _ptr(draft_tokens), _ptr(draft_logits),
                 _ptr(target_logits), float(temperature), _ptr(uniforms), _ptr(accept_out), _ptr(next_out),
                 _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream, dev))
    _check(rc, "domino_accept_sample")
    return accept_out, next_out


# ---- rows of logits: top logits, beam selection, distillation ----

MAX_TOP = 128
MAX_BEAMS = 32
_DTYPE_CODE = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _logit_rows(t, name: str):
    """(leading shape, V, ld, dtype code) of a [..., V] tensor whose rows lie a fixed multiple of 8 values apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} has dtype {t.dtype}, expected torch.float32 or torch.bfloat16")
    shape = t.shape
    if len(shape) < 2 or 0 in shape:
        raise ValueError(f"{name} must be a [..., V] tensor with at least one row, not {tuple(shape)}")
    V = shape[-1]
    if V % 8 == 0 and t.is_contiguous():
        return shape[:-1], V, V, code
    strides = t.stride()
    ld = run = None
    for n, s in zip(shape[-2::-1], strides[-2::-1]):
        if n == 1:
            continue
        if ld is None:
            ld = run = s
        elif s != run:
            raise ValueError(f"the rows of {name} must lie one fixed stride apart")
        run *= n
    padded = (V + 7) // 8 * 8
    if ld is None:  # a single row
        ld = padded
    if (strides[-1] != 1 and V > 1) or ld < V or ld % 8:
        raise ValueError(f"the rows of {name} must be contiguous and a multiple of 8 values apart (stride {ld}, "
                         f"V {V}): pad the vocabulary's storage")
    if padded != V:
        rows = t.numel() // V
        if (t.storage_offset() + (rows - 1) * ld + padded) * t.element_size() > t.untyped_storage().nbytes():
            raise ValueError(f"the last row of {name} must be followed by storage up to a multiple of 8 values")
    return shape[:-1], V, ld, code


def _new(like, dims, dtype, stream):
    """An uninitialised tensor on the device of ``like``; its memory belongs to the stream that the call uses it on."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return like.new_empty(dims, dtype=dtype)
    if like.dtype is dtype:
        # the cheapest ways to allocate: small calls are as long as their allocations
        return torch.empty_like(like) if like.shape == dims and like.is_contiguous() else like.new_empty(dims)
    return like.new_empty(dims, dtype=dtype)


def _new_rows(like, lead, V: int, stream):
    """An uninitialised [..., V] tensor of the type of ``like`` in rows padded to a multiple of 8 values."""
    if V % 8 == 0:
        return _new(like, lead + (V,), like.dtype, stream)
    return _new(like, lead + ((V + 7) // 8 * 8,), like.dtype, stream)[..., :V]


def _raw_stream(stream, device) -> int:
    """``_stream`` as a plain handle, without the stream object of the current stream."""
    if device.type != "cuda":
        raise ValueError(f"the call's tensors must be on a CUDA device, not {device}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the call's tensors on {device}")
    return stream.cuda_stream


def _data(t):
    return None if t is None else t.data_ptr()


def top_logits(logits, k: int, temperature: float = 1.0, values_out=None, ids_out=None, lse_out=None, stream=None):
    """The k largest of every row of logits [..., V] with their tokens, and the rows' log-sum-exp at ``temperature``
    (``domino_top_logits``): returns (values [..., k] fp32, ids [..., k] int32, lse [...] fp32).  Logits are fp32 or
    bf16; descending, the lower token first among equals; id -1 and value -inf where a row has fewer than k."""
    lead, V, ld, code = _logit_rows(logits, "logits")
    dev, k = logits.device, int(k)
    if not 1 <= k <= MAX_TOP:
        raise ValueError(f"k is {k}, expected 1 to {MAX_TOP}")
    sp = _raw_stream(stream, dev)
    if values_out is None:
        values_out = _new(logits, lead + (k,), torch.float32, stream)
    else:
        _expect_out(values_out, "values_out", lead + (k,), torch.float32, dev)
    if ids_out is None:
        ids_out = _new(logits, lead + (k,), torch.int32, stream)
    else:
        _expect_out(ids_out, "ids_out", lead + (k,), torch.int32, dev)
    if lse_out is None:
        lse_out = _new(values_out, lead, torch.float32, stream)
    else:
        _expect_out(lse_out, "lse_out", lead, torch.float32, dev)
    rc = _launch(dev, lib().domino_top_logits, logits.numel() // V, V, ld, code, logits.data_ptr(), k,
                 float(temperature), values_out.data_ptr(), ids_out.data_ptr(), lse_out.data_ptr(), sp)
    _check(rc, "domino_top_logits")
    return values_out, ids_out, lse_out


def beam_workspace_bytes(B: int, W_in: int, W_out: int, V: int, dtype=torch.float32) -> int:
    """Bytes of workspace that beam_select takes for logits [B, W_in, V] of ``dtype``: 0 for small calls (and for
    sizes that it does not take)."""
    if dtype not in _DTYPE_CODE:
        raise ValueError(f"dtype is {dtype}, expected torch.float32 or torch.bfloat16")
    return int(lib().domino_beam_workspace_bytes(int(B), int(W_in), int(W_out), int(V), _DTYPE_CODE[dtype]))


class BeamStep(NamedTuple):
    """What beam_select returns; ``states``, ``history`` and ``finished`` are None where they do not apply."""
    scores: torch.Tensor              # [B, beams] fp32
    parents: torch.Tensor             # [B, beams] int32
    tokens: torch.Tensor              # [B, beams] int32
    states: Optional[torch.Tensor]    # [B, beams, Hs] fp32
    history: Optional[torch.Tensor]   # [B, beams, hist_len] int32
    finished: Optional[torch.Tensor]  # [B, beams] uint8


def beam_select(logits, scores, beams: int, states=None, history=None, pos: int = 0, finished=None, eos: int = -1,
                out: "BeamStep | None" = None, workspace=None, stream=None) -> BeamStep:
    """One step of beam search (``domino_beam_select``): the ``beams`` best continuations of each group by
    ``scores + log_softmax(logits)``, with states and histories following their parents.

    logits [B, W, V] fp32 or bf16, scores [B, W] fp32 (-inf: a dead beam), states [B, W, Hs] fp32, history
    [B, W, hist_len] int32 (the token goes to column ``pos``), finished [B, W] uint8 with ``eos``.  ``out`` takes a
    BeamStep whose tensors are filled; none of them may share memory with an input."""
    lead, V, ld, code = _logit_rows(logits, "logits")
    if len(lead) != 2:
        raise ValueError("logits must be a [B, W, V] tensor")
    B, W = lead
    dev, n = logits.device, int(beams)
    if not (1 <= n <= MAX_BEAMS and W <= MAX_BEAMS):
        raise ValueError(f"{W} beams to {n}: expected 1 to {MAX_BEAMS}")
    _expect(scores, "scores", (B, W), torch.float32, dev)
    Hs = hist_len = 0
    if states is not None:
        if not isinstance(states, torch.Tensor) or states.dim() != 3:
            raise ValueError("states must be a [B, W, Hs] tensor")
        Hs = states.shape[2]
        _expect(states, "states", (B, W, Hs), torch.float32, dev)
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dim() != 3:
            raise ValueError("history must be a [B, W, hist_len] tensor")
        hist_len = history.shape[2]
        _expect(history, "history", (B, W, hist_len), torch.int32, dev)
    if finished is not None:
        _expect(finished, "finished", (B, W), torch.uint8, dev)
    sp = _raw_stream(stream, dev)
    if out is None:
        out_scores = _new(scores, (B, n), torch.float32, stream)
        parents = _new(scores, (B, n), torch.int32, stream)
        out = BeamStep(out_scores, parents, _new(parents, (B, n), torch.int32, stream),
                       None if states is None else _new(states, (B, n, Hs), torch.float32, stream),
                       None if history is None else _new(history, (B, n, hist_len), torch.int32, stream),
                       None if eos < 0 else _new(scores, (B, n), torch.uint8, stream))
    else:
        _expect_out(out.scores, "out.scores", (B, n), torch.float32, dev)
        _expect_out(out.parents, "out.parents", (B, n), torch.int32, dev)
        _expect_out(out.tokens, "out.tokens", (B, n), torch.int32, dev)
        for name, given, dims, dt in (("states", states, (B, n, Hs), torch.float32),
                                      ("history", history, (B, n, hist_len), torch.int32)):
            t = getattr(out, name)
            if (t is None) != (given is None):
                raise ValueError(f"out.{name} must be given exactly when {name} is")
            if t is not None:
                _expect_out(t, f"out.{name}", dims, dt, dev)
        if out.finished is not None:
            _expect_out(out.finished, "out.finished", (B, n), torch.uint8, dev)
    nbytes = 0
    if workspace is None:
        nbytes = lib().domino_beam_workspace_bytes(B, W, n, V, code)
        if nbytes:
            workspace = _new(scores, (nbytes,), torch.uint8, stream)
    else:
        _expect_workspace(workspace, dev)
        nbytes = workspace.numel()
    a = BeamArgs(B, W, n, V, ld, code, int(eos), Hs, hist_len, int(pos), logits.data_ptr(), scores.data_ptr(),
                 _data(finished), _data(states), _data(history), out.scores.data_ptr(), out.parents.data_ptr(),
                 out.tokens.data_ptr(), _data(out.finished), _data(out.states), _data(out.history))
    rc = _launch(dev, lib().domino_beam_select, ctypes.byref(a), _data(workspace), nbytes, sp)
    _check(rc, "domino_beam_select")
    return out


def _distill_args(logits, top_ids, top_logits, teacher_lse, temperature, row_weights):
    """Checks what every distillation call reads; returns (arguments, leading shape, V)."""
    lead, V, ld, code = _logit_rows(logits, "logits")
    dev = logits.device
    if not isinstance(top_ids, torch.Tensor) or top_ids.dim() != len(lead) + 1:
        raise ValueError("top_ids must be a [..., K] tensor over the rows of logits")
    K = int(top_ids.shape[-1])
    if not 1 <= K <= MAX_TOP:
        raise ValueError(f"{K} entries per row, expected 1 to {MAX_TOP}")
    _expect(top_ids, "top_ids", lead + (K,), torch.int32, dev)
    _expect(top_logits, "top_logits", lead + (K,), torch.float32, dev)
    if teacher_lse is not None:
        _expect(teacher_lse, "teacher_lse", lead, torch.float32, dev)
    if row_weights is not None:
        _expect(row_weights, "row_weights", lead, torch.float32, dev)
    return DistillArgs(logits.numel() // V, V, ld, code, K, logits.data_ptr(), top_ids.data_ptr(),
                       top_logits.data_ptr(), _data(teacher_lse), _data(row_weights), float(temperature)), lead, V


def _expect_grad(grad, lead, V, dev):
    """(ld, dtype code) of a gradient's rows."""
    glead, gV, gld, gcode = _logit_rows(grad, "grad_out")
    if glead != lead or gV != V:
        raise ValueError(f"grad_out has shape {tuple(grad.shape)}, expected {tuple(lead) + (V,)}")
    if grad.device != dev:
        raise ValueError(f"grad_out is on {grad.device}, expected {dev}")
    torch._C._increment_version((grad,))  # as _expect_out
    return gld, gcode


def distill(logits, top_ids, top_logits, teacher_lse=None, temperature: float = 1.0, row_weights=None, grad_out=None,
            loss_out=None, stats_out=None, status=None, stream=None):
    """Distillation loss of every row of logits [..., V] from a teacher's top logits, and optionally its gradient in
    the same call (``domino_distill``): returns (loss [...] fp32, grad or None, stats [..., 8] fp32 or None).

    top_ids [..., K] int32 (-1: no entry) and top_logits [..., K] fp32 are what ``top_logits`` gives of the teacher;
    ``teacher_lse`` [...] fp32 (its third result, at the same temperature) keeps the teacher's remaining mass as one
    class, without it the entries' probabilities are normalised.  ``row_weights`` [...] fp32 scale the rows' losses
    (0: the row is skipped).  ``grad_out``: True for a gradient in the logits' type, or a tensor (fp32 or bf16) to
    fill, which may be ``logits`` itself; it is the gradient of the sum of the losses.  ``stats`` goes to
    ``distill_backward``: made when no gradient is asked for, or with ``stats_out`` (True, or a tensor to fill)."""
    return _distill(logits, top_ids, top_logits, teacher_lse, temperature, row_weights, grad_out, loss_out, stats_out,
                    status, stream)[:3]


def _distill(logits, top_ids, top_logits, teacher_lse, temperature, row_weights, grad_out, loss_out, stats_out, status,
             stream):
    """distill, with the row stride of the logits."""
    a, lead, V = _distill_args(logits, top_ids, top_logits, teacher_lse, temperature, row_weights)
    dev = logits.device
    sp = _raw_stream(stream, dev)
    if grad_out is False:
        grad_out = None
    if loss_out is None:
        loss_out = _new(top_logits, lead, torch.float32, stream)
    else:
        _expect_out(loss_out, "loss_out", lead, torch.float32, dev)
    if stats_out is None and grad_out is None or stats_out is True:
        stats_out = _new(top_logits, lead + (8,), torch.float32, stream)
    elif stats_out is False:
        stats_out = None
    elif stats_out is not None:
        _expect_out(stats_out, "stats_out", lead + (8,), torch.float32, dev)
    _expect_status(status, dev)
    gld = gcode = 0
    if grad_out is not None:
        if grad_out is True:
            grad_out = _new_rows(logits, lead, V, stream)
        gld, gcode = _expect_grad(grad_out, lead, V, dev)
    rc = _launch(dev, lib().domino_distill, ctypes.byref(a), loss_out.data_ptr(), _data(stats_out),
                 _data(grad_out), gld, gcode, _data(status), sp)
    _check(rc, "domino_distill")
    return loss_out, grad_out, stats_out, a.ld


def distill_backward(logits, top_ids, top_logits, stats, grad_loss=None, teacher_lse=None, temperature: float = 1.0,
                     row_weights=None, grad_out=None, status=None, stream=None):
    """The gradient of ``sum(grad_loss * loss)`` with respect to logits from ``distill``'s arguments and stats
    (``domino_distill_backward``); grad_loss [...] fp32, None: ones.  ``grad_out`` as in ``distill``."""
    a, lead, V = _distill_args(logits, top_ids, top_logits, teacher_lse, temperature, row_weights)
    dev = logits.device
    _expect(stats, "stats", lead + (8,), torch.float32, dev)
    if grad_loss is not None:
        _expect(grad_loss, "grad_loss", lead, torch.float32, dev)
    sp = _raw_stream(stream, dev)
    if grad_out is None or grad_out is True:
        grad_out = _new_rows(logits, lead, V, stream)
    gld, gcode = _expect_grad(grad_out, lead, V, dev)
    _expect_status(status, dev)
    rc = _launch(dev, lib().domino_distill_backward, ctypes.byref(a), stats.data_ptr(), _data(grad_loss),
                 grad_out.data_ptr(), gld, gcode, _data(status), sp)
    _check(rc, "domino_distill_backward")
    return grad_out


def _saved(t, name: str, n: int, dtype, device):
    """``t`` that autograd saved, of n values: itself, or an aligned contiguous copy where a saved-tensor hook has laid
    it out anew."""
    if t.dtype is not dtype or t.numel() != n or t.device != device:
        raise ValueError(f"saved {name} came back with {t.numel()} values of {t.dtype} on {t.device}, expected {n} of "
                         f"{dtype} on {device}")
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _saved_rows(logits, strides, ld):
    """``logits`` that autograd saved, in rows as the library takes them, and their row stride: what they had in the
    forward call.  A saved-tensor hook may have laid them out anew (rows without padding); they are copied then."""
    V = logits.shape[-1]
    if logits.stride() == strides and logits.data_ptr() % 16 == 0 and (
            V % 8 == 0 or (logits.storage_offset() + (logits.numel() // V - 1) * ld + (V + 7) // 8 * 8)
            * logits.element_size() <= logits.untyped_storage().nbytes()):
        return logits, ld
    logits = _new_rows(logits, logits.shape[:-1], V, None).copy_(logits)
    return logits, (V + 7) // 8 * 8


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_ids, top_logits, teacher_lse, temperature, row_weights, status):
        loss, _, stats, ld = _distill(logits, top_ids, top_logits, teacher_lse, temperature, row_weights, None, None,
                                      None, status, None)
        ctx.save_for_backward(logits, top_ids, top_logits, stats)  # stats hold what the others are read for
        ctx.given = temperature, logits.shape, logits.stride(), ld, logits.dtype, top_ids.numel()
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        # the arguments were checked in forward; a saved-tensor hook may give them back in another place and layout
        logits, top_ids, top_logits, stats = ctx.saved_tensors
        temperature, shape, strides, ld, dtype, entries = ctx.given
        dev, rows = grad_loss.device, grad_loss.numel()
        if logits.shape != shape or logits.dtype is not dtype or logits.device != dev:
            raise ValueError(f"saved logits came back as {tuple(logits.shape)} of {logits.dtype} on {logits.device}, "
                             f"expected {tuple(shape)} of {dtype} on {dev}")
        logits, ld = _saved_rows(logits, strides, ld)
        top_ids = _saved(top_ids, "top_ids", entries, torch.int32, dev)
        top_logits = _saved(top_logits, "top_logits", entries, torch.float32, dev)
        stats = _saved(stats, "stats", rows * 8, torch.float32, dev)
        if not grad_loss.is_contiguous():
            grad_loss = grad_loss.contiguous()
        V, code = shape[-1], _DTYPE_CODE[dtype]
        grad = _new_rows(logits, shape[:-1], V, None)
        a = DistillArgs(rows, V, ld, code, entries // rows, logits.data_ptr(), top_ids.data_ptr(),
                        top_logits.data_ptr(), None, None, temperature)
        rc = _launch(dev, lib().domino_distill_backward, ctypes.byref(a), stats.data_ptr(), grad_loss.data_ptr(),
                     grad.data_ptr(), (V + 7) // 8 * 8, code, None, _raw_stream(None, dev))
        _check(rc, "domino_distill_backward")
        return grad, None, None, None, None, None, None


def distill_loss(logits, top_ids, top_logits, teacher_lse=None, temperature: float = 1.0, row_weights=None,
                 status=None):
    """``distill``'s loss as a differentiable function of ``logits``, on the current stream: [...] fp32, one per row.
    The teacher's tensors and the row weights are constants: one that requires a gradient is refused.  A call that fills
    the logits or the entries before the backward pass makes that raise, as an operation in place does.  To capture a
    step with its backward pass into a CUDA graph, run it once on the capturing stream first and drop what earlier
    steps of the same leaves have returned: their nodes belong to another stream."""
    for name, t in (("top_logits", top_logits), ("teacher_lse", teacher_lse), ("row_weights", row_weights)):
        if isinstance(t, torch.Tensor) and t.requires_grad:
            raise ValueError(f"{name} requires a gradient, which distill_loss does not give")
    return _DistillLoss.apply(logits, top_ids, top_logits, teacher_lse, float(temperature), row_weights, status)


def to_device_weights(host: dict, dtype_code: int, device="cuda") -> HeadWeights:
    """Move generator arrays (fp32, or bf16 bit patterns in uint16) to device tensors."""
    def cv(a):
        t = torch.from_numpy(a)
        if dtype_code == DTYPE_BF16:
            t = t.view(torch.int16).view(torch.bfloat16) if t.dtype == torch.uint16 else t
        return t.to(device, non_blocking=False).contiguous()
    return HeadWeights(**{k: cv(host[k]) for k in ("embed", "W_ih", "W_hh", "b_ih", "b_hh", "W1", "W2")})


def to_device(a, dtype_code: int, device="cuda") -> torch.Tensor:
    """One generator array to the device; uint16 arrays are bf16 bit patterns."""
    t = torch.from_numpy(a)
    if t.dtype == torch.uint16:
        t = t.view(torch.int16).view(torch.bfloat16)
    return t.to(device).contiguous()
