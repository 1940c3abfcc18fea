"""Thin ctypes binding of libfadkv (include/fadkv.h), for torch tensors on the GPU.

Argument marshalling only: shapes and dtypes are checked, device pointers and torch's current
HIP stream are passed to the C functions of the same names, and a negative status raises
FadkvError.  Every step of the coder runs in the library's HIP kernels; there is no fallback.
The library is loaded on first use (after torch, so that it binds to torch's HIP runtime) and
a missing library raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import os
from dataclasses import dataclass
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfadkv.so")

FADKV_OK = 0
FADKV_F32, FADKV_F16, FADKV_BF16 = 0, 1, 2
FADKV_SELECT_GM, FADKV_SELECT_PL = 0, 1
FLAG_TRIGGER, FLAG_REPLACED, FLAG_EXHAUSTED, FLAG_NONFINITE = 0x01, 0x02, 0x04, 0x08

_DT = {torch.float32: FADKV_F32, torch.float16: FADKV_F16, torch.bfloat16: FADKV_BF16}
_TORCH_DT = {v: k for k, v in _DT.items()}
_SELECT = {"gm": FADKV_SELECT_GM, "pl": FADKV_SELECT_PL}


class FadkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed with status {status}: {fadkv_status_string(status)}")
        self.status = status


class fadkv_dict(ctypes.Structure):
    _fields_ = [("num_dicts", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("atoms", ctypes.c_void_p), ("usage", ctypes.c_void_p)]


class fadkv_params(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("s", ctypes.c_int32), ("ridge_abs", ctypes.c_float),
                ("ridge_rel", ctypes.c_float), ("delta_key", ctypes.c_float),
                ("delta_value", ctypes.c_float), ("tau_c", ctypes.c_uint32),
                ("select", ctypes.c_int32)]


class fadkv_codes(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("coef", ctypes.c_void_p), ("relerr", ctypes.c_void_p),
                ("flags", ctypes.c_void_p)]


class fadkv_pages(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class fadkv_qkv(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("freqs", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float)]


_lib_handle = None


def lib() -> ctypes.CDLL:
    """The loaded libfadkv.so (raises if it has not been built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_dictionary_coding_amd.build`")
        h = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        h.fadkv_abi_version.restype = ctypes.c_int
        h.fadkv_status_string.restype = ctypes.c_char_p
        h.fadkv_status_string.argtypes = [ctypes.c_int]
        h.fadkv_workspace_bytes.restype = ctypes.c_int
        h.fadkv_workspace_bytes.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_int64,
                                            P(ctypes.c_size_t)]
        h.fadkv_encode.restype = ctypes.c_int
        h.fadkv_encode.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_void_p, ctypes.c_int64,
                                   P(fadkv_codes), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        h.fadkv_encode_noalloc.restype = ctypes.c_int
        h.fadkv_encode_noalloc.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_void_p,
                                           ctypes.c_int64, P(fadkv_codes), ctypes.c_void_p]
        h.fadkv_screen.restype = ctypes.c_int
        h.fadkv_screen.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_void_p, ctypes.c_int64,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p]
        h.fadkv_select_support.restype = ctypes.c_int
        h.fadkv_select_support.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, P(fadkv_codes), ctypes.c_void_p]
        h.fadkv_adapt.restype = ctypes.c_int
        h.fadkv_adapt.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_void_p, ctypes.c_int64,
                                  P(fadkv_codes), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                  ctypes.c_void_p]
        h.fadkv_reconstruct.restype = ctypes.c_int
        h.fadkv_reconstruct.argtypes = [P(fadkv_dict), ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int32, ctypes.c_void_p]
        h.fadkv_adapt_append.restype = ctypes.c_int
        h.fadkv_adapt_append.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_void_p,
                                         ctypes.c_int64, P(fadkv_codes), ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]
        h.fadkv_omp_workspace_bytes.restype = ctypes.c_int
        h.fadkv_omp_workspace_bytes.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_int64,
                                                P(ctypes.c_size_t)]
        h.fadkv_encode_omp.restype = ctypes.c_int
        h.fadkv_encode_omp.argtypes = [P(fadkv_dict), P(fadkv_params), ctypes.c_void_p,
                                       ctypes.c_int64, P(fadkv_codes), ctypes.c_void_p,
                                       ctypes.c_size_t, ctypes.c_void_p]
        h.fadkv_attend_workspace_bytes.restype = ctypes.c_int
        h.fadkv_attend_workspace_bytes.argtypes = [P(fadkv_dict), ctypes.c_int64, ctypes.c_int32,
                                                   P(ctypes.c_size_t)]
        h.fadkv_attend.restype = ctypes.c_int
        h.fadkv_attend.argtypes = [P(fadkv_dict), ctypes.c_int32, ctypes.c_int32,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                   ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]
        i32, i64, ptr, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        h.fadkv_pages_workspace_bytes.restype = ctypes.c_int
        h.fadkv_pages_workspace_bytes.argtypes = [i64, P(size)]
        h.fadkv_pages_advance.restype = ctypes.c_int
        h.fadkv_pages_advance.argtypes = [i32, i32, i64, i32] + [ptr] * 5 + [i64] + [ptr] * 7 + [
            size, ptr]
        h.fadkv_rope_freqs.restype = ctypes.c_int
        h.fadkv_rope_freqs.argtypes = [i32, ctypes.c_double, i32] + [ctypes.c_double] * 4 + [
            P(ctypes.c_double), P(ctypes.c_double)]
        h.fadkv_norm_rope.restype = ctypes.c_int
        h.fadkv_norm_rope.argtypes = [P(fadkv_qkv), ptr, P(fadkv_pages), ptr, ptr, ptr, ptr]
        h.fadkv_attend_paged_workspace_bytes.restype = ctypes.c_int
        h.fadkv_attend_paged_workspace_bytes.argtypes = [P(fadkv_pages), i64, i32, i32, P(size)]
        h.fadkv_attend_paged.restype = ctypes.c_int
        h.fadkv_attend_paged.argtypes = [P(fadkv_pages), ptr, i32, ptr, i64, ptr, i32,
                                         ctypes.c_float, i32, i32, i32, ptr, ptr, size, ptr]
        h.fadkv_attend_prompt_workspace_bytes.restype = ctypes.c_int
        h.fadkv_attend_prompt_workspace_bytes.argtypes = [P(fadkv_pages), i64, i64, i32, i32,
                                                          P(size)]
        h.fadkv_attend_prompt.restype = ctypes.c_int
        h.fadkv_attend_prompt.argtypes = [P(fadkv_pages), ptr, i32, ptr, ptr, i64, ptr, i64, i32,
                                          ctypes.c_float, i32, i32, i32, ptr, ptr, size, ptr]
        _lib_handle = h
    return _lib_handle


def fadkv_status_string(status: int) -> str:
    return lib().fadkv_status_string(int(status)).decode()


def fadkv_abi_version() -> int:
    return int(lib().fadkv_abi_version())


@dataclass(frozen=True)
class Params:
    """fadkv_params (defaults: Table 5, 3B/4B column)."""

    n: int = 256
    s: int = 8
    ridge_abs: float = 1e-4
    ridge_rel: float = 0.20
    delta_key: float = 0.50
    delta_value: float = 0.70
    tau_c: int = 1
    select: str = "gm"

    def c(self) -> fadkv_params:
        return fadkv_params(self.n, self.s, self.ridge_abs, self.ridge_rel, self.delta_key,
                            self.delta_value, self.tau_c, _SELECT[self.select])


@dataclass
class Codes:
    idx: torch.Tensor      # int32 [num_dicts][M][s]
    coef: torch.Tensor     # float32 [num_dicts][M][s]
    relerr: torch.Tensor   # float32 [num_dicts][M]
    flags: torch.Tensor    # uint8 [num_dicts][M]

    @staticmethod
    def empty(num_dicts: int, M: int, s: int, device) -> "Codes":
        return Codes(torch.empty(num_dicts, M, s, dtype=torch.int32, device=device),
                     torch.empty(num_dicts, M, s, dtype=torch.float32, device=device),
                     torch.empty(num_dicts, M, dtype=torch.float32, device=device),
                     torch.empty(num_dicts, M, dtype=torch.uint8, device=device))

    def c(self) -> fadkv_codes:
        return fadkv_codes(self.idx.data_ptr(), self.coef.data_ptr(), self.relerr.data_ptr(),
                           self.flags.data_ptr())


def _check(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dict(atoms: torch.Tensor, usage: Optional[torch.Tensor] = None) -> fadkv_dict:
    _check(atoms, "atoms")
    if atoms.dim() != 3 or atoms.dtype not in _DT:
        raise ValueError("atoms must be [num_dicts][N][d] float32/float16/bfloat16")
    T, N, d = atoms.shape
    if usage is not None:
        _check(usage, "usage", torch.int32, (T, N))
    return fadkv_dict(T, N, d, _DT[atoms.dtype], atoms.data_ptr(),
                      usage.data_ptr() if usage is not None else None)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def fadkv_workspace_bytes(atoms: torch.Tensor, params: Params, M: int) -> int:
    T, N, d = atoms.shape
    dd = fadkv_dict(T, N, d, _DT[atoms.dtype], None, None)
    out = ctypes.c_size_t(0)
    st = lib().fadkv_workspace_bytes(ctypes.byref(dd), ctypes.byref(params.c()), int(M),
                                     ctypes.byref(out))
    if st != FADKV_OK:
        raise FadkvError("fadkv_workspace_bytes", st)
    return int(out.value)


def make_workspace(atoms: torch.Tensor, params: Params, M: int) -> torch.Tensor:
    return torch.empty(max(1, fadkv_workspace_bytes(atoms, params, M)), dtype=torch.uint8,
                       device=atoms.device)


def fadkv_encode(atoms: torch.Tensor, X: torch.Tensor, params: Params,
                 out: Optional[Codes] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Codes:
    """Encode X[t][m] against atoms[t]; returns (or fills) the codes."""
    dd = _dict(atoms)
    T, N, d = atoms.shape
    _check(X, "X", atoms.dtype)
    if X.dim() != 3 or X.shape[0] != T or X.shape[2] != d:
        raise ValueError(f"X must be [{T}][M][{d}]")
    M = X.shape[1]
    if out is None:
        out = Codes.empty(T, M, params.s, atoms.device)
    if workspace is None:
        workspace = make_workspace(atoms, params, M)
    st = lib().fadkv_encode(ctypes.byref(dd), ctypes.byref(params.c()), X.data_ptr(), M,
                            ctypes.byref(out.c()), workspace.data_ptr(), workspace.numel(),
                            _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_encode", st)
    return out


NOALLOC_SCRATCH_BYTES = 128 << 20    # FADKV_NOALLOC_SCRATCH_BYTES
FADKV_ERR_SCRATCH = -6


def fadkv_encode_noalloc(atoms: torch.Tensor, X: torch.Tensor, params: Params,
                         out: Optional[Codes] = None, stream=None) -> Codes:
    """fadkv_encode with the library's static per-GPU scratch instead of a workspace (for
    callers that cannot allocate); `out` is the caller's, allocated here only when not given.
    Calls that overlap on one GPU race on that scratch."""
    dd = _dict(atoms)
    T, N, d = atoms.shape
    _check(X, "X", atoms.dtype)
    if X.dim() != 3 or X.shape[0] != T or X.shape[2] != d:
        raise ValueError(f"X must be [{T}][M][{d}]")
    M = X.shape[1]
    if out is None:
        out = Codes.empty(T, M, params.s, atoms.device)
    st = lib().fadkv_encode_noalloc(ctypes.byref(dd), ctypes.byref(params.c()), X.data_ptr(), M,
                                    ctypes.byref(out.c()), _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_encode_noalloc", st)
    return out


@dataclass
class Pool:
    idx: torch.Tensor      # int16 storage of uint16 atom indices [num_dicts][M][n]
    score: torch.Tensor    # float32 [num_dicts][M][n]
    status: torch.Tensor   # uint8 [num_dicts][M]: 0 encoded, 1 zero vector, 2 non-finite

    @staticmethod
    def empty(num_dicts: int, M: int, n: int, device) -> "Pool":
        return Pool(torch.empty(num_dicts, M, n, dtype=torch.int16, device=device),
                    torch.empty(num_dicts, M, n, dtype=torch.float32, device=device),
                    torch.empty(num_dicts, M, dtype=torch.uint8, device=device))

    def atom_indices(self) -> torch.Tensor:
        """Pool indices as int64 (the uint16 values)."""
        return self.idx.to(torch.int64) & 0xFFFF


def fadkv_screen(atoms: torch.Tensor, X: torch.Tensor, params: Params,
                 out: Optional[Pool] = None, stream=None) -> Pool:
    """Scores and Top-n pool of every vector (first stage of fadkv_encode)."""
    dd = _dict(atoms)
    T, N, d = atoms.shape
    _check(X, "X", atoms.dtype)
    M = X.shape[1]
    if out is None:
        out = Pool.empty(T, M, params.n, atoms.device)
    st = lib().fadkv_screen(ctypes.byref(dd), ctypes.byref(params.c()), X.data_ptr(), M,
                            out.idx.data_ptr(), out.score.data_ptr(), out.status.data_ptr(),
                            _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_screen", st)
    return out


def fadkv_select_support(atoms: torch.Tensor, X: torch.Tensor, params: Params, pool: Pool,
                         out: Optional[Codes] = None, stream=None) -> Codes:
    """Support, ridge coefficients and residual from a screened pool (second stage)."""
    dd = _dict(atoms)
    T, N, d = atoms.shape
    _check(X, "X", atoms.dtype)
    M = X.shape[1]
    if out is None:
        out = Codes.empty(T, M, params.s, atoms.device)
    st = lib().fadkv_select_support(ctypes.byref(dd), ctypes.byref(params.c()), X.data_ptr(), M,
                                    pool.idx.data_ptr(), pool.score.data_ptr(),
                                    pool.status.data_ptr(), ctypes.byref(out.c()), _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_select_support", st)
    return out


def fadkv_adapt(atoms: torch.Tensor, usage: torch.Tensor, X: torch.Tensor, codes: Codes,
                params: Params, replaced: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Commit this step's codes and overwrite inactive atoms in place; returns `replaced`."""
    dd = _dict(atoms, usage)
    T, N, d = atoms.shape
    _check(X, "X", atoms.dtype)
    M = X.shape[1]
    if replaced is None:
        replaced = torch.empty(T, M, dtype=torch.int32, device=atoms.device)
    if workspace is None:
        workspace = make_workspace(atoms, params, M)
    st = lib().fadkv_adapt(ctypes.byref(dd), ctypes.byref(params.c()), X.data_ptr(), M,
                           ctypes.byref(codes.c()), replaced.data_ptr(), workspace.data_ptr(),
                           workspace.numel(), _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_adapt", st)
    return replaced


def fadkv_reconstruct(atoms: torch.Tensor, idx: torch.Tensor, coef: torch.Tensor,
                      out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    dd = _dict(atoms)
    T, N, d = atoms.shape
    _check(idx, "idx", torch.int32)
    _check(coef, "coef", torch.float32, idx.shape)
    M, s = idx.shape[1], idx.shape[2]
    if out is None:
        out = torch.empty(T, M, d, dtype=out_dtype or atoms.dtype, device=atoms.device)
    _check(out, "out", None, (T, M, d))
    st = lib().fadkv_reconstruct(ctypes.byref(dd), idx.data_ptr(), coef.data_ptr(), s, M,
                                 out.data_ptr(), _DT[out.dtype], _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_reconstruct", st)
    return out


def fadkv_attend_workspace_bytes(atoms: torch.Tensor, R: int, G: int) -> int:
    T, N, d = atoms.shape
    dd = fadkv_dict(T, N, d, _DT[atoms.dtype], None, None)
    out = ctypes.c_size_t(0)
    st = lib().fadkv_attend_workspace_bytes(ctypes.byref(dd), int(R), int(G), ctypes.byref(out))
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_workspace_bytes", st)
    return int(out.value)


def fadkv_attend(atoms: torch.Tensor, layer: int, k_idx: torch.Tensor, k_coef: torch.Tensor,
                 v_idx: torch.Tensor, v_coef: torch.Tensor, lens: torch.Tensor, q: torch.Tensor,
                 scale: float, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention of q [R][G][d] over the sparse-coded keys/values of `layer` (codes
    [R][T][s], lens [R]); returns (or fills) out [R][G][d] fp32."""
    dd = _dict(atoms)
    _check(k_idx, "k_idx", torch.int32)
    R, T, s = k_idx.shape
    _check(k_coef, "k_coef", torch.float32, (R, T, s))
    _check(v_idx, "v_idx", torch.int32, (R, T, s))
    _check(v_coef, "v_coef", torch.float32, (R, T, s))
    _check(lens, "lens", torch.int32, (R,))
    _check(q, "q", atoms.dtype)
    if q.dim() != 3 or q.shape[0] != R or q.shape[2] != atoms.shape[2]:
        raise ValueError(f"q must be [{R}][G][{atoms.shape[2]}]")
    G = q.shape[1]
    if out is None:
        out = torch.empty(R, G, atoms.shape[2], dtype=torch.float32, device=atoms.device)
    _check(out, "out", torch.float32, (R, G, atoms.shape[2]))
    if workspace is None:
        workspace = torch.empty(max(1, fadkv_attend_workspace_bytes(atoms, R, G)),
                                dtype=torch.uint8, device=atoms.device)
    st = lib().fadkv_attend(ctypes.byref(dd), int(layer), int(s), k_idx.data_ptr(),
                            k_coef.data_ptr(), v_idx.data_ptr(), v_coef.data_ptr(),
                            lens.data_ptr(), int(R), int(T), q.data_ptr(), int(G), float(scale),
                            out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                            _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend", st)
    return out


def fadkv_adapt_append(atoms: torch.Tensor, usage: torch.Tensor, X: torch.Tensor, codes: Codes,
                       params: Params, n_atoms: torch.Tensor,
                       replaced: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Append-only growth commit: atoms [num_dicts][capacity][d] with n_atoms [num_dicts]
    (int32, advanced in place) slots in use.  Returns replaced [num_dicts][M]."""
    dd = _dict(atoms, usage)
    T, N, d = atoms.shape
    _check(X, "X", atoms.dtype)
    M = X.shape[1]
    _check(n_atoms, "n_atoms", torch.int32, (T,))
    if replaced is None:
        replaced = torch.empty(T, M, dtype=torch.int32, device=atoms.device)
    _check(replaced, "replaced", torch.int32, (T, M))
    if workspace is None:
        workspace = make_workspace(atoms, params, M)
    st = lib().fadkv_adapt_append(ctypes.byref(dd), ctypes.byref(params.c()), X.data_ptr(), M,
                                  ctypes.byref(codes.c()), replaced.data_ptr(), n_atoms.data_ptr(),
                                  workspace.data_ptr(), workspace.numel(), _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_adapt_append", st)
    return replaced


def fadkv_omp_workspace_bytes(atoms: torch.Tensor, params: Params, M: int) -> int:
    T, N, d = atoms.shape
    dd = fadkv_dict(T, N, d, _DT[atoms.dtype], None, None)
    out = ctypes.c_size_t(0)
    st = lib().fadkv_omp_workspace_bytes(ctypes.byref(dd), ctypes.byref(params.c()), int(M),
                                         ctypes.byref(out))
    if st != FADKV_OK:
        raise FadkvError("fadkv_omp_workspace_bytes", st)
    return out.value


def fadkv_encode_omp(atoms: torch.Tensor, X: torch.Tensor, params: Params,
                     out: Optional[Codes] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> Codes:
    """Full-dictionary greedy yardstick (every atom a candidate); codes as fadkv_encode."""
    dd = _dict(atoms, None)
    T, N, d = atoms.shape
    _check(X, "X", atoms.dtype)
    M = X.shape[1]
    if out is None:
        out = Codes.empty(T, M, params.s, atoms.device)
    if workspace is None:
        workspace = torch.empty(max(1, fadkv_omp_workspace_bytes(atoms, params, M)),
                                dtype=torch.uint8, device=atoms.device)
    st = lib().fadkv_encode_omp(ctypes.byref(dd), ctypes.byref(params.c()), X.data_ptr(), M,
                                ctypes.byref(out.c()), workspace.data_ptr(), workspace.numel(),
                                _stream(stream))
    if st != FADKV_OK:
        raise FadkvError("fadkv_encode_omp", st)
    return out


# ---- the dense cache beside the codes ---------------------------------------------------------
# A decode step calls these once per layer and their kernels take a few microseconds, so the
# checks are written to cost little: one chain of comparisons per tensor, the messages apart.
ROW_OK, ROW_REFUSED, ROW_RELEASED = 0, 1, 2    # FADKV_ROW_*
ROPE_PLAIN, ROPE_LINEAR, ROPE_BANDS, ROPE_YARN = 0, 1, 2, 3
_ROPE = {"plain": ROPE_PLAIN, "linear": ROPE_LINEAR, "bands": ROPE_BANDS, "yarn": ROPE_YARN}
_I32 = torch.int32


def _int32(x) -> int:
    """x for an int32 argument: ctypes would cut 2^32 + 3 down to 3, so what is beyond the type
    becomes its end, which a length or a window means anyway or the call refuses."""
    if type(x) is int and -1 <= x <= 0x7fffffff:
        return x
    x = operator.index(x)
    return max(-1, min(x, 0x7fffffff))


def _refuse(t, name: str, dtype, shape, dev: int):
    """Raises what is wrong with the tensor, if anything is."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name} must live on cuda:{dev}, got {t.device}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient: this call has no backward pass "
                         "(detach it or use torch.no_grad())")


def _ptr(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on this device, of which no gradient
    is expected (the calls have no backward pass)."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and
                not t.requires_grad and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:   # no tensor
        pass
    _refuse(t, name, dtype, shape, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must live on the GPU")
    return dev


@contextlib.contextmanager
def _on(dev: int, stream):
    """`dev` and the caller's stream (torch's current one of `dev` if none) made current: what a
    call allocates then belongs to the stream that uses it."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        if stream.device.index != dev:
            raise ValueError(f"the stream must be one of cuda:{dev}")
        with torch.cuda.stream(stream):
            yield


# torch's current device and the handle of its current stream, without what torch.cuda's functions
# of these names do around them (current_stream() alone takes 2.8 us)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _elsewhere(dev: int, stream) -> bool:
    return stream is not None or dev != _current_device()


@dataclass(frozen=True)
class Pages:
    """One layer's dense cache: k and v [num_pages][kv_heads][page_size][d]."""

    k: torch.Tensor
    v: torch.Tensor

    def __post_init__(self):
        dev = _device_of(self.k, "pages.k")
        if self.k.dim() != 4 or self.k.dtype not in _DT:
            raise ValueError("pages must be [num_pages][kv_heads][page_size][d] "
                             "float32/float16/bfloat16")
        _ptr(self.k, "pages.k", self.k.dtype, self.k.shape, dev)
        _ptr(self.v, "pages.v", self.k.dtype, self.k.shape, dev)

    @staticmethod
    def empty(num_pages: int, kv_heads: int, page_size: int, d: int, dtype, device) -> "Pages":
        shape = (num_pages, kv_heads, page_size, d)
        return Pages(torch.empty(shape, dtype=dtype, device=device),
                     torch.empty(shape, dtype=dtype, device=device))

    @property
    def page_size(self) -> int:
        return self.k.shape[2]

    def c(self) -> fadkv_pages:
        n, h, p, d = self.k.shape
        return fadkv_pages(n, p, h, d, _DT[self.k.dtype], self.k.data_ptr(), self.v.data_ptr())


@dataclass(frozen=True)
class PageTable:
    """Which pages hold the rows of a batch, and which are free (fadkv_pages_advance)."""

    table: torch.Tensor        # int32 [R][max_pages]
    lens: torch.Tensor         # int32 [R]
    ring: torch.Tensor         # int32 [num_pages]
    ring_state: torch.Tensor   # int32 [2]: first free entry of ring, free entries
    page_size: int

    def __post_init__(self):
        dev = _device_of(self.table, "table")
        if self.table.dim() != 2:
            raise ValueError("table must be [R][max_pages]")
        _ptr(self.table, "table", _I32, self.table.shape, dev)
        _ptr(self.lens, "lens", _I32, self.table.shape[:1], dev)
        _ptr(self.ring, "ring", _I32, (self.ring.numel(),), dev)
        _ptr(self.ring_state, "ring_state", _I32, (2,), dev)

    @staticmethod
    def empty(rows: int, max_pages: int, num_pages: int, page_size: int, device) -> "PageTable":
        """No row holds a token; every page is free."""
        return PageTable(torch.full((rows, max_pages), -1, dtype=_I32, device=device),
                         torch.zeros(rows, dtype=_I32, device=device),
                         torch.arange(num_pages, dtype=_I32, device=device),
                         torch.tensor([0, num_pages], dtype=_I32, device=device), page_size)


@dataclass(frozen=True)
class PageStep:
    """What fadkv_pages_advance writes.  lens and ring_state may be those of the PageTable."""

    lens: torch.Tensor         # int32 [R]
    ring_state: torch.Tensor   # int32 [2]
    cu: torch.Tensor           # int32 [R + 1]
    status: torch.Tensor       # int32 [R]: ROW_*
    slots: torch.Tensor        # int32 [max_tokens]
    positions: torch.Tensor    # int32 [max_tokens]
    workspace: torch.Tensor    # uint8

    def __post_init__(self):
        dev = _device_of(self.lens, "lens")
        R = self.lens.numel()
        _ptr(self.lens, "lens", _I32, (R,), dev)
        _ptr(self.ring_state, "ring_state", _I32, (2,), dev)
        _ptr(self.cu, "cu", _I32, (R + 1,), dev)
        _ptr(self.status, "status", _I32, (R,), dev)
        _ptr(self.slots, "slots", _I32, (self.slots.numel(),), dev)
        _ptr(self.positions, "positions", _I32, self.slots.shape, dev)
        _ptr(self.workspace, "workspace", torch.uint8, self.workspace.shape, dev)

    @staticmethod
    def empty(pt: PageTable, max_tokens: int, in_place: bool = False) -> "PageStep":
        """Buffers for steps of up to max_tokens new tokens; in_place: the table's own lengths and
        ring state are advanced (a captured step that is replayed), else new ones are written."""
        R, dev = pt.lens.shape[0], pt.lens.device
        out = ctypes.c_size_t(0)
        st = lib().fadkv_pages_workspace_bytes(R, ctypes.byref(out))
        if st != FADKV_OK:
            raise FadkvError("fadkv_pages_workspace_bytes", st)

        def i32(n):
            return torch.empty(n, dtype=_I32, device=dev)
        return PageStep(pt.lens if in_place else i32(R), pt.ring_state if in_place else i32(2),
                        i32(R + 1), i32(R), i32(max_tokens), i32(max_tokens),
                        torch.empty(max(1, out.value), dtype=torch.uint8, device=dev))


def fadkv_pages_advance(pt: PageTable, new_lens: torch.Tensor, max_tokens: Optional[int] = None,
                        out: Optional[PageStep] = None, stream=None) -> PageStep:
    """One step of the bookkeeping: rows add new_lens [R] tokens (negative: the row has ended).
    pt.table and pt.ring are updated in place; give `out` (or the most tokens of a step)."""
    dev = pt.table.get_device()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return fadkv_pages_advance(pt, new_lens, max_tokens, out)
    R, max_pages = pt.table.shape
    new = _ptr(new_lens, "new_lens", _I32, (R,), dev)
    if out is None:
        if max_tokens is None:
            raise ValueError("give out or max_tokens")
        out = PageStep.empty(pt, max_tokens)
    tokens = out.slots.shape[0]
    if max_tokens is not None and max_tokens != tokens:
        raise ValueError(f"out holds {tokens} tokens, not {max_tokens}")
    if out.lens.shape[0] != R or out.lens.get_device() != dev:
        raise ValueError(f"out must be for {R} rows on cuda:{dev}")
    st = lib().fadkv_pages_advance(
        pt.ring.shape[0], _int32(pt.page_size), R, max_pages, new, pt.lens.data_ptr(),
        pt.table.data_ptr(), pt.ring.data_ptr(), pt.ring_state.data_ptr(), tokens,
        out.lens.data_ptr(), out.ring_state.data_ptr(), out.cu.data_ptr(), out.status.data_ptr(),
        out.slots.data_ptr(), out.positions.data_ptr(), out.workspace.data_ptr(),
        out.workspace.numel(), _raw_stream(dev))
    if st != FADKV_OK:
        raise FadkvError("fadkv_pages_advance", st)
    return out


def fadkv_rope_freqs(rot_dim: int, base: float, kind: str = "plain", factor: float = 1.0,
                     low: float = 1.0, high: Optional[float] = None, original_len: float = 8192,
                     device="cuda"):
    """(freqs, mscale) of fadkv_norm_rope: float64 [rot_dim / 2] on `device`, and a float.
    kind: plain, linear, bands (high defaults to 4) or yarn (32)."""
    if high is None:
        high = 32.0 if kind == "yarn" else 4.0
    if kind not in _ROPE:
        raise ValueError(f"kind must be one of {', '.join(_ROPE)}, got {kind!r}")
    rot_dim = _int32(int(rot_dim))
    host = torch.empty(max(0, min(rot_dim, 65536)) // 2, dtype=torch.float64)
    buf = (ctypes.c_double * max(1, host.numel()))()
    mscale = ctypes.c_double(1.0)
    st = lib().fadkv_rope_freqs(rot_dim, float(base), _ROPE[kind], float(factor), float(low),
                                float(high), float(original_len), buf, ctypes.byref(mscale))
    if st != FADKV_OK:
        raise FadkvError("fadkv_rope_freqs", st)
    host.copy_(torch.tensor(buf[:host.numel()], dtype=torch.float64))
    return host.to(device), mscale.value


def _heads(t: torch.Tensor, name: str, dtype, n: int, h: int, d: int, dev: int) -> int:
    """Checks [n][h][d] whose heads lie together; returns the elements between tokens."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != (n, h, d) or
            t.get_device() != dev or t.requires_grad):
        _refuse(t, name, dtype, (n, h, d), dev)
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and s1 != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s0 if n > 1 else h * d


def fadkv_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                    freqs: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                    k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                    interleaved: bool = False, mscale: float = 1.0,
                    pages: Optional[Pages] = None, slots: Optional[torch.Tensor] = None,
                    q_out: Optional[torch.Tensor] = None, k_rows: Optional[torch.Tensor] = None,
                    v_rows: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Norm (where a weight is given) and rotation of q [n][heads][d] and k [n][kv_heads][d],
    which may be views of one projection's output; keys and values also go to `slots` of `pages`
    and to k_rows, v_rows [kv_heads][n][d] (rows of the encoder).  Returns (or fills) q_out."""
    dev = _device_of(q, "q")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return fadkv_norm_rope(q, k, v, positions, freqs, q_weight, k_weight, eps, interleaved,
                                   mscale, pages, slots, q_out, k_rows, v_rows)
    dt = q.dtype
    if q.dim() != 3 or dt not in _DT:
        raise ValueError("q must be [n][heads][d] float32/float16/bfloat16")
    n, heads, d = q.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError(f"k must be [{n}][kv_heads][{d}]")
    kv = k.shape[1]
    qs = _heads(q, "q", dt, n, heads, d, dev)
    ks = _heads(k, "k", dt, n, kv, d, dev)
    vs = _heads(v, "v", dt, n, kv, d, dev)
    pos = _ptr(positions, "positions", _I32, (n,), dev)
    rot, fr = 0, None
    if freqs is not None:
        _device_of(freqs, "freqs")
        rot = 2 * freqs.numel()
        fr = _ptr(freqs, "freqs", torch.float64, (rot // 2,), dev) if rot else None
    qw = None if q_weight is None else _ptr(q_weight, "q_weight", dt, (d,), dev)
    kw = None if k_weight is None else _ptr(k_weight, "k_weight", dt, (d,), dev)
    kr = None if k_rows is None else _ptr(k_rows, "k_rows", dt, (kv, n, d), dev)
    vr = None if v_rows is None else _ptr(v_rows, "v_rows", dt, (kv, n, d), dev)
    if (pages is None) != (slots is None):
        raise ValueError("pages and slots go together")
    pg = sl = None
    if pages is not None:
        if pages.k.get_device() != dev:
            raise ValueError(f"pages must live on cuda:{dev}")
        pg, sl = ctypes.byref(pages.c()), _ptr(slots, "slots", _I32, (n,), dev)
    if q_out is None:
        q_out = torch.empty(n, heads, d, dtype=dt, device=q.device)
    qo = _ptr(q_out, "q_out", dt, (n, heads, d), dev)
    a = fadkv_qkv(n, heads, kv, d, _DT[dt], q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
                  pos, qw, kw, eps, fr, rot, interleaved, mscale)
    st = lib().fadkv_norm_rope(ctypes.byref(a), qo, pg, sl, kr, vr, _raw_stream(dev))
    if st != FADKV_OK:
        raise FadkvError("fadkv_norm_rope", st)
    return q_out


def fadkv_attend_paged_workspace_bytes(pages: Pages, R: int, heads: int, max_len: int) -> int:
    out = ctypes.c_size_t(0)
    st = lib().fadkv_attend_paged_workspace_bytes(ctypes.byref(pages.c()), int(R), _int32(heads),
                                                  _int32(max_len), ctypes.byref(out))
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_paged_workspace_bytes", st)
    return int(out.value)


def _attend_args(pages, table, lens, q, out, dev):
    """Checks what both attention calls take; returns (pages struct, addresses, out, shapes)."""
    p = pages.c()
    dt = pages.k.dtype
    _device_of(table, "table")
    if q.dim() != 3 or table.dim() != 2:
        raise ValueError("q must be [..][heads][d] and table [R][max_pages]")
    n, heads = q.shape[0], q.shape[1]
    R, max_pages = table.shape
    if pages.k.get_device() != dev:
        raise ValueError(f"pages must live on cuda:{dev}")
    qp = _ptr(q, "q", dt, (n, heads, p.d), dev)
    tp = _ptr(table, "table", _I32, (R, max_pages), dev)
    lp = _ptr(lens, "lens", _I32, (R,), dev)
    if out is None:
        out = torch.empty_like(q)
    op = _ptr(out, "out", dt, (n, heads, p.d), dev)
    return p, qp, tp, lp, op, out, n, heads, R, max_pages


def fadkv_attend_paged(pages: Pages, table: torch.Tensor, lens: torch.Tensor, q: torch.Tensor,
                       scale: float, window: int = 0, sinks: int = 0,
                       max_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one new token per row, q [R][heads][d], over lens [R] cached tokens (its own
    included) in the pages of table [R][max_pages]; window > 0: only the last `window` tokens and
    the first `sinks` are visible.  Returns (or fills) out [R][heads][d]."""
    dev = _device_of(q, "q")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return fadkv_attend_paged(pages, table, lens, q, scale, window, sinks, max_len, out,
                                      workspace)
    p, qp, tp, lp, op, out, n, heads, R, max_pages = _attend_args(pages, table, lens, q, out, dev)
    if n != R:
        raise ValueError(f"q must have {R} rows, got {n}")
    if max_len is None:
        max_len = max_pages * p.page_size
    if workspace is None:
        need = fadkv_attend_paged_workspace_bytes(pages, R, heads, max_len)
        workspace = torch.empty(max(1, need), dtype=torch.uint8, device=q.device)
    ws = _ptr(workspace, "workspace", torch.uint8, workspace.shape, dev)
    st = lib().fadkv_attend_paged(ctypes.byref(p), tp, max_pages, lp, R, qp, heads, scale,
                                  _int32(window), _int32(sinks), _int32(max_len), op, ws, workspace.numel(), _raw_stream(dev))
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_paged", st)
    return out


def fadkv_attend_prompt_workspace_bytes(pages: Pages, R: int, n: int, heads: int,
                                        max_len: int) -> int:
    out = ctypes.c_size_t(0)
    st = lib().fadkv_attend_prompt_workspace_bytes(ctypes.byref(pages.c()), int(R), int(n),
                                                   _int32(heads), _int32(max_len),
                                                   ctypes.byref(out))
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_prompt_workspace_bytes", st)
    return int(out.value)


def fadkv_attend_prompt(pages: Pages, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                        q: torch.Tensor, scale: float, window: int = 0, sinks: int = 0,
                        max_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of packed tokens q [n][heads][d]: tokens cu[r] .. cu[r+1] - 1 are the last
    of row r's lens[r] cached ones.  Returns (or fills) out [n][heads][d]; rows of out behind the
    last token stay as they were (undefined where out is allocated here)."""
    dev = _device_of(q, "q")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return fadkv_attend_prompt(pages, table, lens, cu, q, scale, window, sinks, max_len,
                                       out, workspace)
    p, qp, tp, lp, op, out, n, heads, R, max_pages = _attend_args(pages, table, lens, q, out, dev)
    cp = _ptr(cu, "cu", _I32, (R + 1,), dev)
    if max_len is None:
        max_len = max_pages * p.page_size
    if workspace is None:
        need = fadkv_attend_prompt_workspace_bytes(pages, R, n, heads, max_len)
        ws = None
        if need:   # held until the call has launched: another thread could be given it
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        ws, need = _ptr(workspace, "workspace", torch.uint8, workspace.shape, dev), workspace.numel()
    st = lib().fadkv_attend_prompt(ctypes.byref(p), tp, max_pages, lp, cp, R, qp, n, heads, scale,
                                   _int32(window), _int32(sinks), _int32(max_len), op, ws, need,
                                   _raw_stream(dev))
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_prompt", st)
    return out
