"""Thin ctypes binding of libfadkv (include/fadkv.h), for torch tensors on the GPU.

Argument marshalling only: shapes and dtypes are checked, device pointers and torch's current
HIP stream are passed to the C functions of the same names, and a negative status raises
FadkvError.  Every step of the coder runs in the library's HIP kernels; there is no fallback.
The library is loaded on first use (after torch, so that it binds to torch's HIP runtime) and
a missing library raises.
"""
from __future__ import annotations

import ctypes
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
        h.fadkv_attend_prompt.restype = ctypes.c_int
        h.fadkv_attend_prompt.argtypes = [P(fadkv_pages), ptr, i32, ptr, ptr, i64, ptr, i64, i32,
                                          ctypes.c_float, i32, i32, ptr, ptr]
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
ROW_OK, ROW_REFUSED, ROW_RELEASED = 0, 1, 2    # FADKV_ROW_*
ROPE_PLAIN, ROPE_LINEAR, ROPE_BANDS, ROPE_YARN = 0, 1, 2, 3
_ROPE = {"plain": ROPE_PLAIN, "linear": ROPE_LINEAR, "bands": ROPE_BANDS, "yarn": ROPE_YARN}


def _inputs(device, **tensors):
    """Every tensor given lies on `device`, and none of them expects a gradient: these calls have
    no backward pass."""
    grad = torch.is_grad_enabled()
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != device:
            raise ValueError(f"{name} must live on {device}, got {t.device}")
        if grad and t.requires_grad:
            raise ValueError(f"{name} requires a gradient: this call has no backward pass "
                             "(detach it or use torch.no_grad())")


class _Launch:
    """The device a call runs on made current, and its stream: torch's current one of that device,
    or the caller's, on which what the call allocates then lives."""

    def __init__(self, device, stream):
        self.device = device
        self.stream = stream
        self.stack = []

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.stack.append(torch.cuda.device(self.device))
            self.stack[-1].__enter__()
        if self.stream is None:
            return torch.cuda.current_stream().cuda_stream
        s = self.stream
        if not hasattr(s, "cuda_stream"):
            s = torch.cuda.ExternalStream(int(s), device=self.device)
        self.stack.append(torch.cuda.stream(s))
        self.stack[-1].__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        while self.stack:
            self.stack.pop().__exit__(*exc)


@dataclass
class Pages:
    """One layer's dense cache: k and v [num_pages][kv_heads][page_size][d]."""

    k: torch.Tensor
    v: torch.Tensor

    @staticmethod
    def empty(num_pages: int, kv_heads: int, page_size: int, d: int, dtype, device) -> "Pages":
        shape = (num_pages, kv_heads, page_size, d)
        return Pages(torch.empty(shape, dtype=dtype, device=device),
                     torch.empty(shape, dtype=dtype, device=device))

    @property
    def page_size(self) -> int:
        return self.k.shape[2]

    def c(self) -> fadkv_pages:
        k, v = self.k, self.v
        if k.dim() != 4 or k.dtype not in _DT:
            raise ValueError("pages must be [num_pages][kv_heads][page_size][d] "
                             "float32/float16/bfloat16")
        _check(k, "pages.k")
        _check(v, "pages.v", k.dtype, k.shape)
        n, h, p, d = k.shape
        return fadkv_pages(n, p, h, d, _DT[k.dtype], k.data_ptr(), v.data_ptr())


@dataclass
class PageTable:
    """Which pages hold the rows of a batch, and which are free (fadkv_pages_advance)."""

    table: torch.Tensor        # int32 [R][max_pages]
    lens: torch.Tensor         # int32 [R]
    ring: torch.Tensor         # int32 [num_pages]
    ring_state: torch.Tensor   # int32 [2]: first free entry of ring, free entries
    page_size: int

    @staticmethod
    def empty(rows: int, max_pages: int, num_pages: int, page_size: int, device) -> "PageTable":
        """No row holds a token; every page is free."""
        return PageTable(torch.full((rows, max_pages), -1, dtype=torch.int32, device=device),
                         torch.zeros(rows, dtype=torch.int32, device=device),
                         torch.arange(num_pages, dtype=torch.int32, device=device),
                         torch.tensor([0, num_pages], dtype=torch.int32, device=device), page_size)


@dataclass
class PageStep:
    """What fadkv_pages_advance writes.  lens and ring_state may be those of the PageTable."""

    lens: torch.Tensor         # int32 [R]
    ring_state: torch.Tensor   # int32 [2]
    cu: torch.Tensor           # int32 [R + 1]
    status: torch.Tensor       # int32 [R]: ROW_*
    slots: torch.Tensor        # int32 [max_tokens]
    positions: torch.Tensor    # int32 [max_tokens]
    workspace: torch.Tensor

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
            return torch.empty(n, dtype=torch.int32, device=dev)
        return PageStep(pt.lens if in_place else i32(R), pt.ring_state if in_place else i32(2),
                        i32(R + 1), i32(R), i32(max_tokens), i32(max_tokens),
                        torch.empty(max(1, out.value), dtype=torch.uint8, device=dev))


def fadkv_pages_advance(pt: PageTable, new_lens: torch.Tensor, max_tokens: Optional[int] = None,
                        out: Optional[PageStep] = None, stream=None) -> PageStep:
    """One step of the bookkeeping: rows add new_lens [R] tokens (negative: the row has ended).
    pt.table and pt.ring are updated in place; give `out` (or the most tokens of a step)."""
    dev = pt.table.device
    i32 = torch.int32
    _check(pt.table, "table", i32)
    if pt.table.dim() != 2:
        raise ValueError("table must be [R][max_pages]")
    R, max_pages = pt.table.shape
    _check(pt.lens, "lens", i32, (R,))
    _check(pt.ring, "ring", i32)
    _check(pt.ring_state, "ring_state", i32, (2,))
    _check(new_lens, "new_lens", i32, (R,))
    if out is None and max_tokens is None:
        raise ValueError("give out or max_tokens")
    with _Launch(dev, stream) as strm:
        if out is None:
            out = PageStep.empty(pt, max_tokens)
        if max_tokens is not None and max_tokens != out.slots.numel():
            raise ValueError(f"out holds {out.slots.numel()} tokens, not {max_tokens}")
        _check(out.lens, "out.lens", i32, (R,))
        _check(out.ring_state, "out.ring_state", i32, (2,))
        _check(out.cu, "out.cu", i32, (R + 1,))
        _check(out.status, "out.status", i32, (R,))
        _check(out.slots, "out.slots", i32)
        _check(out.positions, "out.positions", i32, out.slots.shape)
        _check(out.workspace, "out.workspace", torch.uint8)
        _inputs(dev, lens=pt.lens, ring=pt.ring, ring_state=pt.ring_state, new_lens=new_lens,
                out=out.cu, out_lens=out.lens, out_ring_state=out.ring_state, status=out.status,
                slots=out.slots, positions=out.positions, workspace=out.workspace)
        st = lib().fadkv_pages_advance(
            pt.ring.numel(), pt.page_size, R, max_pages, new_lens.data_ptr(), pt.lens.data_ptr(),
            pt.table.data_ptr(), pt.ring.data_ptr(), pt.ring_state.data_ptr(), out.slots.numel(),
            out.lens.data_ptr(), out.ring_state.data_ptr(), out.cu.data_ptr(),
            out.status.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(),
            out.workspace.data_ptr(), out.workspace.numel(), strm)
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
    host = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.float64)
    buf = (ctypes.c_double * max(1, host.numel()))()
    mscale = ctypes.c_double(1.0)
    st = lib().fadkv_rope_freqs(int(rot_dim), float(base), _ROPE[kind], float(factor), float(low),
                                float(high), float(original_len), buf, ctypes.byref(mscale))
    if st != FADKV_OK:
        raise FadkvError("fadkv_rope_freqs", st)
    host.copy_(torch.tensor(buf[:host.numel()], dtype=torch.float64))
    return host.to(device), mscale.value


def _heads(t: torch.Tensor, name: str, dtype, n: int, d: int) -> int:
    """Checks [n][heads][d] whose heads lie together; returns the elements between tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != n or t.shape[2] != d:
        raise ValueError(f"{name} must be [{n}][heads][{d}], got {tuple(t.shape)}")
    h = t.shape[1]
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
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.dtype not in _DT:
        raise ValueError("q must be [n][heads][d] float32/float16/bfloat16")
    if q.device.type != "cuda":
        raise ValueError("q must live on the GPU")
    dev, dt = q.device, q.dtype
    n, heads, d = q.shape
    qs, ks, vs = _heads(q, "q", dt, n, d), _heads(k, "k", dt, n, d), _heads(v, "v", dt, n, d)
    kv = k.shape[1]
    if v.shape[1] != kv:
        raise ValueError(f"v must have {kv} heads as k, got {v.shape[1]}")
    _check(positions, "positions", torch.int32, (n,))
    rot = 0
    if freqs is not None:
        _check(freqs, "freqs", torch.float64)
        rot = 2 * freqs.numel()
    if q_weight is not None:
        _check(q_weight, "q_weight", dt, (d,))
    if k_weight is not None:
        _check(k_weight, "k_weight", dt, (d,))
    if (pages is None) != (slots is None):
        raise ValueError("pages and slots go together")
    if slots is not None:
        _check(slots, "slots", torch.int32, (n,))
    if k_rows is not None:
        _check(k_rows, "k_rows", dt, (kv, n, d))
    if v_rows is not None:
        _check(v_rows, "v_rows", dt, (kv, n, d))
    _inputs(dev, q=q, k=k, v=v, positions=positions, freqs=freqs, q_weight=q_weight,
            k_weight=k_weight, slots=slots, k_rows=k_rows, v_rows=v_rows,
            k_pages=pages and pages.k, v_pages=pages and pages.v, q_out=q_out)
    with _Launch(dev, stream) as strm:
        if q_out is None:
            q_out = torch.empty(n, heads, d, dtype=dt, device=dev)
        else:
            _check(q_out, "q_out", dt, (n, heads, d))
        a = fadkv_qkv(n, heads, kv, d, _DT[dt], q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks,
                      vs, positions.data_ptr(),
                      None if q_weight is None else q_weight.data_ptr(),
                      None if k_weight is None else k_weight.data_ptr(), eps,
                      freqs.data_ptr() if rot else None, rot, int(interleaved), mscale)
        st = lib().fadkv_norm_rope(
            ctypes.byref(a), q_out.data_ptr(),
            None if pages is None else ctypes.byref(pages.c()),
            None if slots is None else slots.data_ptr(),
            None if k_rows is None else k_rows.data_ptr(),
            None if v_rows is None else v_rows.data_ptr(), strm)
    if st != FADKV_OK:
        raise FadkvError("fadkv_norm_rope", st)
    return q_out


def fadkv_attend_paged_workspace_bytes(pages: Pages, R: int, heads: int, max_len: int) -> int:
    out = ctypes.c_size_t(0)
    st = lib().fadkv_attend_paged_workspace_bytes(ctypes.byref(pages.c()), int(R), int(heads),
                                                  int(max_len), ctypes.byref(out))
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_paged_workspace_bytes", st)
    return int(out.value)


def _attend_inputs(pages, table, lens, q, out):
    _check(q, "q", pages.k.dtype)
    if q.dim() != 3 or q.shape[2] != pages.k.shape[3]:
        raise ValueError(f"q must be [..][heads][{pages.k.shape[3]}]")
    _check(table, "table", torch.int32)
    if table.dim() != 2:
        raise ValueError("table must be [R][max_pages]")
    _check(lens, "lens", torch.int32, (table.shape[0],))
    if out is not None:
        _check(out, "out", q.dtype, q.shape)
    _inputs(q.device, q=q, table=table, lens=lens, k_pages=pages.k, v_pages=pages.v, out=out)


def fadkv_attend_paged(pages: Pages, table: torch.Tensor, lens: torch.Tensor, q: torch.Tensor,
                       scale: float, window: int = 0, sinks: int = 0,
                       max_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one new token per row, q [R][heads][d], over lens [R] cached tokens (its own
    included) in the pages of table [R][max_pages]; window > 0: only the last `window` tokens and
    the first `sinks` are visible.  Returns (or fills) out [R][heads][d]."""
    p = pages.c()
    _attend_inputs(pages, table, lens, q, out)
    R, max_pages = table.shape
    if q.shape[0] != R:
        raise ValueError(f"q must have {R} rows, got {q.shape[0]}")
    heads = q.shape[1]
    if max_len is None:
        max_len = max_pages * p.page_size
    with _Launch(q.device, stream) as strm:
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            need = fadkv_attend_paged_workspace_bytes(pages, R, heads, max_len)
            workspace = torch.empty(max(1, need), dtype=torch.uint8, device=q.device)
        else:
            _check(workspace, "workspace", torch.uint8)
            _inputs(q.device, workspace=workspace)
        st = lib().fadkv_attend_paged(ctypes.byref(p), table.data_ptr(), max_pages,
                                      lens.data_ptr(), R, q.data_ptr(), heads, scale, window,
                                      sinks, max_len, out.data_ptr(), workspace.data_ptr(),
                                      workspace.numel(), strm)
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_paged", st)
    return out


def fadkv_attend_prompt(pages: Pages, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                        q: torch.Tensor, scale: float, window: int = 0, sinks: int = 0,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of packed tokens q [n][heads][d]: tokens cu[r] .. cu[r+1] - 1 are the last
    of row r's lens[r] cached ones.  Returns (or fills) out [n][heads][d]; rows of out behind the
    last token stay as they were (undefined where out is allocated here)."""
    p = pages.c()
    _attend_inputs(pages, table, lens, q, out)
    R, max_pages = table.shape
    _check(cu, "cu", torch.int32, (R + 1,))
    _inputs(q.device, cu=cu)
    n, heads = q.shape[0], q.shape[1]
    with _Launch(q.device, stream) as strm:
        if out is None:
            out = torch.empty_like(q)
        st = lib().fadkv_attend_prompt(ctypes.byref(p), table.data_ptr(), max_pages,
                                       lens.data_ptr(), cu.data_ptr(), R, q.data_ptr(), n, heads,
                                       scale, window, sinks, out.data_ptr(), strm)
    if st != FADKV_OK:
        raise FadkvError("fadkv_attend_prompt", st)
    return out
