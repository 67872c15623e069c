"""Python binding of the densegemm C ABI (``include/densegemm.h``).

Argument marshalling only: tensors become device pointers, leading dimensions
and the current HIP stream; every step of the computation runs in the HIP
library ``libdensegemm.so``.  There is no fallback: if the library is missing
the import of this package fails.

Functions mirror the C entry points:

  select_tile(M, N, K, dtype="bf16", num_cus=0) -> Tile
  shuffle_b_bytes(N, K, dtype="bf16") -> int
  shuffle_b(B, dtype=None, out=None) -> Bs (uint8 device tensor)
  gemm_bf16(A, Bs, N, out=None, tile=None) -> C
  gemm_fp8_scaled(A, Bs, N, scale_a, scale_b, out=None, tile=None) -> C
  linear_cross_entropy(X, W, labels, ...) -> (loss, lse)
  linear_cross_entropy_grad(X, W, labels, loss, lse, dloss, ...) -> (dX, dW)
  linear_distillation(X, W, index, teacher, ...) -> (loss, lse, logp)
  linear_distillation_grad(X, W, index, teacher, lse, logp, dloss, ...) -> (dX, dW)
  group_sort(ids, groups) -> (offsets, order, place)
  group_gather(X, place) -> Xs
  group_combine(Y, place, weights=None) -> out
  group_combine_grad(dout, Y, place, weights) -> (dY, dweights)
  group_linear(X, W, offsets, order=None, ...) -> Y
  group_linear_grad(dY, X, W, offsets, order=None, ...) -> (dX, dW)
  linear_adapters(X, W, A, B, offsets, order, ...) -> Y
  gemm_status_string(code) -> str
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, replace

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdensegemm.so")

GEMM_OK = 0
GEMM_ERR_INVALID_VALUE = 1
GEMM_ERR_UNSUPPORTED = 2
GEMM_ERR_HIP = 3

GEMM_BF16 = 0
GEMM_FP8_E4M3 = 1

# bytes of the library's own split-K scratch behind gemm_bf16_noalloc
NOALLOC_SCRATCH_BYTES = 32 << 20
READ_PROBE_SLOTS = 32768

GEMM_KERNEL_TILED = 0
GEMM_KERNEL_SKINNY = 1
GEMM_KERNEL_TILED_AB = 2
GEMM_KERNEL_TILED_PP = 3

EXPORTS = ("select_tile", "shuffle_b_bytes", "shuffle_b", "gemm_bf16", "gemm_fp8_scaled",
           "gemm_tile_check", "gemm_status_string", "select_tile_ws", "gemm_workspace_bytes",
           "gemm_bf16_ws", "gemm_fp8_scaled_ws", "gemm_bf16_ex", "gemm_fp8_scaled_ex", "shuffle_b_t",
           "transpose_2d", "gemm_plan", "gemm_bf16_noalloc", "gemm_read_probe",
           "linear_loss_workspace_bytes", "linear_cross_entropy", "linear_cross_entropy_grad",
           "linear_distillation", "linear_distillation_grad", "group_sort_workspace_bytes", "group_sort",
           "group_gather", "group_combine", "group_combine_grad", "group_linear",
           "group_linear_grad_workspace_bytes", "group_linear_grad", "linear_adapters_workspace_bytes",
           "linear_adapters")

# gemm_activation
GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_SILU, GEMM_ACT_GELU_ERF, GEMM_ACT_GELU_TANH = 0, 1, 2, 3, 4
ACTIVATIONS = {None: GEMM_ACT_NONE, "none": GEMM_ACT_NONE, "relu": GEMM_ACT_RELU,
               "silu": GEMM_ACT_SILU, "gelu": GEMM_ACT_GELU_ERF, "gelu_erf": GEMM_ACT_GELU_ERF,
               "gelu_tanh": GEMM_ACT_GELU_TANH}


class GemmEpilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("scale_m", ctypes.c_void_p),
                ("scale_n", ctypes.c_void_p), ("mul", ctypes.c_void_p),
                ("ld_mul", ctypes.c_int64), ("activation", ctypes.c_int32)]


class GemmTile(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("atom", ctypes.c_int32), ("waves", ctypes.c_int32),
                ("k_split", ctypes.c_int32), ("lds_stages", ctypes.c_int32),
                ("tile_eff", ctypes.c_float), ("wq_eff", ctypes.c_float),
                ("predicted_us", ctypes.c_float), ("stream_k", ctypes.c_int32)]


@dataclass(frozen=True)
class Tile:
    kernel: int
    tile_m: int
    tile_n: int
    tile_k: int = 0
    atom: int = 16
    waves: int = 4
    k_split: int = 1
    lds_stages: int = 0
    tile_eff: float = 0.0
    wq_eff: float = 0.0
    predicted_us: float = 0.0
    stream_k: int = 0

    @property
    def name(self) -> str:
        """e.g. tiled128x128 (4 waves, 16x16 atom), ab256x256w8a32s4k32 (8 waves,
        32x32 atom, 4 stages, 32-element k-tile), tiled128x128a32s3k64sk4 (split
        over 4 K slices); unset fields are omitted."""
        atom = "" if self.atom in (0, 16) else f"a{self.atom}"
        pipe = (f"s{self.lds_stages}" if self.lds_stages else "") + (f"k{self.tile_k}" if self.tile_k else "")
        if self.kernel != GEMM_KERNEL_SKINNY and self.k_split > 1:
            pipe += f"sk{self.k_split}"
        if self.stream_k:
            pipe += "streamk"
        if self.kernel == GEMM_KERNEL_TILED:
            return f"tiled{self.tile_m}x{self.tile_n}" + ("" if self.waves == 4 else f"w{self.waves}") + \
                atom + pipe
        if self.kernel == GEMM_KERNEL_TILED_AB:
            return f"ab{self.tile_m}x{self.tile_n}w{self.waves}" + atom + pipe
        if self.kernel == GEMM_KERNEL_TILED_PP:
            return f"pp{self.tile_m}x{self.tile_n}" + atom + pipe
        return f"skinny{self.tile_m}x{self.tile_n}" + ("" if self.k_split in (0, 4) else f"w{self.k_split}")

    def to_c(self) -> GemmTile:
        return GemmTile(self.kernel, self.tile_m, self.tile_n, self.tile_k, self.atom, self.waves,
                        self.k_split, self.lds_stages, self.tile_eff, self.wq_eff, self.predicted_us,
                        self.stream_k)

    @staticmethod
    def from_c(t: GemmTile) -> "Tile":
        return Tile(t.kernel, t.tile_m, t.tile_n, t.tile_k, t.atom, t.waves, t.k_split,
                    t.lds_stages, t.tile_eff, t.wq_eff, t.predicted_us, t.stream_k)


def tiled(tm: int, tn: int, waves: int = 4, atom: int = 16, stages: int = 0, tile_k: int = 0,
          k_split: int = 1) -> Tile:
    """A rung of the tiled ladder; stages / tile_k (K elements per stage) 0 = any;
    k_split > 1 splits K over that many workgroups (needs a workspace)."""
    return Tile(GEMM_KERNEL_TILED, tm, tn, tile_k=tile_k, atom=atom, waves=waves, k_split=k_split,
                lds_stages=stages)


def tiled_ab(tm: int, tn: int, waves: int = 4, atom: int = 16, stages: int = 0, tile_k: int = 0,
             k_split: int = 1) -> Tile:
    """A rung of the A+B-in-LDS ladder; stages / tile_k 0 = any."""
    return Tile(GEMM_KERNEL_TILED_AB, tm, tn, tile_k=tile_k, atom=atom, waves=waves,
                k_split=k_split, lds_stages=stages)


def tiled_pp(tm: int, tn: int, atom: int = 32, stages: int = 0, tile_k: int = 0,
             k_split: int = 1) -> Tile:
    """A rung of the ping-pong A+B ladder (8 waves); stages / tile_k 0 = any."""
    return Tile(GEMM_KERNEL_TILED_PP, tm, tn, tile_k=tile_k, atom=atom, waves=8, k_split=k_split,
                lds_stages=stages)


def with_stream_k(tile: Tile) -> Tile:
    """The same one-pass tiled / A+B rung as a stream-K launch (needs a
    workspace of workspace_bytes(...) bytes)."""
    if tile.kernel not in (GEMM_KERNEL_TILED, GEMM_KERNEL_TILED_AB):
        raise ValueError("stream-K runs on tiled and A+B rungs")
    return replace(tile, stream_k=1, k_split=1)


def with_split(tile: Tile, k_split: int) -> Tile:
    """The same tiled rung split over k_split K slices."""
    if tile.kernel == GEMM_KERNEL_SKINNY:
        raise ValueError("the skinny kernel splits K inside one workgroup")
    return replace(tile, k_split=k_split)


def skinny(tm: int, tn: int, waves: int = 4) -> Tile:
    """A rung of the skinny ladder; `waves` split K inside one workgroup."""
    return Tile(GEMM_KERNEL_SKINNY, tm, tn, waves=waves, k_split=waves, lds_stages=0)


# The ladders of include/densegemm.h, as (tile_m, tile_n, waves, stages, atom,
# k-tile bytes).  8-wave tiled rungs arrange the waves 2 (M) x 4 (N); A+B
# rungs form 2 x (waves / 2).
TILED_LADDER = [(256, 128, 8, 2, 16, 128), (128, 256, 8, 2, 16, 128), (128, 128, 8, 2, 16, 128)] + \
    [(m, n, 4, 3, 16, 128) for m in (256, 128, 64, 32) for n in (256, 128, 64) if (m, n) != (256, 256)] + \
    [(256, 256, 8, 2, 32, 128), (256, 128, 8, 2, 32, 128), (128, 256, 8, 2, 32, 128),
     (128, 128, 8, 2, 32, 128), (256, 128, 4, 3, 32, 128), (128, 256, 4, 3, 32, 128),
     (128, 128, 4, 3, 32, 128), (64, 256, 4, 3, 32, 128), (64, 128, 4, 3, 32, 128),
     (128, 256, 4, 4, 32, 64), (128, 128, 4, 4, 32, 64), (256, 128, 4, 4, 32, 64)]
AB_LADDER = [(256, 128, 4, 3, 16, 128), (128, 256, 4, 3, 16, 128), (128, 128, 4, 3, 16, 128),
             (256, 256, 8, 2, 32, 128), (256, 256, 4, 2, 32, 128), (256, 128, 8, 3, 32, 128),
             (256, 128, 4, 3, 32, 128), (128, 256, 4, 3, 32, 128), (128, 128, 4, 3, 32, 128),
             (256, 256, 8, 4, 32, 64), (256, 256, 4, 4, 32, 64),
             (256, 128, 8, 6, 32, 64), (128, 256, 4, 6, 32, 64), (256, 256, 8, 4, 16, 64)]
# (tile_m, tile_n, waves splitting K)
# (tile_m, tile_n, stages, atom, k-tile bytes)
PP_LADDER = [(256, 256, 4, 32, 64)]
SKINNY_LADDER = [(m, n, 4) for m in (16, 32, 48, 64) for n in (16, 32, 64)] + \
    [(16, 16, 8), (16, 32, 8), (32, 16, 8), (32, 32, 8), (16, 16, 16), (32, 16, 16)]


def ladder_tiles(dtype="bf16"):
    """Every tiled and A+B rung, fully specified for an element type."""
    e = 2 if _dtype_code(dtype) == GEMM_BF16 else 1
    # e4m3 16 x 16 atoms take 128 K bytes per MFMA: 128-byte k-tiles only
    fits = lambda a, kb: not (e == 1 and a == 16 and kb != 128)  # noqa: E731
    return [tiled(m, n, w, a, st, kb // e) for m, n, w, st, a, kb in TILED_LADDER if fits(a, kb)] + \
        [tiled_ab(m, n, w, a, st, kb // e) for m, n, w, st, a, kb in AB_LADDER if fits(a, kb)] + \
        [tiled_pp(m, n, a, st, kb // e) for m, n, st, a, kb in PP_LADDER]


def all_tiles(M: int, dtype="bf16"):
    """Every rung usable for a GEMM with M rows."""
    t = ladder_tiles(dtype)
    if M <= 64:
        t += [skinny(m, n, w) for m, n, w in SKINNY_LADDER if M <= m < M + 16]
    return t


class GemmError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {gemm_status_string(code)}")
        self.code = code


def _load_lib():
    # Load torch's HIP runtime first.  torch ships its own libamdhip64 (soname
    # libamdhip64.so.7); once it is mapped, this library's dependency on that
    # soname resolves to the same copy, so the memory and streams torch hands
    # us belong to the runtime our kernels launch on.  Loading this library
    # first would map /opt/rocm's runtime as well: two HIP runtimes in one
    # process, and launches on torch's streams fail.
    import torch  # noqa: F401

    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g;"
                          f" g.build()'` (hipcc, gfx950). There is no fallback implementation.")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    I64 = ctypes.c_int64
    lib.select_tile.argtypes = [I64, I64, I64, ctypes.c_int, ctypes.c_int32, ctypes.POINTER(GemmTile)]
    lib.select_tile.restype = ctypes.c_int
    lib.shuffle_b_bytes.argtypes = [I64, I64, ctypes.c_int]
    lib.shuffle_b_bytes.restype = ctypes.c_size_t
    lib.shuffle_b.argtypes = [P, I64, P, I64, I64, ctypes.c_int, P]
    lib.shuffle_b.restype = ctypes.c_int
    lib.gemm_bf16.argtypes = [P, I64, P, P, I64, I64, I64, I64, ctypes.POINTER(GemmTile), P]
    lib.gemm_bf16.restype = ctypes.c_int
    lib.gemm_fp8_scaled.argtypes = [P, I64, P, P, P, P, I64, I64, I64, I64,
                                    ctypes.POINTER(GemmTile), P]
    lib.gemm_fp8_scaled.restype = ctypes.c_int
    lib.select_tile_ws.argtypes = [I64, I64, I64, ctypes.c_int, ctypes.c_int32, ctypes.c_size_t,
                                   ctypes.POINTER(GemmTile)]
    lib.select_tile_ws.restype = ctypes.c_int
    lib.gemm_workspace_bytes.argtypes = [I64, I64, I64, ctypes.c_int, ctypes.POINTER(GemmTile)]
    lib.gemm_workspace_bytes.restype = ctypes.c_size_t
    lib.gemm_bf16_ws.argtypes = [P, I64, P, P, I64, I64, I64, I64, ctypes.POINTER(GemmTile), P,
                                 ctypes.c_size_t, P]
    lib.gemm_bf16_ws.restype = ctypes.c_int
    lib.gemm_fp8_scaled_ws.argtypes = [P, I64, P, P, P, P, I64, I64, I64, I64,
                                       ctypes.POINTER(GemmTile), P, ctypes.c_size_t, P]
    lib.gemm_fp8_scaled_ws.restype = ctypes.c_int
    lib.gemm_bf16_ex.argtypes = [P, I64, P, P, I64, I64, I64, I64, ctypes.POINTER(GemmTile),
                                 ctypes.POINTER(GemmEpilogue), P, ctypes.c_size_t, P]
    lib.gemm_bf16_ex.restype = ctypes.c_int
    lib.gemm_fp8_scaled_ex.argtypes = [P, I64, P, P, P, P, I64, I64, I64, I64,
                                       ctypes.POINTER(GemmTile), ctypes.POINTER(GemmEpilogue), P,
                                       ctypes.c_size_t, P]
    lib.gemm_fp8_scaled_ex.restype = ctypes.c_int
    lib.shuffle_b_t.argtypes = [P, I64, P, I64, I64, ctypes.c_int, P]
    lib.shuffle_b_t.restype = ctypes.c_int
    lib.transpose_2d.argtypes = [P, I64, P, I64, I64, I64, ctypes.c_int32, P]
    lib.transpose_2d.restype = ctypes.c_int
    lib.gemm_bf16_noalloc.argtypes = [P, I64, P, P, I64, I64, I64, I64, ctypes.POINTER(GemmTile), P]
    lib.gemm_bf16_noalloc.restype = ctypes.c_int
    lib.gemm_plan.argtypes = [I64, I64, I64, ctypes.c_int, ctypes.c_int32, ctypes.c_size_t,
                              ctypes.POINTER(GemmTile), ctypes.POINTER(GemmTile),
                              ctypes.POINTER(I64), ctypes.POINTER(I64)]
    lib.gemm_plan.restype = ctypes.c_int
    lib.gemm_tile_check.argtypes = [ctypes.POINTER(GemmTile), I64, ctypes.c_int]
    lib.gemm_tile_check.restype = ctypes.c_int
    lib.gemm_read_probe.argtypes = [P, ctypes.c_uint64, P, P]
    lib.gemm_read_probe.restype = ctypes.c_int
    F = ctypes.c_float
    head = [P, I64, P, I64]                                       # X, W and their pitches
    space = [P, ctypes.c_size_t, P]                               # workspace, stream
    grads = [P, I64, P, I64, P, I64]                              # dloss, dX, dW
    lib.linear_loss_workspace_bytes.argtypes = [I64, I64, I64, I64, ctypes.c_int32]
    lib.linear_loss_workspace_bytes.restype = ctypes.c_size_t
    lib.linear_cross_entropy.argtypes = head + [P, I64, I64, I64, F, F, I64, P, P] + space
    lib.linear_cross_entropy.restype = ctypes.c_int
    lib.linear_cross_entropy_grad.argtypes = head + [P, I64, I64, I64, F, F, I64, P, P] + grads + space
    lib.linear_cross_entropy_grad.restype = ctypes.c_int
    lib.linear_distillation.argtypes = head + [P, I64, P, I64, I64, I64, I64, I64, F, P, P, P] + space
    lib.linear_distillation.restype = ctypes.c_int
    lib.linear_distillation_grad.argtypes = head + [P, I64, P, I64, I64, I64, I64, I64, F, P, P] + \
        grads + space
    lib.linear_distillation_grad.restype = ctypes.c_int
    stack = [P, I64, I64]                                         # pointer, pitch, group stride
    lib.group_sort_workspace_bytes.argtypes = [I64, I64, I64]
    lib.group_sort_workspace_bytes.restype = ctypes.c_size_t
    lib.group_sort.argtypes = [P, I64, I64, I64, I64, P, P, P] + space
    lib.group_sort.restype = ctypes.c_int
    lib.group_gather.argtypes = [P, I64, P, I64, I64, I64, ctypes.c_int32, P, I64, P]
    lib.group_gather.restype = ctypes.c_int
    lib.group_combine.argtypes = [P, I64, P, P, I64, I64, I64, I64, P, I64, P]
    lib.group_combine.restype = ctypes.c_int
    lib.group_combine_grad.argtypes = [P, I64, P, I64, P, P, I64, I64, I64, I64, P, I64, P, P]
    lib.group_combine_grad.restype = ctypes.c_int
    lib.group_linear.argtypes = [P, I64] + stack + [P, P, I64, I64, I64, I64, I64, ctypes.c_int32, P, I64,
                                                    P, I64, P]
    lib.group_linear.restype = ctypes.c_int
    lib.group_linear_grad_workspace_bytes.argtypes = [I64, I64, I64]
    lib.group_linear_grad_workspace_bytes.restype = ctypes.c_size_t
    lib.group_linear_grad.argtypes = [P, I64, P, I64] + stack + [P, P, I64, I64, I64, I64, I64, P, I64] + \
        stack + space
    lib.group_linear_grad.restype = ctypes.c_int
    lib.linear_adapters_workspace_bytes.argtypes = [I64, I64, I64]
    lib.linear_adapters_workspace_bytes.restype = ctypes.c_size_t
    lib.linear_adapters.argtypes = head + stack + stack + [P, P, P, I64, I64, I64, I64, I64, P, I64] + space
    lib.linear_adapters.restype = ctypes.c_int
    lib.gemm_status_string.argtypes = [ctypes.c_int]
    lib.gemm_status_string.restype = ctypes.c_char_p
    return lib


lib = _load_lib()


def gemm_status_string(code: int) -> str:
    return lib.gemm_status_string(int(code)).decode()


def _dtype_code(dtype) -> int:
    if dtype in ("bf16", GEMM_BF16):
        return GEMM_BF16
    if dtype in ("fp8", "e4m3", GEMM_FP8_E4M3):
        return GEMM_FP8_E4M3
    raise ValueError(f"unknown dtype {dtype!r}")


def select_tile(M: int, N: int, K: int, dtype="bf16", num_cus: int = 0,
                workspace_bytes: int = 0) -> Tile:
    """The library's choice; with workspace_bytes > 0, split-K tiles whose
    partials fit are candidates too (select_tile_ws)."""
    t = GemmTile()
    if workspace_bytes:
        st = lib.select_tile_ws(M, N, K, _dtype_code(dtype), num_cus, workspace_bytes, ctypes.byref(t))
    else:
        st = lib.select_tile(M, N, K, _dtype_code(dtype), num_cus, ctypes.byref(t))
    if st != GEMM_OK:
        raise GemmError("select_tile", st)
    return Tile.from_c(t)


def workspace_bytes(M: int, N: int, K: int, dtype, tile: Tile) -> int:
    """Device workspace `tile` needs on M x N x K (0 unless it splits K)."""
    return int(lib.gemm_workspace_bytes(M, N, K, _dtype_code(dtype), ctypes.byref(tile.to_c())))


def plan(M: int, N: int, K: int, dtype="bf16", num_cus: int = 256, workspace_bytes: int = 0):
    """The launches a GEMM with tile=None makes: (first tile, second tile or
    None, columns of the first launch, rows of the first launch).  A second
    launch takes the remaining columns (first columns < N) or the remaining
    rows (first rows < M)."""
    a, b, n, m = GemmTile(), GemmTile(), ctypes.c_int64(0), ctypes.c_int64(0)
    st = lib.gemm_plan(M, N, K, _dtype_code(dtype), num_cus, workspace_bytes, ctypes.byref(a),
                       ctypes.byref(b), ctypes.byref(n), ctypes.byref(m))
    if st != GEMM_OK:
        raise GemmError("gemm_plan", st)
    two = n.value < N or m.value < M
    return Tile.from_c(a), (Tile.from_c(b) if two else None), n.value, m.value


def tile_check(tile: Tile, M: int, dtype="bf16") -> int:
    """Status of forcing `tile` on an M-row GEMM of this dtype (GEMM_OK if a rung)."""
    return int(lib.gemm_tile_check(ctypes.byref(tile.to_c()), M, _dtype_code(dtype)))


def shuffle_b_bytes(N: int, K: int, dtype="bf16") -> int:
    return int(lib.shuffle_b_bytes(N, K, _dtype_code(dtype)))


# ------------------------------------------------------------ torch layer
def _torch():
    import torch
    return torch


def _stream_ptr(t) -> int:
    torch = _torch()
    return torch.cuda.current_stream(t.device).cuda_stream


def _tensor_dtype_code(t) -> int:
    torch = _torch()
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return GEMM_BF16
    if t.dtype in (torch.uint8, torch.int8, torch.float8_e4m3fn):
        return GEMM_FP8_E4M3
    raise TypeError(f"unsupported element type {t.dtype}")


def _check_rows(name: str, t):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def shuffle_b(B, dtype=None, out=None):
    """Preshuffle the row-major weight B [N, K] (bf16 or e4m3) into a new (or
    the given) uint8 device tensor of shuffle_b_bytes(N, K) bytes."""
    torch = _torch()
    _check_rows("B", B)
    code = _tensor_dtype_code(B) if dtype is None else _dtype_code(dtype)
    N, K = B.shape
    nbytes = shuffle_b_bytes(N, K, code)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=B.device)
    elif out.numel() * out.element_size() < nbytes:
        raise ValueError("out is too small")
    st = lib.shuffle_b(B.data_ptr(), B.stride(0), out.data_ptr(), N, K, code, _stream_ptr(B))
    if st != GEMM_OK:
        raise GemmError("shuffle_b", st)
    return out


def read_probe(buf, out=None):
    """Read every byte of the contiguous device tensor `buf` once with the
    library's streaming-read probe (a measurement aid: the time floor of a
    kernel that reads the same bytes).  Returns `out`, READ_PROBE_SLOTS
    uint32 values (as int32) whose XOR is the XOR of all 32-bit words of
    buf."""
    torch = _torch()
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous device tensor")
    nbytes = buf.numel() * buf.element_size()
    if out is None:
        out = torch.empty(READ_PROBE_SLOTS, dtype=torch.int32, device=buf.device)
    elif (not out.is_cuda or out.dtype != torch.int32 or out.numel() < READ_PROBE_SLOTS
          or out.device != buf.device):
        raise ValueError(f"out must be an int32 device tensor of {READ_PROBE_SLOTS} elements "
                         "on buf's device")
    st = lib.gemm_read_probe(buf.data_ptr(), nbytes, out.data_ptr(), _stream_ptr(buf))
    if st != GEMM_OK:
        raise GemmError("gemm_read_probe", st)
    return out


def shuffle_b_t(Bt, dtype=None, out=None):
    """The preshuffled weight of B = Bt^T, from Bt [K, N] (bf16 or e4m3): the
    same bytes as shuffle_b(Bt.T) without materialising the transpose."""
    torch = _torch()
    _check_rows("Bt", Bt)
    code = _tensor_dtype_code(Bt) if dtype is None else _dtype_code(dtype)
    K, N = Bt.shape
    nbytes = shuffle_b_bytes(N, K, code)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=Bt.device)
    elif out.numel() * out.element_size() < nbytes:
        raise ValueError("out is too small")
    st = lib.shuffle_b_t(Bt.data_ptr(), Bt.stride(0), out.data_ptr(), N, K, code, _stream_ptr(Bt))
    if st != GEMM_OK:
        raise GemmError("shuffle_b_t", st)
    return out


def transpose(X, out=None):
    """X^T of a 2-D device tensor of 1- or 2-byte elements, into a new (or the
    given [cols, rows]) tensor of the same dtype."""
    torch = _torch()
    _check_rows("X", X)
    rows, cols = X.shape
    if out is None:
        out = torch.empty((cols, rows), dtype=X.dtype, device=X.device)
    else:
        _check_rows("out", out)
        if tuple(out.shape) != (cols, rows) or out.element_size() != X.element_size():
            raise ValueError("out must be [cols, rows] with X's element size")
    st = lib.transpose_2d(X.data_ptr(), X.stride(0), out.data_ptr(), out.stride(0), rows, cols,
                          X.element_size(), _stream_ptr(X))
    if st != GEMM_OK:
        raise GemmError("transpose_2d", st)
    return out


def grad_input(dY, W, out=None, Ws_t=None, **kw):
    """dX = dY W for a linear layer Y = X W^T (bf16): the GEMM C = A B^T with
    A = dY [M, N_out] and B = W^T, preshuffled by shuffle_b_t(W) (pass it as
    Ws_t to reuse it across calls).  Extra keywords go to gemm_bf16."""
    Bs = shuffle_b_t(W) if Ws_t is None else Ws_t
    return gemm_bf16(dY, Bs, W.shape[1], out=out, **kw)


def grad_weight(dY, X, out=None, **kw):
    """dW = dY^T X for a linear layer Y = X W^T (bf16): A = transpose(dY)
    [N_out, M] and B = X^T, preshuffled by shuffle_b_t(X); the sum runs over
    the M tokens, so M is this GEMM's K and follows its contract (a multiple
    of 16; pad the token dimension with zero rows otherwise).  Extra keywords
    go to gemm_bf16."""
    return gemm_bf16(transpose(dY), shuffle_b_t(X), X.shape[1], out=out, **kw)


def _out(A, N, out):
    torch = _torch()
    M = A.shape[0]
    if out is None:
        return torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check_rows("out", out)
    if tuple(out.shape) != (M, N) or out.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise ValueError("out must be a bf16 [M, N] view")
    return out


def _check_operands(code: int, A, Bs, N: int, scales=()):
    """Everything the C ABI cannot see behind its plain pointers, checked
    before any launch: A's element type matches the entry point (an e4m3 A
    handed to the bf16 GEMM would have its byte pitch read as a bf16 pitch),
    Bs is a device buffer at least shuffle_b_bytes(N, K) long (the kernels
    size their B bounds from N and K, not from the buffer), and each scale is
    a float32 device tensor with at least one element (a host tensor would
    hand the kernel a host pointer).  Element types are checked first, so
    the checks also run on a machine without a GPU."""
    torch = _torch()
    want = (torch.bfloat16, torch.int16, torch.uint16) if code == GEMM_BF16 else \
        (torch.uint8, torch.int8, torch.float8_e4m3fn)
    fn = "gemm_bf16" if code == GEMM_BF16 else "gemm_fp8_scaled"
    if A.dtype not in want:
        raise ValueError(f"{fn}: A has element type {A.dtype}, expected one of "
                         f"{', '.join(str(d) for d in want)}")
    for name, t in scales:
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() < 1:
            raise ValueError(f"{fn}: {name} must be a float32 device tensor with one element")
    if not isinstance(Bs, torch.Tensor):
        raise ValueError(f"{fn}: Bs must be the device tensor shuffle_b returned")
    _check_rows("A", A)
    if not Bs.is_cuda or Bs.device != A.device:
        raise ValueError(f"{fn}: Bs must be a device tensor on A's device")
    if not Bs.is_contiguous():
        raise ValueError(f"{fn}: Bs must be contiguous (the preshuffled layout is dense)")
    need = shuffle_b_bytes(N, A.shape[1], code)
    if Bs.numel() * Bs.element_size() < need:
        raise ValueError(f"{fn}: Bs holds {Bs.numel() * Bs.element_size()} bytes, the "
                         f"preshuffled B of N={N}, K={A.shape[1]} needs {need}")
    for name, t in scales:
        if not t.is_cuda or t.device != A.device:
            raise ValueError(f"{fn}: {name} must be on A's device, not {t.device}")


def _tile_ptr(tile):
    if tile is None:
        return None
    return ctypes.byref(tile.to_c())


def _workspace(A, N: int, K: int, code: int, tile, workspace):
    """(pointer, bytes) of the split-K workspace: the caller's uint8 device
    tensor, or a new one when a forced split-K tile needs it, else none."""
    if workspace is not None:
        if not workspace.is_cuda:
            raise ValueError("workspace must be a device tensor")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if tile is None or tile.kernel == GEMM_KERNEL_SKINNY or (tile.k_split <= 1 and not tile.stream_k):
        return None, 0
    nbytes = workspace_bytes(A.shape[0], N, K, code, tile)
    if nbytes == 0:
        return None, 0
    # torch's caching allocator hands this block out again only to work
    # ordered after ours on the same (current) stream, so it may be freed on
    # return
    ws = _torch().empty(nbytes, dtype=_torch().uint8, device=A.device)
    return ws.data_ptr(), nbytes


def _epilogue(A, N: int, bias, scale_m, scale_n, activation, mul):
    """The gemm_epilogue struct for the given parts, or None when there are none."""
    act = ACTIVATIONS[activation] if not isinstance(activation, int) else activation
    if bias is None and scale_m is None and scale_n is None and mul is None and act == GEMM_ACT_NONE:
        return None
    torch = _torch()
    M = A.shape[0]

    def vec(name, t, n, dtypes):
        if t.dim() != 1 or t.shape[0] != n or t.stride(0) != 1 or not t.is_cuda or t.dtype not in dtypes:
            raise ValueError(f"{name} must be a contiguous device vector of {n} {dtypes[0]}")
        return t.data_ptr()
    e = GemmEpilogue()
    bf = (torch.bfloat16, torch.int16, torch.uint16)
    if bias is not None:
        e.bias = vec("bias", bias, N, bf)
    if scale_m is not None:
        e.scale_m = vec("scale_m", scale_m, M, (torch.float32,))
    if scale_n is not None:
        e.scale_n = vec("scale_n", scale_n, N, (torch.float32,))
    if mul is not None:
        _check_rows("mul", mul)
        if tuple(mul.shape) != (M, N) or mul.dtype not in bf:
            raise ValueError("mul must be a bf16 [M, N] view")
        e.mul = mul.data_ptr()
        e.ld_mul = mul.stride(0)
    e.activation = act
    return e


def gemm_bf16(A, Bs, N: int, out=None, tile: Tile | None = None, workspace=None, *, bias=None,
              scale_m=None, scale_n=None, activation=None, mul=None):
    """C[M, N] = A[M, K] * B[N, K]^T with Bs = shuffle_b(B); returns C (bf16).
    workspace: a uint8 device tensor for split-K (then tile None lets the
    library weigh split-K tiles that fit in it).  Fused epilogue (all
    optional): C = act(acc * scale_m[m] * scale_n[n] + bias[n]) * mul[m, n],
    activation one of ACTIVATIONS; mul may be `out` itself."""
    _check_operands(GEMM_BF16, A, Bs, N)
    C = _out(A, N, out)
    M, K = A.shape
    ws, nbytes = _workspace(A, N, K, GEMM_BF16, tile, workspace)
    epi = _epilogue(A, N, bias, scale_m, scale_n, activation, mul)
    if epi is not None:
        st = lib.gemm_bf16_ex(A.data_ptr(), A.stride(0), Bs.data_ptr(), C.data_ptr(), C.stride(0),
                              M, N, K, _tile_ptr(tile), ctypes.byref(epi), ws, nbytes,
                              _stream_ptr(A))
    elif ws is None:
        st = lib.gemm_bf16(A.data_ptr(), A.stride(0), Bs.data_ptr(), C.data_ptr(), C.stride(0), M,
                           N, K, _tile_ptr(tile), _stream_ptr(A))
    else:
        st = lib.gemm_bf16_ws(A.data_ptr(), A.stride(0), Bs.data_ptr(), C.data_ptr(), C.stride(0),
                              M, N, K, _tile_ptr(tile), ws, nbytes, _stream_ptr(A))
    if st != GEMM_OK:
        raise GemmError("gemm_bf16", st)
    return C


def gemm_fp8_scaled(A, Bs, N: int, scale_a, scale_b, out=None, tile: Tile | None = None,
                    workspace=None, *, bias=None, scale_m=None, scale_n=None, activation=None,
                    mul=None):
    """C = (A * B^T) * scale_a * scale_b for e4m3 A [M, K] and Bs = shuffle_b(B);
    scale_a / scale_b are one-element float32 device tensors.  The fused
    epilogue parts are those of gemm_bf16 (scale_m / scale_n: per-token and
    per-channel fp32 multipliers)."""
    _check_operands(GEMM_FP8_E4M3, A, Bs, N, (("scale_a", scale_a), ("scale_b", scale_b)))
    C = _out(A, N, out)
    M, K = A.shape
    ws, nbytes = _workspace(A, N, K, GEMM_FP8_E4M3, tile, workspace)
    epi = _epilogue(A, N, bias, scale_m, scale_n, activation, mul)
    if epi is not None:
        st = lib.gemm_fp8_scaled_ex(A.data_ptr(), A.stride(0), Bs.data_ptr(), scale_a.data_ptr(),
                                    scale_b.data_ptr(), C.data_ptr(), C.stride(0), M, N, K,
                                    _tile_ptr(tile), ctypes.byref(epi), ws, nbytes,
                                    _stream_ptr(A))
    elif ws is None:
        st = lib.gemm_fp8_scaled(A.data_ptr(), A.stride(0), Bs.data_ptr(), scale_a.data_ptr(),
                                 scale_b.data_ptr(), C.data_ptr(), C.stride(0), M, N, K,
                                 _tile_ptr(tile), _stream_ptr(A))
    else:
        st = lib.gemm_fp8_scaled_ws(A.data_ptr(), A.stride(0), Bs.data_ptr(), scale_a.data_ptr(),
                                    scale_b.data_ptr(), C.data_ptr(), C.stride(0), M, N, K,
                                    _tile_ptr(tile), ws, nbytes, _stream_ptr(A))
    if st != GEMM_OK:
        raise GemmError("gemm_fp8_scaled", st)
    return C


def gemm_bf16_noalloc(A, Bs, N: int, out, tile: Tile | None = None):
    """gemm_bf16 for callers that cannot allocate: split-K partials go to the
    library's fixed scratch array (NOALLOC_SCRATCH_BYTES per GPU), `out` must
    be given, and nothing is allocated.  Calls on one GPU must not overlap."""
    _check_operands(GEMM_BF16, A, Bs, N)
    if out is None:
        raise ValueError("gemm_bf16_noalloc: out must be given (the call allocates nothing)")
    C = _out(A, N, out)
    M, K = A.shape
    st = lib.gemm_bf16_noalloc(A.data_ptr(), A.stride(0), Bs.data_ptr(), C.data_ptr(), C.stride(0),
                               M, N, K, _tile_ptr(tile), _stream_ptr(A))
    if st != GEMM_OK:
        raise GemmError("gemm_bf16_noalloc", st)
    return C


# ------------------------------------------------- losses of a linear head
def linear_loss_workspace_bytes(T: int, V: int, D: int, slots: int = 0, backward: bool = False) -> int:
    """Workspace of the linear_* losses for X [T, D], W [V, D] and `slots`
    target slots a row (0: cross entropy).  backward: of the gradient call; it
    serves the forward call too.  0 for T == 0 and for sizes the calls refuse."""
    return int(lib.linear_loss_workspace_bytes(T, V, D, slots, int(bool(backward))))


def _loss_operands(fn: str, X, W, per_row=(), per_slot=()):
    """Element types, shapes and devices the C ABI cannot see.  per_row: (name,
    tensor, dtype) vectors of T; per_slot: [T, k] tensors.  Types first, so
    that the checks also run on a machine without a GPU."""
    torch = _torch()
    for name, t in (("X", X), ("W", W)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16:
            raise ValueError(f"{fn}: {name} must be a bfloat16 tensor")
    for name, t, dt in tuple(per_row) + tuple(per_slot):
        if not isinstance(t, torch.Tensor) or t.dtype != dt:
            raise ValueError(f"{fn}: {name} must be a {dt} tensor")
    for name, t in (("X", X), ("W", W)):
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{fn}: {name} must be a 2-D tensor with contiguous rows")
    if X.shape[1] != W.shape[1]:
        raise ValueError(f"{fn}: X has {X.shape[1]} columns, W {W.shape[1]}")
    T = X.shape[0]
    for name, t, _ in per_row:
        if tuple(t.shape) != (T,) or (T > 1 and t.stride(0) != 1):
            raise ValueError(f"{fn}: {name} must be a contiguous vector of {T} values")
    for name, t, _ in per_slot:
        if t.dim() != 2 or tuple(t.shape) != (T, per_slot[0][1].shape[-1]) or \
                (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{fn}: {name} must be a [{T}, slots] tensor with contiguous rows")
    for name, t in [("X", X), ("W", W)] + [(a, b) for a, b, _ in tuple(per_row) + tuple(per_slot)]:
        if not t.is_cuda or t.device != X.device:
            raise ValueError(f"{fn}: {name} must be a device tensor on X's device")


def _pitch(t):
    """Row pitch in elements (a single row's stride means nothing to a call)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _row_pitch8(t):
    """_pitch for operands whose pitch the C ABI wants in multiples of 8."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def _loss_workspace(fn: str, X, V: int, slots: int, backward: bool, workspace):
    torch = _torch()
    need = linear_loss_workspace_bytes(X.shape[0], V, X.shape[1], slots, backward)
    if workspace is None:
        # freed on return: the caching allocator reuses it on this stream only
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=X.device)
    elif not workspace.is_cuda or workspace.device != X.device or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be a contiguous device tensor on X's device")
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"{fn}: workspace holds {workspace.numel() * workspace.element_size()} "
                         f"bytes, {need} are needed")
    return workspace, workspace.numel() * workspace.element_size()


def _loss_grads(fn: str, X, W, dloss, need_dX, need_dW, dX, dW):
    """(dloss, count, dX or None, dW or None) with the outputs made or checked."""
    torch = _torch()
    if not isinstance(dloss, torch.Tensor) or dloss.dtype != torch.float32:
        raise ValueError(f"{fn}: dloss must be a float32 tensor")
    T = X.shape[0]
    if dloss.numel() != 1:
        if tuple(dloss.shape) != (T,):
            raise ValueError(f"{fn}: dloss must hold {T} values or one")
        if dloss.stride(0) == 0:
            dloss = dloss[:1]                    # one value expanded to every row
        elif dloss.stride(0) != 1:
            raise ValueError(f"{fn}: dloss must be contiguous")
    if not dloss.is_cuda or dloss.device != X.device:
        raise ValueError(f"{fn}: dloss must be a device tensor on X's device")
    outs = []
    for name, need, given, like in (("dX", need_dX, dX, X), ("dW", need_dW, dW, W)):
        if not need:
            if given is not None:
                raise ValueError(f"{fn}: {name} given, but need_{name} is false")
            outs.append(None)
            continue
        if given is None:
            given = torch.empty(like.shape, dtype=torch.bfloat16, device=X.device)
        elif given.dtype != torch.bfloat16 or tuple(given.shape) != tuple(like.shape) or \
                not given.is_cuda or given.device != X.device or \
                (given.shape[1] > 1 and given.stride(1) != 1) or \
                (given.shape[0] > 1 and given.stride(0) < given.shape[1]):
            raise ValueError(f"{fn}: {name} must be a bfloat16 {tuple(like.shape)} view with "
                             "contiguous rows on X's device")
        outs.append(given)
    if outs[0] is None and outs[1] is None:
        raise ValueError(f"{fn}: neither dX nor dW is asked for")
    return dloss, (T if dloss.numel() == T else 1), outs[0], outs[1]


def _grad_pointers(dX, dW):
    out = []
    for t in (dX, dW):
        out += [None, 0] if t is None else [t.data_ptr(), _pitch(t)]
    return out


def _loss_call(fn: str, X, args, ws, nbytes):
    # launches go to X's device, whichever device is current
    with _torch().cuda.device(X.device):
        st = getattr(lib, fn)(*args, ws.data_ptr(), nbytes, _stream_ptr(X))
    if st != GEMM_OK:
        raise GemmError(fn, st)


def linear_cross_entropy(X, W, labels, *, scale: float = 1.0, z_loss: float = 0.0,
                         ignore_index: int = -100, workspace=None):
    """Softmax cross entropy of a linear head, one loss a row, without the
    logits in memory: z = scale * X W^T (X [T, D], W [V, D] bf16), labels int64
    [T]; loss[t] = lse[t] - z[t, labels[t]] + z_loss * lse[t]^2.  Returns (loss,
    lse), float32 [T].  Rows with label ignore_index get 0 in both; a label
    outside the vocabulary gives a NaN loss.  workspace: a uint8 device tensor
    of linear_loss_workspace_bytes bytes (made for the call if not given)."""
    torch = _torch()
    fn = "linear_cross_entropy"
    _loss_operands(fn, X, W, (("labels", labels, torch.int64),))
    (T, D), V = X.shape, W.shape[0]
    loss = torch.empty(T, dtype=torch.float32, device=X.device)
    lse = torch.empty(T, dtype=torch.float32, device=X.device)
    ws, nbytes = _loss_workspace(fn, X, V, 0, False, workspace)
    _loss_call(fn, X, (X.data_ptr(), _row_pitch8(X), W.data_ptr(), _row_pitch8(W), labels.data_ptr(), T, V,
                       D, scale, z_loss, ignore_index, loss.data_ptr(), lse.data_ptr()), ws, nbytes)
    return loss, lse


def linear_cross_entropy_grad(X, W, labels, loss, lse, dloss, *, scale: float = 1.0,
                              z_loss: float = 0.0, ignore_index: int = -100, need_dX: bool = True,
                              need_dW: bool = True, dX=None, dW=None, workspace=None):
    """The gradients of linear_cross_entropy, with the loss and lse it returned
    for the same arguments and dloss (float32, [T] or one value) the gradient
    with respect to each row's loss.  Returns (dX, dW), bf16, None for one that
    is not needed (need_dX, need_dW); dX / dW: views to write instead of new
    tensors, which must not overlap the inputs or each other."""
    torch = _torch()
    fn = "linear_cross_entropy_grad"
    _loss_operands(fn, X, W, (("labels", labels, torch.int64), ("loss", loss, torch.float32),
                              ("lse", lse, torch.float32)))
    (T, D), V = X.shape, W.shape[0]
    dloss, count, dX, dW = _loss_grads(fn, X, W, dloss, need_dX, need_dW, dX, dW)
    ws, nbytes = _loss_workspace(fn, X, V, 0, True, workspace)
    _loss_call(fn, X, (X.data_ptr(), _row_pitch8(X), W.data_ptr(), _row_pitch8(W), labels.data_ptr(), T, V,
                       D, scale, z_loss, ignore_index, loss.data_ptr(), lse.data_ptr(),
                       dloss.data_ptr(), count, *_grad_pointers(dX, dW)), ws, nbytes)
    return dX, dW


def linear_distillation(X, W, index, teacher, *, scale: float = 1.0, workspace=None):
    """Distillation loss of a linear head against a teacher's top logits,
    without the student's logits in memory.  index int64 [T, slots] names the
    teacher's columns, teacher float32 [T, slots] its logits there; a negative
    index or a logit of -inf leaves a slot empty.  With z = scale * X W^T and q =
    softmax(scale * teacher) over a row's filled slots, loss[t] = sum_j q_j (log
    q_j - logp[t, j]), logp[t, j] = z[t, index[t, j]] - lse[t].  Returns (loss,
    lse, logp), float32; a row with no filled slot gets 0 in all three."""
    torch = _torch()
    fn = "linear_distillation"
    _loss_operands(fn, X, W, (), (("index", index, torch.int64), ("teacher", teacher, torch.float32)))
    (T, D), V, k = X.shape, W.shape[0], index.shape[1]
    loss = torch.empty(T, dtype=torch.float32, device=X.device)
    lse = torch.empty(T, dtype=torch.float32, device=X.device)
    logp = torch.empty((T, k), dtype=torch.float32, device=X.device)
    ws, nbytes = _loss_workspace(fn, X, V, k, False, workspace)
    _loss_call(fn, X, (X.data_ptr(), _row_pitch8(X), W.data_ptr(), _row_pitch8(W), index.data_ptr(),
                       _pitch(index), teacher.data_ptr(), _pitch(teacher), T, V, D, k, scale,
                       loss.data_ptr(), lse.data_ptr(), logp.data_ptr()), ws, nbytes)
    return loss, lse, logp


def linear_distillation_grad(X, W, index, teacher, lse, logp, dloss, *, scale: float = 1.0,
                             need_dX: bool = True, need_dW: bool = True, dX=None, dW=None,
                             workspace=None):
    """The gradients of linear_distillation, with the lse and logp it returned
    for the same arguments; dloss, need_*, dX, dW and the result as for
    linear_cross_entropy_grad.  The teacher's logits get no gradient."""
    torch = _torch()
    fn = "linear_distillation_grad"
    _loss_operands(fn, X, W, (("lse", lse, torch.float32),),
                   (("index", index, torch.int64), ("teacher", teacher, torch.float32),
                    ("logp", logp, torch.float32)))
    (T, D), V, k = X.shape, W.shape[0], index.shape[1]
    if not logp.is_contiguous():
        raise ValueError(f"{fn}: logp must be contiguous")
    dloss, count, dX, dW = _loss_grads(fn, X, W, dloss, need_dX, need_dW, dX, dW)
    ws, nbytes = _loss_workspace(fn, X, V, k, True, workspace)
    _loss_call(fn, X, (X.data_ptr(), _row_pitch8(X), W.data_ptr(), _row_pitch8(W), index.data_ptr(),
                       _pitch(index), teacher.data_ptr(), _pitch(teacher), T, V, D, k, scale,
                       lse.data_ptr(), logp.data_ptr(), dloss.data_ptr(), count,
                       *_grad_pointers(dX, dW)), ws, nbytes)
    return dX, dW


# ------------------------- linear layers whose weight depends on the row
def group_sort_workspace_bytes(T: int, slots: int, groups: int) -> int:
    """Workspace of group_sort for ids [T, slots]: 0 up to 4096 slots."""
    return int(lib.group_sort_workspace_bytes(T, slots, groups))


def group_linear_grad_workspace_bytes(T: int, slots: int, K: int) -> int:
    """Workspace of group_linear_grad for X [T, K] with an order, where dW is asked for."""
    return int(lib.group_linear_grad_workspace_bytes(T, slots, K))


def linear_adapters_workspace_bytes(T: int, R: int, groups: int) -> int:
    """Workspace of linear_adapters for T rows and adapters of rank R."""
    return int(lib.linear_adapters_workspace_bytes(T, R, groups))


# Element types and allocation as plain globals: a call of these takes 3 us in the
# driver, and as much again went to looking things up.
import torch as _pt  # noqa: E402  (loaded by _load_lib already)

_BF16, _F32, _I32, _I64 = _pt.bfloat16, _pt.float32, _pt.int32, _pt.int64
_new = _pt.empty_strided


def _public_stream(dev: int) -> int:
    return _pt.cuda.current_stream(dev).cuda_stream


# (where this build of torch has the shorter ways)
_raw_stream = getattr(_pt._C, "_cuda_getCurrentRawStream", _public_stream)
_current_device = getattr(_pt._C, "_cuda_getDevice", _pt.cuda.current_device)


def _refuse(fn: str, name: str, what: str):
    raise ValueError(f"{fn}: {name} must be {what}")


def _extent(shape) -> str:
    return "[" + ", ".join("any" if n is None else str(n) for n in shape) + "]"


def _matrix(fn: str, name: str, t, dtype, rows=None, cols=None):
    """A 2-D view (rows, cols None: any) with contiguous rows: (rows, columns, pitch).
    A single row's stride says nothing; its pitch is the columns in whole 8."""
    if getattr(t, "dtype", None) is not dtype:
        _refuse(fn, name, f"a {dtype} tensor")
    shape = t.shape
    if len(shape) == 2:
        n, w = shape
        p, q = t.stride()
        if (rows is None or n == rows) and (cols is None or w == cols) and (q == 1 or w < 2):
            if n < 2:
                return n, w, (w + 7) // 8 * 8
            if p >= w:
                return n, w, p
    _refuse(fn, name, f"a {_extent((rows, cols))} tensor with contiguous rows")


def _stack(fn: str, name: str, t, dtype, groups=None, rows=None, cols=None):
    """A 3-D view with contiguous rows: (groups, rows, columns, pitch, group stride)."""
    if getattr(t, "dtype", None) is not dtype:
        _refuse(fn, name, f"a {dtype} tensor")
    shape = t.shape
    if len(shape) == 3:
        g, n, w = shape
        s, p, q = t.stride()
        if (groups is None or g == groups) and (rows is None or n == rows) and \
                (cols is None or w == cols) and (q == 1 or w < 2) and (n < 2 or p >= w):
            pitch = p if n > 1 else (w + 7) // 8 * 8
            return g, n, w, pitch, (s if g > 1 else n * pitch)
    _refuse(fn, name, f"a {_extent((groups, rows, cols))} tensor with contiguous rows")


def _vector(fn: str, name: str, t, dtype, n: int):
    if getattr(t, "dtype", None) is not dtype:
        _refuse(fn, name, f"a {dtype} tensor")
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        _refuse(fn, name, f"a contiguous vector of {n} values")


def _place(fn: str, place, T=None):
    T, k, _ = _matrix(fn, "place", place, _I32, T)
    if not place.is_contiguous():
        _refuse(fn, "place", "contiguous")
    return T, k


def _one_device(fn: str, names: str, first, *others) -> int:
    """The device of the first tensor, which the others (None: absent) share."""
    dev = first.get_device()
    if dev < 0:
        _refuse(fn, names.split()[0], "a device tensor")
    for t in others:
        if t is not None and t.get_device() != dev:
            name = next(n for n, o in zip(names.split()[1:], others) if o is t)
            _refuse(fn, name, f"a device tensor on cuda:{dev}")
    return dev


def _group_workspace(fn: str, device, need: int, workspace):
    """(tensor, pointer, bytes): the caller's, or one made for the call."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        # freed on return: the caching allocator reuses it on this stream only
        workspace = _pt.empty(need, dtype=_pt.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        _refuse(fn, "workspace", f"a contiguous device tensor on {device}")
    nbytes = workspace.numel() * workspace.element_size()
    if nbytes < need:
        raise ValueError(f"{fn}: workspace holds {nbytes} bytes, {need} are needed")
    return workspace, workspace.data_ptr(), nbytes


def _ptr(t):
    return None if t is None else t.data_ptr()


def _group_call(fn: str, dev: int, *args):
    """The C call on the current stream of the operands' device, whichever device is
    current.  (The stream's handle without the Stream object, and no device guard
    where none is needed: together 3 of 13 us a call.)"""
    if _current_device() == dev:
        st = getattr(lib, fn)(*args, _raw_stream(dev))
    else:
        with _pt.cuda.device(dev):
            st = getattr(lib, fn)(*args, _raw_stream(dev))
    if st != GEMM_OK:
        raise GemmError(fn, st)


def group_sort(ids, groups: int, *, workspace=None):
    """Sort the slots of ids (int64 [T, slots], or [T]) by group id, stable.
    Returns int32 (offsets [groups + 1], order [T * slots], place [T, slots]):
    group g's rows are the sorted positions offsets[g] .. offsets[g + 1] - 1,
    order[p] is the slot t * slots + j at position p, place[t, j] the position of a
    slot.  An id outside [0, groups) takes no part: its place is -1, and it
    stands in order behind the others."""
    fn = "group_sort"
    if isinstance(ids, _pt.Tensor) and ids.dim() == 1:
        ids = ids[:, None]
    T, k, ld = _matrix(fn, "ids", ids, _I64)
    dev = _one_device(fn, "ids", ids)
    if groups < 1:
        raise ValueError(f"{fn}: groups must be at least 1")
    device = ids.device
    offsets = _new((groups + 1,), (1,), dtype=_I32, device=device)
    order = _new((T * k,), (1,), dtype=_I32, device=device)
    place = _new((T, k), (k, 1), dtype=_I32, device=device)
    need = lib.group_sort_workspace_bytes(T, k, groups)
    ws, at, nbytes = _group_workspace(fn, device, need, workspace) if need else (None, None, 0)
    _group_call(fn, dev, ids.data_ptr(), ld, T, k, groups, offsets.data_ptr(), order.data_ptr(),
                place.data_ptr(), at, nbytes)
    return offsets, order, place


def group_gather(X, place, out=None):
    """Xs [T * slots, D] with Xs[place[t, j]] = X[t]: the rows of X (elements of 1, 2
    or 4 bytes) in sorted order.  Rows behind the last slot that takes part are
    not written.  The gradient of X is group_combine(dXs, place)."""
    fn = "group_gather"
    if not isinstance(X, _pt.Tensor) or X.element_size() not in (1, 2, 4):
        _refuse(fn, "X", "a tensor of 1-, 2- or 4-byte elements")
    T, D, ldx = _matrix(fn, "X", X, X.dtype)
    T, k = _place(fn, place, T)
    if out is None:
        out = _new((T * k, D), (D, 1), dtype=X.dtype, device=X.device)
    _, _, ldo = _matrix(fn, "out", out, X.dtype, T * k, D)
    dev = _one_device(fn, "X place out", X, place, out)
    _group_call(fn, dev, X.data_ptr(), ldx, place.data_ptr(), T, k, D, X.element_size(), out.data_ptr(), ldo)
    return out


def group_combine(Y, place, weights=None, out=None):
    """out [T, D] with out[t] = sum_j weights[t, j] * Y[place[t, j]] (Y bf16 [T * slots,
    D], weights float32 [T, slots] or None for 1), in fp32, rounded once; slots that
    take no part are left out."""
    fn = "group_combine"
    T, k = _place(fn, place)
    _, D, ldy = _matrix(fn, "Y", Y, _BF16, T * k)
    ldw = 0 if weights is None else _matrix(fn, "weights", weights, _F32, T, k)[2]
    if out is None:
        out = _new((T, D), (D, 1), dtype=_BF16, device=Y.device)
    _, _, ldo = _matrix(fn, "out", out, _BF16, T, D)
    dev = _one_device(fn, "Y place weights out", Y, place, weights, out)
    _group_call(fn, dev, Y.data_ptr(), ldy, place.data_ptr(), _ptr(weights), ldw, T, k, D, out.data_ptr(), ldo)
    return out


def group_combine_grad(dout, Y, place, weights=None, *, need_dY: bool = True, need_dweights: bool = True,
                       dY=None):
    """The gradients of group_combine for dout bf16 [T, D]: (dY bf16 [T * slots, D],
    dweights float32 [T, slots]), None for one that is not needed.  Rows of dY
    behind the last slot that takes part are not written; dY may be Y itself.  Y is
    used for dweights only (None if not needed)."""
    fn = "group_combine_grad"
    T, k = _place(fn, place)
    _, D, ldd = _matrix(fn, "dout", dout, _BF16, T)
    ldy = 0
    if need_dweights or Y is not None:
        ldy = _matrix(fn, "Y", Y, _BF16, T * k, D)[2]
    ldw = 0 if weights is None else _matrix(fn, "weights", weights, _F32, T, k)[2]
    if not need_dY and not need_dweights:
        raise ValueError(f"{fn}: neither dY nor dweights is asked for")
    lddy, dweights = 0, None
    if need_dY:
        if dY is None:
            dY = _new((T * k, D), (D, 1), dtype=_BF16, device=dout.device)
        lddy = _matrix(fn, "dY", dY, _BF16, T * k, D)[2]
    elif dY is not None:
        raise ValueError(f"{fn}: dY given, but need_dY is false")
    dev = _one_device(fn, "dout Y place weights dY", dout, Y, place, weights, dY)
    if need_dweights:
        dweights = _new((T, k), (k, 1), dtype=_F32, device=dout.device)
    _group_call(fn, dev, dout.data_ptr(), ldd, _ptr(Y), ldy, place.data_ptr(), _ptr(weights), ldw, T, k, D,
                _ptr(dY), lddy, _ptr(dweights))
    return dY, dweights


def _group_order(fn: str, order, T: int, slots: int):
    if order is None:
        if slots != 1:
            raise ValueError(f"{fn}: slots needs an order")
    else:
        if slots < 1:
            raise ValueError(f"{fn}: slots must be at least 1")
        _vector(fn, "order", order, _I32, T * slots)


def group_linear(X, W, offsets, order=None, *, slots: int = 1, activation=None, mul=None, out=None):
    """Y [S, N] with Y[p] = act(x W[g]^T) * mul[p] for the rows p of group g, offsets[g] <=
    p < offsets[g + 1]; W bf16 [groups, N, K] as it lies in memory.  x is X[order[p] //
    slots] (X bf16 [T, K] of less than 2 GiB, S = T * slots; no sorted copy is made), or
    X[p] without an order (X sorted, S = T).  activation: one of ACTIVATIONS; mul bf16 [S, N], which
    may be `out` itself.  Rows from offsets[-1] on are not written."""
    fn = "group_linear"
    T, K, ldx = _matrix(fn, "X", X, _BF16)
    G, N, _, ldw, strw = _stack(fn, "W", W, _BF16, None, None, K)
    _vector(fn, "offsets", offsets, _I32, G + 1)
    _group_order(fn, order, T, slots)
    S = T * slots
    act = activation if isinstance(activation, int) else \
        ACTIVATIONS.get(activation) if activation is None or isinstance(activation, str) else None
    if act is None:
        _refuse(fn, "activation", "one of " + ", ".join(str(a) for a in ACTIVATIONS))
    ldm = 0 if mul is None else _matrix(fn, "mul", mul, _BF16, S, N)[2]
    if out is None:
        out = _new((S, N), (N, 1), dtype=_BF16, device=X.device)
    ldo = _matrix(fn, "out", out, _BF16, S, N)[2]
    dev = _one_device(fn, "X W offsets order mul out", X, W, offsets, order, mul, out)
    _group_call(fn, dev, X.data_ptr(), ldx, W.data_ptr(), ldw, strw, offsets.data_ptr(), _ptr(order), T, slots, G,
                N, K, act, _ptr(mul), ldm, out.data_ptr(), ldo)
    return out


def group_linear_grad(dY, X, W, offsets, order=None, *, slots: int = 1, need_dX: bool = True,
                      need_dW: bool = True, dX=None, dW=None, workspace=None):
    """The gradients of group_linear without activation and mul, for dY bf16 [S, N] in
    sorted order: (dX bf16 [S, K], sorted, dW bf16 like W), None for one that is not
    needed.  group_combine(dX, place) joins the rows of a token.  Rows of dX from
    offsets[-1] on are not written; dW is zero for a group without rows.  workspace:
    a uint8 tensor of group_linear_grad_workspace_bytes bytes (with an order, for dW)."""
    fn = "group_linear_grad"
    T, K, ldx = _matrix(fn, "X", X, _BF16)
    G, N, _, ldw, strw = _stack(fn, "W", W, _BF16, None, None, K)
    _vector(fn, "offsets", offsets, _I32, G + 1)
    _group_order(fn, order, T, slots)
    S = T * slots
    lddy = _matrix(fn, "dY", dY, _BF16, S, N)[2]
    if not need_dX and not need_dW:
        raise ValueError(f"{fn}: neither dX nor dW is asked for")
    for name, need, given in (("dX", need_dX, dX), ("dW", need_dW, dW)):
        if given is not None and not need:
            raise ValueError(f"{fn}: {name} given, but need_{name} is false")
    lddx, ld_dw = 0, (0, 0)
    if need_dX:
        if dX is None:
            dX = _new((S, K), (K, 1), dtype=_BF16, device=X.device)
        lddx = _matrix(fn, "dX", dX, _BF16, S, K)[2]
    if need_dW:
        if dW is None:
            dW = _new((G, N, K), (N * K, K, 1), dtype=_BF16, device=X.device)
        ld_dw = _stack(fn, "dW", dW, _BF16, G, N, K)[3:]
    dev = _one_device(fn, "X W offsets order dY dX dW", X, W, offsets, order, dY, dX, dW)
    need = lib.group_linear_grad_workspace_bytes(T, slots, K) if need_dW and order is not None else 0
    ws, at, nbytes = _group_workspace(fn, X.device, need, workspace) if need else (None, None, 0)
    _group_call(fn, dev, dY.data_ptr(), lddy, X.data_ptr(), ldx, W.data_ptr(), ldw, strw, offsets.data_ptr(),
                _ptr(order), T, slots, G, N, K, _ptr(dX), lddx, _ptr(dW), *ld_dw, at, nbytes)
    return dX, dW


def linear_adapters(X, W, A, B, offsets, order, *, scale=None, out=None, workspace=None):
    """Y [T, N] = X W^T, plus scale[g] * (X A[g]^T) B[g]^T in the rows of group g: one
    shared projection (W bf16 [N, K]) and the low-rank adapters of many requests
    (A bf16 [groups, R, K], B bf16 [groups, N, R], scale float32 [groups] or None for 1).
    offsets and order as group_sort(adapter of each row, groups) gives them; rows of
    no adapter get the projection alone.  X of 2 GiB or more goes in pieces of rows, each
    sorted by itself.  workspace: a uint8 tensor of linear_adapters_workspace_bytes bytes."""
    fn = "linear_adapters"
    T, K, ldx = _matrix(fn, "X", X, _BF16)
    N, _, ldw = _matrix(fn, "W", W, _BF16, None, K)
    G, R, _, lda, stra = _stack(fn, "A", A, _BF16, None, None, K)
    _, _, _, ldb, strb = _stack(fn, "B", B, _BF16, G, N, R)
    _vector(fn, "offsets", offsets, _I32, G + 1)
    _vector(fn, "order", order, _I32, T)
    if scale is not None:
        _vector(fn, "scale", scale, _F32, G)
    if out is None:
        out = _new((T, N), (N, 1), dtype=_BF16, device=X.device)
    ldo = _matrix(fn, "out", out, _BF16, T, N)[2]
    dev = _one_device(fn, "X W A B offsets order scale out", X, W, A, B, offsets, order, scale, out)
    ws, at, nbytes = _group_workspace(fn, X.device, lib.linear_adapters_workspace_bytes(T, R, G), workspace)
    _group_call(fn, dev, X.data_ptr(), ldx, W.data_ptr(), ldw, A.data_ptr(), lda, stra, B.data_ptr(), ldb, strb,
                _ptr(scale), offsets.data_ptr(), order.data_ptr(), T, N, K, R, G, out.data_ptr(), ldo, at, nbytes)
    return out
