"""MI355X (gfx950) prover for fixed-point linear layers: the witness of each
quantized matmul and the sum-check proof of its claim over Goldilocks.

This module is the thin binding over ``libfp.so`` (declared in
``include/fp.h``): it marshals torch tensors into device pointers and the
current HIP stream, and nothing else. Every step runs in the library's HIP
kernels; there is no CPU fallback. Field elements travel as int64 tensors
holding the raw 64-bit patterns of canonical values in [0, p).
"""
from __future__ import annotations

import ctypes
import os

import torch

P = 0xFFFFFFFF00000001
FP_I8, FP_I32, FP_F32, FP_F16, FP_BF16 = 0, 1, 2, 3, 4
MAX_GROUPS = 256  # FP_MAX_GROUPS
HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfp.so")
EXPORTS = [
    "fp_last_error", "fp_witness_linear", "fp_witness_linear_grouped", "fp_moe_plan", "fp_gather_rows",
    "fp_eq_table", "fp_eq_table_batched", "fp_eq_table_batched_workspace",
    "fp_fold_matrix", "fp_fold_matrix_workspace", "fp_fold_matrix_batched", "fp_fold_matrix_batched_workspace",
    "fp_mle_eval", "fp_mle_eval_workspace", "fp_sumcheck_prove", "fp_sumcheck_workspace",
    "fp_sumcheck_prove_multi", "fp_combine_claims", "fp_claim_eval_batched", "fp_claim_eval_batched_workspace",
    "fp_linear_combine", "fp_fold_claim_batched", "fp_fold_claim_batched_workspace",
    "fp_witness_linear_with_sumcheck", "fp_fold_weights_prepare", "fp_fold_matrix_multi",
    "fp_fold_matrix_multi_workspace", "fp_commit_pack", "fp_rs_encode", "fp_rs_encode_workspace",
    "fp_merkle_commit", "fp_lookup_tree", "fp_lookup_counts", "fp_sumcheck3_prove", "fp_sumcheck3_workspace",
    "fp_lookup_prove", "fp_lookup_prove_workspace", "fp_fs_init", "fp_fs_absorb", "fp_fs_challenges",
    "fp_eq_table_ext", "fp_ext_claim_combine", "fp_sumcheck_ext_fs", "fp_witness_packed_weights_bytes",
    "fp_witness_pack_weights", "fp_witness_linear_packed", "fp_witness_linear_packed_with_sumcheck",
    "fp_layer_step", "fp_layer_step_workspace", "fp_witness_multi", "fp_witness_multi_workspace",
    "fp_witness_multi_noalloc", "fp_layer_step_multi", "fp_layer_step_multi_workspace",
    "fp_witness_grouped_packed", "fp_witness_grouped_packed_workspace",
    "fp_sumcheck_ext_fs_multi", "fp_sumcheck_ext_fs_multi_workspace", "fp_commit_tables", "fp_commit_fold_ext",
    "fp_commit_fold_ext_workspace", "fp_merkle_open", "fp_lookup_tree_pairs", "fp_lookup_counts_field",
    "fp_quantize_rows", "fp_scaled_matmul", "fp_scaled_linear", "fp_scaled_linear_workspace", "fp_scaled_matmul_grouped",
    "fp_moe_sort", "fp_moe_sort_workspace", "fp_moe_permute", "fp_moe_dispatch", "fp_moe_combine",
    "fp_moe_combine_backward", "fp_moe_layer", "fp_moe_layer_workspace", "fp_rms_norm", "fp_rms_norm_backward",
    "fp_rms_norm_backward_workspace", "fp_token_logprobs", "fp_token_logprobs_workspace", "fp_token_logprobs_backward",
]

_lib = None


class FPError(RuntimeError):
    pass


class _EqDesc(ctypes.Structure):
    _fields_ = [("r", ctypes.c_void_p), ("n", ctypes.c_int32), ("E", ctypes.c_void_p)]


class _ClaimDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_void_p), ("ld", ctypes.c_int64), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("E_rows", ctypes.c_void_p), ("E_cols", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class _TableDesc(ctypes.Structure):
    _fields_ = [("Z", ctypes.c_void_p), ("ldz", ctypes.c_int64), ("T", ctypes.c_int32), ("d_out", ctypes.c_int32),
                ("n_o", ctypes.c_int32), ("row_q", ctypes.c_int32), ("row_r", ctypes.c_int32),
                ("row_y", ctypes.c_int32)]


class _OpenClaim(ctypes.Structure):
    _fields_ = [("row0", ctypes.c_int32), ("nrows", ctypes.c_int32), ("z1", ctypes.c_void_p), ("n1", ctypes.c_int32),
                ("z2", ctypes.c_void_p), ("n2", ctypes.c_int32)]


class _MatmulDesc(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("T", ctypes.c_int32), ("d_in", ctypes.c_int32),
                ("d_out", ctypes.c_int32), ("Wp", ctypes.c_void_p), ("Z", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("R", ctypes.c_void_p), ("E_t", ctypes.c_void_p), ("E_o", ctypes.c_void_p), ("claim", ctypes.c_void_p)]


class _SumcheckDesc(ctypes.Structure):
    _fields_ = [("n_pairs", ctypes.c_int32), ("n", ctypes.c_int32), ("A", ctypes.c_void_p * 8),
                ("B", ctypes.c_void_p * 8), ("rho", ctypes.c_void_p), ("r", ctypes.c_void_p),
                ("rounds", ctypes.c_void_p), ("finals", ctypes.c_void_p), ("claim0", ctypes.c_void_p)]


class _FoldDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_void_p), ("ld", ctypes.c_int64), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("cols_pad", ctypes.c_int32), ("E", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("E2", ctypes.c_void_p), ("out2", ctypes.c_void_p)]


def _fold_desc(f):
    """(M, E, cols_pad, out) or, in the step launches, (M, E, cols_pad, out, E2, out2): M folded by E into
    out and by E2 into out2 from one read."""
    M, E, cp, out = f[:4]
    E2, out2 = f[4:6] if len(f) > 4 else (None, None)
    return _FoldDesc(M.data_ptr(), _ld(M), M.shape[0], M.shape[1], cp, E.data_ptr(), out.data_ptr(), _ptr(E2),
                     _ptr(out2))


def lib():
    """Load libfp.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FPError("libfp.so is not built (run __graft_entry__.build()): %s" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint64
        f32 = ctypes.c_float
        sig = {
            "fp_last_error": (ctypes.c_char_p, []),
            "fp_witness_linear": (ctypes.c_int, [vp, i64, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp]),
            "fp_witness_linear_grouped": (ctypes.c_int, [vp, i64, vp, i64, vp, i32, i32, i32, i32, vp, vp, vp, vp]),
            "fp_moe_plan": (ctypes.c_int, [vp, i32, i32, vp, vp, vp]),
            "fp_gather_rows": (ctypes.c_int, [vp, i64, vp, i32, i32, vp, vp]),
            "fp_eq_table": (ctypes.c_int, [vp, i32, vp, vp]),
            "fp_eq_table_batched": (ctypes.c_int, [i32, vp, vp, sz, vp]),
            "fp_eq_table_batched_workspace": (sz, [i32]),
            "fp_fold_matrix": (ctypes.c_int, [i32, vp, i64, i32, i32, vp, vp, i32, vp, sz, vp]),
            "fp_fold_matrix_workspace": (sz, [i32, i32, i32]),
            "fp_fold_matrix_batched": (ctypes.c_int, [i32, i32, vp, vp, sz, vp]),
            "fp_fold_matrix_batched_workspace": (sz, [i32, i32, vp]),
            "fp_mle_eval": (ctypes.c_int, [i32, vp, i64, i32, i32, vp, i32, vp, i32, vp, vp, sz, vp]),
            "fp_mle_eval_workspace": (sz, [i32, i32, i32, i32, i32]),
            "fp_sumcheck_prove": (ctypes.c_int, [i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "fp_sumcheck_workspace": (sz, [i32, i32]),
            "fp_sumcheck_prove_multi": (ctypes.c_int, [i32, i32, vp, vp, vp, vp, vp, vp, vp]),
            "fp_combine_claims": (ctypes.c_int, [i32, vp, vp, vp, vp, vp]),
            "fp_claim_eval_batched": (ctypes.c_int, [i32, i32, vp, vp, sz, vp]),
            "fp_claim_eval_batched_workspace": (sz, [i32, i32, vp]),
            "fp_linear_combine": (ctypes.c_int, [i32, vp, vp, vp, vp]),
            "fp_fold_claim_batched": (ctypes.c_int, [i32, i32, vp, i32, i32, vp, vp, sz, vp]),
            "fp_fold_claim_batched_workspace": (sz, [i32, i32, vp, i32, i32, vp]),
            "fp_witness_linear_with_sumcheck": (ctypes.c_int, [vp, i64, vp, i64, i32, i32, i32, i32, vp, vp, vp,
                                                               i32, vp, vp, vp, i32, vp, vp, vp, vp, vp]),
            "fp_fold_weights_prepare": (ctypes.c_int, [vp, i64, i32, i32, vp, i64, vp, vp]),
            "fp_fold_matrix_multi": (ctypes.c_int, [vp, i64, vp, i32, i32, i32, vp, i64, vp, i64, i32, vp, sz, vp]),
            "fp_fold_matrix_multi_workspace": (sz, [i32, i32, i32]),
            "fp_commit_pack": (ctypes.c_int, [vp, i64, vp, i64, i32, i32, vp, vp]),
            "fp_rs_encode": (ctypes.c_int, [vp, i64, i32, i32, vp, i64, vp, sz, vp]),
            "fp_rs_encode_workspace": (sz, [i32, i32]),
            "fp_merkle_commit": (ctypes.c_int, [vp, i64, i32, i32, vp, vp, vp]),
            "fp_lookup_tree": (ctypes.c_int, [vp, i64, i32, vp, vp, vp]),
            "fp_lookup_counts": (ctypes.c_int, [vp, i64, i32, i32, vp, vp]),
            "fp_sumcheck3_prove": (ctypes.c_int, [vp, vp, i32, vp, vp, vp, vp, sz, vp]),
            "fp_sumcheck3_workspace": (sz, [i32]),
            "fp_lookup_prove": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, sz, vp]),
            "fp_lookup_prove_workspace": (sz, [i32]),
            "fp_fs_init": (ctypes.c_int, [vp, ctypes.c_char_p, i32, vp]),
            "fp_fs_absorb": (ctypes.c_int, [vp, vp, i32, vp]),
            "fp_fs_challenges": (ctypes.c_int, [vp, i32, vp, vp]),
            "fp_eq_table_ext": (ctypes.c_int, [vp, i32, vp, vp, vp]),
            "fp_ext_claim_combine": (ctypes.c_int, [vp, vp, vp]),
            "fp_sumcheck_ext_fs": (ctypes.c_int, [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp]),
            "fp_witness_packed_weights_bytes": (sz, [i32, i32]),
            "fp_witness_pack_weights": (ctypes.c_int, [vp, i64, i32, i32, vp, vp]),
            "fp_witness_linear_packed": (ctypes.c_int, [vp, i64, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp]),
            "fp_witness_linear_packed_with_sumcheck": (ctypes.c_int, [vp, i64, vp, i32, i32, i32, i32, vp, vp, vp,
                                                                      i32, vp, vp, vp, i32, vp, vp, vp, vp, i32, vp,
                                                                      vp]),
            "fp_layer_step": (ctypes.c_int, [vp, i64, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, i32, vp, i32, vp,
                                             i32, vp, vp, sz, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp]),
            "fp_witness_multi": (ctypes.c_int, [i32, vp, i32, i32, i32, vp, vp, sz, vp]),
            "fp_witness_multi_workspace": (sz, [i32, vp]),
            "fp_witness_multi_noalloc": (ctypes.c_int, [i32, vp, i32, i32, i32, vp, vp]),
            "fp_layer_step_multi": (ctypes.c_int, [i32, vp, i32, i32, i32, vp, i32, vp, i32, vp, vp, sz, vp]),
            "fp_layer_step_multi_workspace": (sz, [i32, vp, i32, vp, i32, vp]),
            "fp_witness_grouped_packed": (ctypes.c_int, [vp, i64, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, i64,
                                                         vp, vp, i64, i32, vp, sz, vp]),
            "fp_witness_grouped_packed_workspace": (sz, [vp, i32, i32, i32, i32]),
            "fp_layer_step_workspace": (sz, [i32, i32, i32, i32, vp, i32, vp]),
            "fp_sumcheck_ext_fs_multi": (ctypes.c_int, [i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "fp_sumcheck_ext_fs_multi_workspace": (sz, [i32, i32]),
            "fp_commit_tables": (ctypes.c_int, [i32, vp, i32, i32, i32, vp, i64, i32, vp]),
            "fp_commit_fold_ext": (ctypes.c_int, [vp, i64, i32, i32, vp, i32, i32, vp, vp, vp, sz, vp]),
            "fp_commit_fold_ext_workspace": (sz, [i32]),
            "fp_merkle_open": (ctypes.c_int, [vp, i64, i32, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp]),
            "fp_lookup_tree_pairs": (ctypes.c_int, [vp, vp, i64, u64, u64, i32, vp, vp, vp]),
            "fp_lookup_counts_field": (ctypes.c_int, [vp, i64, i64, i32, vp, vp]),
            "fp_quantize_rows": (ctypes.c_int, [i32, vp, i64, i32, i32, vp, i64, vp, vp]),
            "fp_scaled_matmul": (ctypes.c_int, [vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, i64, vp]),
            "fp_scaled_linear": (ctypes.c_int, [i32, vp, i64, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, i64, vp, sz,
                                                vp]),
            "fp_scaled_linear_workspace": (sz, [i32, i32]),
            "fp_scaled_matmul_grouped": (ctypes.c_int, [vp, i64, vp, i32, vp, i32, vp, vp, vp, i64, vp, i32, i32, i32,
                                                        i32, vp, i64, vp, i64, vp]),
            "fp_moe_sort": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "fp_moe_sort_workspace": (sz, [i32, i32, i32]),
            "fp_moe_permute": (ctypes.c_int, [i32, vp, i64, i32, i32, i32, vp, vp, i64, vp]),
            "fp_moe_dispatch": (ctypes.c_int, [i32, vp, i64, i32, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, i64, vp,
                                               sz, vp]),
            "fp_moe_combine": (ctypes.c_int, [i32, vp, i64, i32, vp, vp, i32, i32, i32, vp, i64, vp]),
            "fp_moe_combine_backward": (ctypes.c_int, [i32, vp, i64, vp, i64, i32, vp, vp, i32, i32, i32, vp, i64, vp,
                                                       vp]),
            "fp_moe_layer": (ctypes.c_int, [i32, vp, i64, vp, vp, i32, vp, i32, i32, i32, vp, vp, i64, vp, vp, i64, vp, vp,
                                            i64, i32, i32, i32, vp, i64, vp, sz, vp]),
            "fp_moe_layer_workspace": (sz, [i32, i32, i32, i32]),
            "fp_rms_norm": (ctypes.c_int, [i32, vp, i64, vp, i64, i32, vp, f32, i32, i32, vp, i64, vp, i64, vp, i64, vp,
                                           vp]),
            "fp_rms_norm_backward": (ctypes.c_int, [i32, vp, i64, vp, i64, i32, vp, f32, vp, i64, i32, i32, vp, i64, vp, vp,
                                                    sz, vp]),
            "fp_rms_norm_backward_workspace": (sz, [i32, i32]),
            "fp_token_logprobs": (ctypes.c_int, [i32, vp, i64, i32, i32, vp, i32, f32, i32, vp, vp, vp, vp, vp, vp, vp, sz,
                                                 vp]),
            "fp_token_logprobs_workspace": (sz, [i32, i32, i32, i32]),
            "fp_token_logprobs_backward": (ctypes.c_int, [i32, vp, i64, i32, i32, vp, i32, f32, vp, vp, vp, vp, vp, vp, i64,
                                                          vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def require_gpu():
    """Raise unless a GPU and the built library are both present."""
    if not torch.cuda.is_available():
        raise FPError("no GPU visible: the prover runs only on the GPU")
    lib()


def _check(rc: int, name: str):
    if rc != 0:
        raise FPError("%s failed (code %d): %s" % (name, rc, lib().fp_last_error().decode()))


def _ptr(t) -> int | None:
    if t is None:
        return None
    assert t.is_cuda, "device tensor expected"
    return t.data_ptr()


def _need(t, dtype, numel: int, name: str):
    """Check a buffer handed to the library: its dtype, contiguity and at least
    numel elements (a short buffer would be written past its end on the device)."""
    if t is None:
        raise ValueError("%s: missing buffer" % name)
    if t.dtype != dtype:
        raise ValueError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.numel() and not t.is_contiguous():
        raise ValueError("%s: must be contiguous" % name)
    if t.numel() < numel:
        raise ValueError("%s: %d elements, at least %d needed" % (name, t.numel(), numel))


def _ld(M) -> int:
    """Leading dimension of a row-major 2-D tensor (any value >= cols when it has <= 1 row)."""
    return M.stride(0) if M.shape[0] > 1 else max(M.stride(0), M.shape[1])


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


# the same without a Stream object (4 us a call), where torch offers it
_device_index = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


class Workspace:
    """A growable device scratch buffer; each entry-point family keeps its own
    (calls on one stream run in order, so a family may reuse its buffer)."""

    def __init__(self):
        self.buf = None

    def get(self, nbytes: int):
        if nbytes == 0:
            return None, 0
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=_dev())
        return self.buf.data_ptr(), self.buf.numel()


_ws_fold, _ws_claim, _ws_mle, _ws_sc = Workspace(), Workspace(), Workspace(), Workspace()
_ws_multi, _ws_rs, _ws_lookup = Workspace(), Workspace(), Workspace()
_ws_open, _ws_scx = Workspace(), Workspace()


def to_field_tensor(vals, device=None) -> torch.Tensor:
    """Field values (ints or a uint64 array) as a device int64 tensor."""
    import numpy as np
    a = np.ascontiguousarray(np.asarray(vals, dtype=np.uint64)).view(np.int64)
    return torch.from_numpy(a.copy()).to(device or _dev())


def field_numpy(t: torch.Tensor):
    """A device int64 field tensor as a numpy uint64 array."""
    return t.detach().cpu().numpy().view("uint64")


# ------------------------------------------------------------------ witness --
def witness_linear(X, W, s: int, Z=None, Y=None, R=None, with_z: bool = True):
    T, d_in = X.shape
    d_out = W.shape[0]
    assert X.dtype == torch.int8 and W.dtype == torch.int8
    assert (X.numel() == 0 or X.stride(1) == 1) and (W.numel() == 0 or W.stride(1) == 1), "rows must be contiguous"
    if with_z and Z is None:
        Z = torch.empty((T, d_out), dtype=torch.int32, device=X.device)
    Y = torch.empty((T, d_out), dtype=torch.int8, device=X.device) if Y is None else Y
    R = torch.empty((T, d_out), dtype=torch.int8, device=X.device) if R is None else R
    _check(lib().fp_witness_linear(_ptr(X), _ld(X), _ptr(W), _ld(W), T, d_in, d_out, s,
                                   _ptr(Z) if with_z else None, _ptr(Y), _ptr(R), _stream()),
           "fp_witness_linear")
    return Z, Y, R


def witness_linear_with_sumcheck(X, W, s: int, Z, Y, R, As, Bs, r, rho=None, rounds=None, finals=None, claim0=None):
    """witness_linear(X, W, s, Z, Y, R) and sumcheck_prove(As, Bs, r, rho, ...) in one launch."""
    T, d_in = X.shape
    d_out = W.shape[0]
    assert X.dtype == torch.int8 and W.dtype == torch.int8
    assert (X.numel() == 0 or X.stride(1) == 1) and (W.numel() == 0 or W.stride(1) == 1), "rows must be contiguous"
    k = len(As)
    n = r.numel()
    dev = r.device
    rounds = torch.empty((n, 3), dtype=torch.int64, device=dev) if rounds is None else rounds
    finals = torch.empty((k, 2), dtype=torch.int64, device=dev) if finals is None else finals
    claim0 = torch.empty(1, dtype=torch.int64, device=dev) if claim0 is None else claim0
    pa = (ctypes.c_void_p * k)(*[a.data_ptr() for a in As])
    pb = (ctypes.c_void_p * k)(*[b.data_ptr() for b in Bs])
    _check(lib().fp_witness_linear_with_sumcheck(_ptr(X), _ld(X), _ptr(W), _ld(W), T, d_in, d_out, s, _ptr(Z),
                                                 _ptr(Y), _ptr(R), k, pa, pb, _ptr(rho), n, _ptr(r), _ptr(rounds),
                                                 _ptr(finals), _ptr(claim0), _stream()),
           "fp_witness_linear_with_sumcheck")
    return (Z, Y, R), (rounds, finals, claim0)


class PackedWeights:
    """The weights of one layer packed for the matrix cores (fp_witness_pack_weights):
    ``data`` is the packed int8 buffer, ``d_out`` and ``d_in`` the shape of W."""

    def __init__(self, data: torch.Tensor, d_out: int, d_in: int):
        self.data, self.d_out, self.d_in = data, d_out, d_in


def pack_weights(W, out: PackedWeights | None = None) -> PackedWeights:
    d_out, d_in = W.shape
    assert W.dtype == torch.int8 and (W.numel() == 0 or W.stride(1) == 1), "rows must be contiguous"
    nbytes = lib().fp_witness_packed_weights_bytes(d_out, d_in)
    if out is not None:
        assert (out.d_out, out.d_in) == (d_out, d_in) and out.data.numel() >= nbytes
        Wp = out.data
    else:
        Wp = torch.empty(max(nbytes, 16), dtype=torch.int8, device=W.device)
    _check(lib().fp_witness_pack_weights(_ptr(W), _ld(W), d_out, d_in, _ptr(Wp), _stream()),
           "fp_witness_pack_weights")
    return PackedWeights(Wp, d_out, d_in)


def _eq_descs(eq):
    """fp_eq_desc array of (r, E) pairs (None: no tables)."""
    eq = list(eq or [])
    return len(eq), (_EqDesc * max(len(eq), 1))(*[_EqDesc(r.data_ptr() if r.numel() else None, r.numel(),
                                                          E.data_ptr()) for r, E in eq])


def witness_linear_packed(X, Wp: PackedWeights, s: int, Z=None, Y=None, R=None, with_z: bool = True, eq=None):
    """witness_linear(X, W, s) with W given packed (pack_weights(W)); eq: (r, E) pairs of eq tables
    written by the same launch (eq_table_batched of them)."""
    T, d_in = X.shape
    assert X.dtype == torch.int8 and d_in == Wp.d_in
    assert X.numel() == 0 or X.stride(1) == 1, "rows must be contiguous"
    d_out = Wp.d_out
    if with_z and Z is None:
        Z = torch.empty((T, d_out), dtype=torch.int32, device=X.device)
    Y = torch.empty((T, d_out), dtype=torch.int8, device=X.device) if Y is None else Y
    R = torch.empty((T, d_out), dtype=torch.int8, device=X.device) if R is None else R
    ne, descs = _eq_descs(eq)
    _check(lib().fp_witness_linear_packed(_ptr(X), _ld(X), _ptr(Wp.data), T, d_in, d_out, s,
                                          _ptr(Z) if with_z else None, _ptr(Y), _ptr(R), ne, descs, _stream()),
           "fp_witness_linear_packed")
    return Z, Y, R


def witness_linear_packed_with_sumcheck(X, Wp: PackedWeights, s: int, Z, Y, R, As, Bs, r, rho=None, rounds=None,
                                        finals=None, claim0=None, eq=None):
    """witness_linear_packed(X, Wp, s, Z, Y, R, eq=eq) and sumcheck_prove(As, Bs, r, rho, ...) in one launch."""
    T, d_in = X.shape
    assert X.dtype == torch.int8 and d_in == Wp.d_in
    assert X.numel() == 0 or X.stride(1) == 1, "rows must be contiguous"
    k = len(As)
    n = r.numel()
    dev = r.device
    rounds = torch.empty((n, 3), dtype=torch.int64, device=dev) if rounds is None else rounds
    finals = torch.empty((k, 2), dtype=torch.int64, device=dev) if finals is None else finals
    claim0 = torch.empty(1, dtype=torch.int64, device=dev) if claim0 is None else claim0
    pa = (ctypes.c_void_p * k)(*[a.data_ptr() for a in As])
    pb = (ctypes.c_void_p * k)(*[b.data_ptr() for b in Bs])
    _check(lib().fp_witness_linear_packed_with_sumcheck(_ptr(X), _ld(X), _ptr(Wp.data), T, d_in, Wp.d_out, s,
                                                        _ptr(Z), _ptr(Y), _ptr(R), k, pa, pb, _ptr(rho), n, _ptr(r),
                                                        _ptr(rounds), _ptr(finals), _ptr(claim0), *_eq_descs(eq),
                                                        _stream()),
           "fp_witness_linear_packed_with_sumcheck")
    return (Z, Y, R), (rounds, finals, claim0)


class StepWorkspace:
    """Workspace of fp_layer_step: arrival counters (zeroed once, here) and the
    folds' partial values."""

    def __init__(self):
        self.buf = None

    def get(self, nbytes: int):
        if nbytes == 0:
            return None, 0
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=_dev())
        return self.buf.data_ptr(), self.buf.numel()


_ws_step = StepWorkspace()


def layer_step(X, Wp: PackedWeights, s: int, Z, Y, R, eq=None, folds=(), claims=(), As=(), Bs=(), r=None, rho=None,
               rounds=None, finals=None, claim0=None, ws: StepWorkspace | None = None, own_claim=None):
    """One launch: the witness and eq tables of a proof (as witness_linear_packed), the int8 folds
    (M, E, cols_pad, out[, E2, out2]) and int32 claims (M, E_rows, E_cols, out) of another (as fold_claim_batched), and
    the sum-check of a third (as sumcheck_prove over As, Bs, r; none when As is empty). own_claim =
    (E_t, E_o, out): the witness's own claim sum E_t[t] E_o[o] Z[t, o] from the accumulators (Z may then
    be None; E_t and E_o must be finished before the call)."""
    T, d_in = X.shape
    assert X.dtype == torch.int8 and d_in == Wp.d_in
    assert X.numel() == 0 or X.stride(1) == 1, "rows must be contiguous"
    ne, eqd = _eq_descs(eq)
    nf, nc = len(folds), len(claims)
    fd = (_FoldDesc * max(nf, 1))(*[_fold_desc(f) for f in folds])
    cd = (_ClaimDesc * max(nc, 1))(*[_ClaimDesc(M.data_ptr(), _ld(M), M.shape[0], M.shape[1], Er.data_ptr(),
                                                Ec.data_ptr(), out.data_ptr()) for (M, Er, Ec, out) in claims])
    ws = _ws_step if ws is None else ws
    cEt, cEo, cout = own_claim if own_claim is not None else (None, None, None)
    p, nb = ws.get(lib().fp_layer_step_workspace(T, Wp.d_out, int(own_claim is not None), nf, fd, nc, cd))
    k = len(As)
    pa = (ctypes.c_void_p * max(k, 1))(*[a.data_ptr() for a in As])
    pb = (ctypes.c_void_p * max(k, 1))(*[b.data_ptr() for b in Bs])
    n = r.numel() if r is not None else 0
    _check(lib().fp_layer_step(_ptr(X), _ld(X), _ptr(Wp.data), T, d_in, Wp.d_out, s, _ptr(Z), _ptr(Y), _ptr(R),
                               _ptr(cEt), _ptr(cEo), _ptr(cout),
                               ne, eqd, nf, fd, nc, cd, p, nb, k, pa, pb, _ptr(rho), n, _ptr(r), _ptr(rounds),
                               _ptr(finals), _ptr(claim0), _stream()), "fp_layer_step")


class MatmulJob:
    """One linear map of fp_witness_multi: X int8 [T, d_in], its packed weights, the outputs Y, R
    (and Z, or None) int8/int32 [T, d_out], and for the claim from the accumulators the eq tables
    E_t, E_o and the one-element claim output (all None: no claim)."""

    def __init__(self, X, Wp: PackedWeights, Y, R, Z=None, E_t=None, E_o=None, claim=None):
        self.X, self.Wp, self.Y, self.R, self.Z = X, Wp, Y, R, Z
        self.E_t, self.E_o, self.claim = E_t, E_o, claim


def _multi_descs(jobs):
    """fp_matmul_desc array of MatmulJobs (buffers checked)."""
    assert len(jobs) > 0, "no maps"
    descs = []
    for j in jobs:
        T, d_in = j.X.shape
        assert j.X.dtype == torch.int8 and d_in == j.Wp.d_in and (j.X.numel() == 0 or j.X.stride(1) == 1)
        d_out = j.Wp.d_out
        _need(j.Y, torch.int8, T * d_out, "Y")
        _need(j.R, torch.int8, T * d_out, "R")
        if j.Z is not None:
            _need(j.Z, torch.int32, T * d_out, "Z")
        if j.E_t is not None:
            _need(j.E_t, torch.int64, T, "E_t")
            _need(j.E_o, torch.int64, d_out, "E_o")
            _need(j.claim, torch.int64, 1, "claim")
        descs.append(_MatmulDesc(_ptr(j.X), _ld(j.X), T, d_in, d_out, _ptr(j.Wp.data), _ptr(j.Z), _ptr(j.Y),
                                 _ptr(j.R), _ptr(j.E_t), _ptr(j.E_o), _ptr(j.claim)))
    return (_MatmulDesc * len(descs))(*descs)


def witness_multi(jobs, s: int, group_o: int = 1, eq=None, ws: StepWorkspace | None = None):
    """The witness GEMMs of several linear maps (MatmulJob) in one launch, each map's claim
    sum_t sum_o E_t[t] E_o[o] Z[t, o] taken from its accumulators; eq: (r, E) tables of another
    proof built by the same launch."""
    arr = _multi_descs(jobs)
    ne, eqd = _eq_descs(eq)
    ws = _ws_step if ws is None else ws
    p, nb = ws.get(lib().fp_witness_multi_workspace(len(jobs), arr))
    _check(lib().fp_witness_multi(len(jobs), arr, s, group_o, ne, eqd, p, nb, _stream()), "fp_witness_multi")


class SumcheckJob:
    """One sum-check instance of layer_step_multi: pairs of tables As[j], Bs[j] (int64 [2^n]), the round
    challenges r [n], weights rho [n_pairs] or None, outputs rounds [n, 3], finals [n_pairs, 2] and claim0 [1]
    (or None)."""

    def __init__(self, As, Bs, r, rounds, finals, claim0=None, rho=None):
        self.As, self.Bs, self.r, self.rounds, self.finals, self.claim0, self.rho = As, Bs, r, rounds, finals, claim0, rho


def _sc_descs(scs):
    out = []
    for j in scs:
        n, k = j.r.numel(), len(j.As)
        assert 1 <= k <= 8 and len(j.Bs) == k
        for t in list(j.As) + list(j.Bs):
            _need(t, torch.int64, 1 << n, "sum-check table")
        _need(j.r, torch.int64, n, "r")
        _need(j.rounds, torch.int64, 3 * n, "rounds")
        _need(j.finals, torch.int64, 2 * k, "finals")
        if j.rho is not None:
            _need(j.rho, torch.int64, k, "rho")
        d = _SumcheckDesc()
        d.n_pairs, d.n = k, n
        for i in range(k):
            d.A[i], d.B[i] = j.As[i].data_ptr(), j.Bs[i].data_ptr()
        d.rho, d.r, d.rounds, d.finals, d.claim0 = _ptr(j.rho), _ptr(j.r), _ptr(j.rounds), _ptr(j.finals), _ptr(j.claim0)
        out.append(d)
    return len(out), (_SumcheckDesc * max(len(out), 1))(*out)


def _fold_descs(folds):
    nf = len(folds)
    return nf, (_FoldDesc * max(nf, 1))(*[_fold_desc(f) for f in folds])


def layer_step_multi(jobs, s: int, group_o: int = 1, eq=None, folds=(), sumchecks=(), ws: StepWorkspace | None = None):
    """One launch: the witness GEMMs and claims of a proof's maps (as witness_multi), the int8 folds
    (M, E, cols_pad, out) of another proof (as fold_matrix_batched; (M, E, cols_pad, out, E2, out2) also
    folds M by E2 into out2 from the same read) and whole sum-check instances (SumcheckJob) of a third, side
    by side."""
    arr = _multi_descs(jobs)
    ne, eqd = _eq_descs(eq)
    nf, fd = _fold_descs(folds)
    ns, sd = _sc_descs(sumchecks)
    ws = _ws_step if ws is None else ws
    p, nb = ws.get(lib().fp_layer_step_multi_workspace(len(jobs), arr, nf, fd, ns, sd))
    _check(lib().fp_layer_step_multi(len(jobs), arr, s, group_o, ne, eqd, nf, fd, ns, sd, p, nb, _stream()),
           "fp_layer_step_multi")


def witness_multi_noalloc(jobs, s: int, group_o: int = 1, eq=None):
    """witness_multi without a workspace: the library's own scratch array holds the claims' slots and
    counters (calls that overlap on one GPU race)."""
    arr = _multi_descs(jobs)
    ne, eqd = _eq_descs(eq)
    _check(lib().fp_witness_multi_noalloc(len(jobs), arr, s, group_o, ne, eqd, _stream()), "fp_witness_multi_noalloc")


def witness_grouped_packed(Xg, Wps, row_off, s: int, Y, R, Z=None, E_ts=None, E_o=None, claims=None, w_fold=None,
                           ws: StepWorkspace | None = None):
    """Grouped witness from packed weights (Wps: PackedWeights per group), rows row_off (host ints, G + 1);
    with E_ts (per-group tables), E_o (int64 [G, >= d_out]) and claims (int64 [G]) every non-empty group's
    claim sum_t sum_o E_t[t] E_o[o] Z[t, o] from the accumulators; with w_fold (int64 [G, cols_pad], E_o
    given) every non-empty group's weight fold sum_o E_o[o] W[o, k] from the same pass over the weights."""
    G = len(Wps)
    T, d_in = Xg.shape
    d_out = Wps[0].d_out if G else 0
    assert Xg.dtype == torch.int8 and (Xg.numel() == 0 or Xg.stride(1) == 1) and len(row_off) == G + 1
    assert all(w.d_in == d_in and w.d_out == d_out for w in Wps) and row_off[-1] <= T
    _need(Y, torch.int8, row_off[-1] * d_out, "Y")
    _need(R, torch.int8, row_off[-1] * d_out, "R")
    if Z is not None:
        _need(Z, torch.int32, row_off[-1] * d_out, "Z")
    ro = (ctypes.c_int32 * (G + 1))(*row_off)
    wp = (ctypes.c_void_p * max(G, 1))(*[w.data.data_ptr() for w in Wps])
    et = None
    ldeo = 0
    p, nb = None, 0
    ld_fold, cols_pad = 0, 0
    if E_o is not None:
        assert E_o.dim() == 2 and E_o.shape[0] >= G and E_o.stride(1) == 1 and E_o.dtype == torch.int64
        assert E_o.shape[1] >= d_out
        ldeo = E_o.stride(0)
    if E_ts is not None:
        for g in range(G):
            if row_off[g + 1] > row_off[g]:
                _need(E_ts[g], torch.int64, row_off[g + 1] - row_off[g], "E_t")
        _need(claims, torch.int64, G, "claims")
        et = (ctypes.c_void_p * max(G, 1))(*[e.data_ptr() for e in E_ts])
    if w_fold is not None:
        assert w_fold.dim() == 2 and w_fold.shape[0] >= G and w_fold.stride(1) == 1 and w_fold.dtype == torch.int64
        ld_fold, cols_pad = w_fold.stride(0), w_fold.shape[1]
    if E_ts is not None or w_fold is not None:
        ws = _ws_step if ws is None else ws
        p, nb = ws.get(lib().fp_witness_grouped_packed_workspace(ro, G, d_in, d_out, int(w_fold is not None)))
    _check(lib().fp_witness_grouped_packed(_ptr(Xg), _ld(Xg), wp, ro, G, d_in, d_out, s, _ptr(Z), _ptr(Y), _ptr(R),
                                           et, _ptr(E_o), ldeo, _ptr(claims), _ptr(w_fold), ld_fold, cols_pad, p, nb,
                                           _stream()), "fp_witness_grouped_packed")


def witness_linear_grouped(Xg, Ws, row_off, s: int, Z=None, Y=None, R=None, with_z: bool = True):
    """Xg: int8 [row_off[-1], d_in]; Ws: list of int8 [d_out, d_in]; row_off: host ints (G+1)."""
    G = len(Ws)
    d_in = Xg.shape[1]
    d_out = Ws[0].shape[0]
    total = int(row_off[-1])
    if with_z and Z is None:
        Z = torch.empty((total, d_out), dtype=torch.int32, device=Xg.device)
    Y = torch.empty((total, d_out), dtype=torch.int8, device=Xg.device) if Y is None else Y
    R = torch.empty((total, d_out), dtype=torch.int8, device=Xg.device) if R is None else R
    wp = (ctypes.c_void_p * G)(*[w.data_ptr() for w in Ws])
    ro = (ctypes.c_int32 * (G + 1))(*[int(v) for v in row_off])
    _check(lib().fp_witness_linear_grouped(_ptr(Xg), _ld(Xg), wp, _ld(Ws[0]), ro, G, d_in, d_out, s,
                                           _ptr(Z) if with_z else None, _ptr(Y), _ptr(R), _stream()),
           "fp_witness_linear_grouped")
    return Z, Y, R


def moe_plan(route, n_experts: int):
    """Host-only grouping plan: (counts, offsets, perm) as numpy int32 arrays."""
    import numpy as np
    route = np.ascontiguousarray(route, dtype=np.int32)
    T = len(route)
    counts = np.empty(n_experts, np.int32)
    offsets = np.empty(n_experts + 1, np.int32)
    perm = np.empty(max(T, 1), np.int32)
    _check(lib().fp_moe_plan(route.ctypes.data, T, n_experts, counts.ctypes.data, offsets.ctypes.data,
                             perm.ctypes.data), "fp_moe_plan")
    return counts, offsets, perm[:T]


def gather_rows(X, perm_dev, out=None):
    n = perm_dev.numel()
    cols = X.shape[1]
    out = torch.empty((n, cols), dtype=X.dtype, device=X.device) if out is None else out
    _check(lib().fp_gather_rows(_ptr(X), _ld(X), _ptr(perm_dev), n, cols, _ptr(out), _stream()),
           "fp_gather_rows")
    return out


# ---------------------------------------------------------- scaled products --
_FLOATS = {torch.float32: FP_F32, torch.float16: FP_F16, torch.bfloat16: FP_BF16}


def _float_dt(dtype, name: str) -> int:
    dt = _FLOATS.get(dtype)
    if dt is None:
        raise ValueError("%s: dtype %s, expected float32, float16 or bfloat16" % (name, dtype))
    return dt


def _matrix(t, dtype, rows, cols: int, name: str) -> int:
    """Check a row-major device matrix: dtype (None: any), shape (rows None: any) and unit column stride; a matrix that
    is written (or read) row by row has rows that do not overlap. Returns its leading dimension."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise ValueError("%s: shape %s, expected (%s, %d)" % (name, tuple(shape), "*" if rows is None else rows, cols))
    if dtype is not None and t.dtype is not dtype:
        raise ValueError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    ld = stride[0]
    if shape[0] > 1:
        if cols and ((cols > 1 and stride[1] != 1) or ld < cols):
            raise ValueError("%s: rows must be contiguous and must not overlap" % name)
        return ld
    if cols > 1 and stride[1] != 1 and shape[0]:
        raise ValueError("%s: rows must be contiguous and must not overlap" % name)
    return max(ld, cols)


def _vector(t, dtype, shape, name: str):
    """Check a dense device array of this dtype and shape."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError("%s: %s %s, expected %s %s" % (name, t.dtype, tuple(t.shape), dtype, tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s: must be contiguous" % name)


def _here(*tensors) -> int:
    """The current device's current stream; every given tensor is on that device, where the call runs."""
    dev = _device_index()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensor on %s, the current device is cuda:%d" % (t.device, dev))
    return _raw_stream(dev)


def _whole_rows(X, ld: int) -> int:
    """X's rows, when they start on 16 bytes, are read in whole 16-byte chunks: the last row's must be in its storage.
    Returns the leading dimension to pass: a single row without the bytes for its last chunk is read to its end only."""
    T, d = X.shape
    up = (d + 15) // 16 * 16
    if up != d and T and ld >= up and ld % 16 == 0 and X.data_ptr() % 16 == 0:
        if X.storage_offset() + (T - 1) * ld + up > X.untyped_storage().nbytes():
            if T == 1:
                return d
            raise ValueError("X: the last row is read up to column %d, past its storage (copy X, or pad its rows)" % up)
    return ld


def _readable(X, ld: int):
    """X and the leading dimension that a product reads it with: where the last row's chunk is not in X's storage, a copy
    with padded rows."""
    try:
        return X, _whole_rows(X, ld)
    except ValueError:
        T, d = X.shape
        up = (d + 15) // 16 * 16
        copy = torch.empty((T, up), dtype=X.dtype, device=X.device)[:, :d]
        return copy.copy_(X), up


def quantize_rows(X, out=None, scale=None):
    """(Xq, scale): each row of X [T, d] (float32, float16 or bfloat16) as int8 with the scale max|x| / 127, rounded to
    the nearest (ties to even). Without ``out``, Xq's rows are a multiple of 16 bytes apart, so that the products read
    them in whole chunks."""
    if X.dim() != 2:
        raise ValueError("X: shape %s, expected two dimensions" % (tuple(X.shape),))
    T, d = X.shape
    dt = _float_dt(X.dtype, "X")
    ldx = _matrix(X, None, T, d, "X")
    if out is None:
        out = torch.empty((T, (d + 15) // 16 * 16), dtype=torch.int8, device=X.device)
        if d % 16:
            out = out[:, :d]
    ldq = _matrix(out, torch.int8, T, d, "out")
    if scale is None:
        scale = torch.empty(T, dtype=torch.float32, device=X.device)
    else:
        _vector(scale, torch.float32, (T,), "scale")
    st = _here(X, out, scale)
    _check(lib().fp_quantize_rows(dt, X.data_ptr(), ldx, T, d, out.data_ptr(), ldq, scale.data_ptr(), st),
           "fp_quantize_rows")
    return out, scale


def _product_out(T, d_out, out, dtype, Z, device):
    """out (made if None), its type, its leading dimension, Z's address and leading dimension."""
    if out is None:
        _float_dt(dtype, "out")
        out = torch.empty((T, d_out), dtype=dtype, device=device)
    ldy = _matrix(out, None, T, d_out, "out")
    dt = _float_dt(out.dtype, "out")
    if Z is None:
        return out, dt, ldy, 0, d_out
    return out, dt, ldy, Z.data_ptr(), _matrix(Z, torch.int32, T, d_out, "Z")


def scaled_matmul(X, x_scale, Wp: PackedWeights, w_scale, bias=None, out=None, dtype=torch.bfloat16, Z=None):
    """Y[t, o] = x_scale[t] w_scale[o] sum_k X[t, k] W[o, k] + bias[o] for int8 X [T, d_in] and packed weights, in
    ``out``'s type or ``dtype``; Z (int32 [T, d_out] or None) also receives the integer product, the layer's witness. The
    products have no gradients: what they return carries none, whatever the scales and the bias ask for."""
    d_in, d_out = Wp.d_in, Wp.d_out
    ldx = _matrix(X, torch.int8, None, d_in, "X")
    T = X.shape[0]
    _vector(x_scale, torch.float32, (T,), "x_scale")
    _vector(w_scale, torch.float32, (d_out,), "w_scale")
    if bias is not None:
        _vector(bias, torch.float32, (d_out,), "bias")
    out, dt, ldy, z, ldz = _product_out(T, d_out, out, dtype, Z, X.device)
    X, ldx = _readable(X, ldx)
    st = _here(X, x_scale, Wp.data, w_scale, bias, out, Z)
    _check(lib().fp_scaled_matmul(X.data_ptr(), ldx, x_scale.data_ptr(), Wp.data.data_ptr(), w_scale.data_ptr(),
                                  0 if bias is None else bias.data_ptr(), T, d_in, d_out, dt, out.data_ptr(), ldy, z,
                                  ldz, st), "fp_scaled_matmul")
    return out


def scaled_linear(X, Wp: PackedWeights, w_scale, bias=None, out=None, dtype=None, Z=None):
    """scaled_matmul of quantize_rows(X) for X [T, d_in] in float32, float16 or bfloat16; the answer is in ``out``'s
    type, ``dtype`` or X's."""
    d_in, d_out = Wp.d_in, Wp.d_out
    ldx = _matrix(X, None, None, d_in, "X")
    x_dt = _float_dt(X.dtype, "X")
    T = X.shape[0]
    _vector(w_scale, torch.float32, (d_out,), "w_scale")
    if bias is not None:
        _vector(bias, torch.float32, (d_out,), "bias")
    out, dt, ldy, z, ldz = _product_out(T, d_out, out, dtype or X.dtype, Z, X.device)
    st = _here(X, Wp.data, w_scale, bias, out, Z)
    nbytes = lib().fp_scaled_linear_workspace(T, d_in)
    # from the allocator each time, which keeps scratch of different streams and captured graphs apart
    ws = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    _check(lib().fp_scaled_linear(x_dt, X.data_ptr(), ldx, Wp.data.data_ptr(), w_scale.data_ptr(),
                                  0 if bias is None else bias.data_ptr(), T, d_in, d_out, dt, out.data_ptr(), ldy, z,
                                  ldz, ws.data_ptr(), nbytes, st), "fp_scaled_linear")
    return out


# ------------------------------------------------------------------- norms --
def _rows_like(t, dtype, shape, name: str) -> int:
    """_matrix of a given type and shape, at once where its rows are as they mostly are."""
    if t.dtype is dtype and t.shape == shape:
        ld, one = t.stride()
        if one == 1 and ld >= shape[1]:
            return ld
    return _matrix(t, dtype, shape[0], shape[1], name)


def _norm_args(X, weight, name: str):
    """Rows' shape, type, the library's name for it, leading dimension, the weights' type and address."""
    shape, dtype = X.shape, X.dtype
    if len(shape) != 2:
        raise ValueError("%s: shape %s, expected two dimensions" % (name, tuple(shape)))
    dt = _float_dt(dtype, name)
    ld = _rows_like(X, dtype, shape, name)
    if weight is None:
        return shape, dtype, dt, ld, dt, 0
    wt = weight.dtype
    if wt is not dtype and wt is not torch.float32:
        raise ValueError("weight: %s, expected %s or float32" % (wt, dtype))
    _vector(weight, wt, shape[1:], "weight")
    return shape, dtype, dt, ld, _FLOATS[wt], weight.data_ptr()


def _stream_rows(X, shape, dtype, residual, residual_out):
    """The residual's address and leading dimension, and where the sum goes (made if None and there is a residual)."""
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out: no residual to add")
        return 0, shape[1], None, 0, shape[1]
    ldr = _rows_like(residual, dtype, shape, "residual")
    if residual_out is None:
        residual_out = torch.empty(shape, dtype=dtype, device=X.device)
    ldh = _rows_like(residual_out, dtype, shape, "residual_out")
    return residual.data_ptr(), ldr, residual_out, residual_out.data_ptr(), ldh


def rms_norm(X, weight, eps: float = 1e-5, residual=None, residual_out=None, out=None):
    """Y = h / sqrt(mean(h^2) + eps) * weight for the rows h of X [T, d] (float32, float16 or bfloat16), in X's type; weight
    [d] in X's type or float32 (None: ones). With a ``residual`` h = X + residual, and (Y, H) is returned, H being the sum
    in X's type (``residual_out``, which may be the residual itself or X, but not ``out``); the norm is of the sum before
    that rounding. Sums in fp32. The gradient is rms_norm_backward; no graph is recorded, and tensors that require a gradient are refused
    unless under torch.no_grad."""
    _no_graph("rms_norm_backward", X, weight, residual)
    shape, dtype, dt, ldx, w_dt, w = _norm_args(X, weight, "X")
    T, d = shape
    r, ldr, H, h, ldh = _stream_rows(X, shape, dtype, residual, residual_out)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=X.device)
    ldy = _rows_like(out, dtype, shape, "out")
    st = _here(X, weight, residual, H, out)
    _check(lib().fp_rms_norm(dt, X.data_ptr(), ldx, r, ldr, w_dt, w, eps, T, d, h, ldh, out.data_ptr(), ldy, 0, d, 0, st),
           "fp_rms_norm")
    return out if H is None else (out, H)


def rms_norm_quantize(X, weight, eps: float = 1e-5, residual=None, residual_out=None, out=None, scale=None, Y=None):
    """(Xq, scale), with a ``residual`` (Xq, scale, H): quantize_rows of rms_norm's fp32 rows, for scaled_matmul or
    moe_layer. ``Y`` (X's type) also receives the rows themselves, which a router reads. The int8 rows have no gradient."""
    _no_graph("rms_norm_backward", X, weight, residual)
    shape, dtype, dt, ldx, w_dt, w = _norm_args(X, weight, "X")
    T, d = shape
    r, ldr, H, h, ldh = _stream_rows(X, shape, dtype, residual, residual_out)
    if out is None:
        out = torch.empty((T, (d + 15) // 16 * 16), dtype=torch.int8, device=X.device)
        if d % 16:
            out = out[:, :d]
    ldq = _rows_like(out, torch.int8, shape, "out")
    if scale is None:
        scale = torch.empty(T, dtype=torch.float32, device=X.device)
    else:
        _vector(scale, torch.float32, shape[:1], "scale")
    y, ldy = (0, d) if Y is None else (Y.data_ptr(), _rows_like(Y, dtype, shape, "Y"))
    st = _here(X, weight, residual, H, out, scale, Y)
    _check(lib().fp_rms_norm(dt, X.data_ptr(), ldx, r, ldr, w_dt, w, eps, T, d, h, ldh, y, ldy, out.data_ptr(), ldq,
                             scale.data_ptr(), st), "fp_rms_norm")
    return (out, scale) if H is None else (out, scale, H)


def rms_norm_backward(dY, H, weight, eps: float = 1e-5, dH=None, out=None, dw=None):
    """(dX, dw), the gradients of rms_norm at H [T, d] (its X, or the sum it returned, as that was rounded) from dY: dX [T, d]
    in H's type, of X and of the residual alike, with ``dH``, the gradient of H's other uses, added; dw float32 [d] (None
    without weights). d is at most 16384."""
    shape, dtype, dt, ldh, w_dt, w = _norm_args(H, weight, "H")
    T, d = shape
    lddy = _rows_like(dY, dtype, shape, "dY")
    lddh = d if dH is None else _rows_like(dH, dtype, shape, "dH")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=H.device)
    lddx = _rows_like(out, dtype, shape, "out")
    if weight is None:
        if dw is not None:
            raise ValueError("dw: there are no weights")
    elif dw is None:
        dw = torch.empty(d, dtype=torch.float32, device=H.device)
    else:
        _vector(dw, torch.float32, (d,), "dw")
    st = _here(dY, H, weight, dH, out, dw)
    nbytes = 0 if dw is None else lib().fp_rms_norm_backward_workspace(T, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=H.device)
    _check(lib().fp_rms_norm_backward(dt, dY.data_ptr(), lddy, H.data_ptr(), ldh, w_dt, w, eps,
                                      0 if dH is None else dH.data_ptr(), lddh, T, d, out.data_ptr(), lddx,
                                      0 if dw is None else dw.data_ptr(), ws.data_ptr(), nbytes, st), "fp_rms_norm_backward")
    return out, dw


class PackedExperts:
    """The packed weights of G experts of one shape (pack_experts): ``weights`` holds each one's PackedWeights."""

    def __init__(self, weights):
        weights = list(weights)
        if not weights:
            raise ValueError("no experts")
        if any((w.d_out, w.d_in) != (weights[0].d_out, weights[0].d_in) for w in weights):
            raise ValueError("experts of different shapes")
        self.weights, self.d_out, self.d_in = weights, weights[0].d_out, weights[0].d_in
        self.device = weights[0].data.device
        if any(w.data.device != self.device for w in weights):
            raise ValueError("experts on different devices")
        self.ptrs = (ctypes.c_void_p * len(weights))(*[w.data.data_ptr() for w in weights])
        # (first expert, how many, their addresses in ptrs): a launch takes MAX_GROUPS
        counts = [(g, min(MAX_GROUPS, len(weights) - g)) for g in range(0, len(weights), MAX_GROUPS)]
        self.parts = [(g, n, (ctypes.c_void_p * n).from_buffer(self.ptrs, g * ctypes.sizeof(ctypes.c_void_p))) for g, n in counts]
        self._table = self._sent = None
        if not self._capturing():
            self._send()  # now, so that a call may be captured

    def __len__(self):
        return len(self.weights)

    def _capturing(self) -> bool:
        return self.device.type == "cuda" and torch.cuda.is_current_stream_capturing()

    def _send(self):
        """The addresses on their way to the device, behind what the current stream has; the host does not wait."""
        on_gpu = self.device.type == "cuda"
        host = torch.empty(len(self.weights), dtype=torch.int64, pin_memory=on_gpu)
        ctypes.memmove(host.data_ptr(), self.ptrs, ctypes.sizeof(self.ptrs))
        self._table = host.to(self.device, non_blocking=True)
        if on_gpu:
            self._sent = torch.cuda.Event()
            self._sent.record(torch.cuda.current_stream(self.device))

    @property
    def table(self):
        """The weights' addresses on the device (int64 [G]), for calls whose experts only the device knows. The current
        stream waits for them where they are still on their way."""
        if self._table is None:
            if self._capturing():
                raise ValueError("experts packed inside a capture: their addresses reach the device only outside of one")
            self._send()
        if self._sent is not None and not self._capturing():  # (torch.cuda.graph has waited for the device)
            if self._sent.query():
                self._sent = None
            else:
                self._sent.wait(torch.cuda.current_stream(self.device))
        return self._table


def pack_experts(W) -> PackedExperts:
    """The weights of every expert packed once: W int8 [G, d_out, d_in], or a list of int8 [d_out, d_in]."""
    return PackedExperts([pack_weights(w) for w in W])


def scaled_matmul_grouped(X, x_scale, We: PackedExperts, w_scale, offsets, rows=None, bias=None, out=None,
                          dtype=torch.bfloat16, Z=None):
    """scaled_matmul of each expert with its own rows: output rows [offsets[g], offsets[g + 1]) (int32 [G + 1] on the
    device, as moe_sort writes them) by expert g with w_scale[g] (float32 [G, d_out]; bias likewise). Output row i is
    made from X's row rows[i] (int32 on the device, e.g. moe_sort's tokens; None: row i). Rows of no expert are left as
    they were in ``out`` and Z (a new ``out`` holds whatever its memory held there). More than 256 experts take a launch
    for every 256."""
    G, d_in, d_out = len(We.weights), We.d_in, We.d_out
    ldx = _matrix(X, torch.int8, None, d_in, "X")
    n = x_rows = X.shape[0]
    _vector(x_scale, torch.float32, (x_rows,), "x_scale")
    ldw = _matrix(w_scale, torch.float32, G, d_out, "w_scale")
    if bias is not None and _matrix(bias, torch.float32, G, d_out, "bias") != ldw and G > 1:
        raise ValueError("bias: its rows are not as far apart as w_scale's")
    _vector(offsets, torch.int32, (G + 1,), "offsets")
    if rows is not None:
        n = rows.numel()
        _vector(rows, torch.int32, (n,), "rows")
    out, dt, ldy, z, ldz = _product_out(n, d_out, out, dtype, Z, X.device)
    X, ldx = _readable(X, ldx)
    st = _here(X, x_scale, We.weights[0].data, w_scale, offsets, rows, bias, out, Z)
    for g, count, ptrs in We.parts:
        _check(lib().fp_scaled_matmul_grouped(X.data_ptr(), ldx, x_scale.data_ptr(), x_rows,
                                              0 if rows is None else rows.data_ptr(), n, ptrs,
                                              w_scale.data_ptr() + 4 * g * ldw,
                                              0 if bias is None else bias.data_ptr() + 4 * g * ldw, ldw,
                                              offsets.data_ptr() + 4 * g, count, d_in, d_out, dt, out.data_ptr(), ldy, z,
                                              ldz, st), "fp_scaled_matmul_grouped")
    return out


# ------------------------------------------------------- tokens by expert --
def _no_graph(name: str, *tensors):
    """No call here records a graph for autograd: one whose gradient is a call of its own refuses a tensor that asks for
    a gradient, which would be lost. (Inside a torch.autograd.Function, and under torch.no_grad, nothing asks.)"""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("a tensor requires a gradient, which this call does not record: wrap it and %s in a "
                             "torch.autograd.Function, or detach the tensor" % name)


class MoePlan:
    """The device sort of T tokens with K experts each out of E: offsets int32 [E + 1], slots and tokens int32 [T K]
    (sorted row -> slot t K + k, and -> t; -1 past the last row with an expert) and rows int32 [T, K] (slot -> sorted
    row; -1: no expert). Filled by moe_sort or moe_dispatch, on the stream of that call; a program that sorts at every
    step may keep one."""

    def __init__(self, T: int, K: int, E: int, device=None):
        if T < 0 or K < 1 or E < 1:
            raise ValueError("MoePlan: T=%d K=%d E=%d" % (T, K, E))
        self.T, self.K, self.E = T, K, E
        n = T * K
        self.nbytes = lib().fp_moe_sort_workspace(T, K, E)
        buf = torch.empty(E + 1 + 3 * n + self.nbytes // 4, dtype=torch.int32, device=device or _dev())
        self.offsets = buf[:E + 1]
        self.slots, self.tokens = buf[E + 1:E + 1 + n], buf[E + 1 + n:E + 1 + 2 * n]
        self.rows = buf[E + 1 + 2 * n:E + 1 + 3 * n].view(T, K)
        self.ws = buf[E + 1 + 3 * n:]
        self.buf = buf
        # offsets, slots, tokens, rows: where the calls write them
        self.ptrs = tuple(t.data_ptr() for t in (self.offsets, self.slots, self.tokens, self.rows))


def _sort_args(ids, n_experts: int, plan):
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids: %s %s, expected int32 or int64 (T, K)" % (ids.dtype, tuple(ids.shape)))
    if not ids.is_contiguous():
        raise ValueError("ids: must be contiguous")
    T, K = ids.shape
    if plan is None:
        plan = MoePlan(T, K, n_experts, ids.device)
    elif (plan.T, plan.K, plan.E) != (T, K, n_experts):
        raise ValueError("plan: for T=%d K=%d E=%d, the call has T=%d K=%d E=%d" % (plan.T, plan.K, plan.E, T, K, n_experts))
    return plan


def moe_sort(ids, n_experts: int, plan: MoePlan | None = None) -> MoePlan:
    """The slots of ids [T, K] (each token's experts, int32 or int64 on the device) sorted by expert, stably; an id
    outside [0, n_experts) is a slot without an expert. Nothing is read back by the host (compare moe_plan)."""
    plan = _sort_args(ids, n_experts, plan)
    st = _here(ids, plan.buf)
    _check(lib().fp_moe_sort(ids.data_ptr(), ids.element_size(), plan.T, plan.K, plan.E, *plan.ptrs,
                             plan.ws.data_ptr(), plan.nbytes, st), "fp_moe_sort")
    return plan


def _permute_out(X, plan, out):
    """X's element size and leading dimension, out (made if None) and its leading dimension."""
    eb = X.element_size()
    if eb not in (1, 2, 4):
        raise ValueError("X: elements of %d bytes, expected 1, 2 or 4" % eb)
    if X.dim() != 2:
        raise ValueError("X: shape %s, expected two dimensions" % (tuple(X.shape),))
    d, n = X.shape[1], plan.T * plan.K
    ldx = _matrix(X, None, plan.T, d, "X")
    if out is None:
        out = torch.empty((n, d), dtype=X.dtype, device=X.device)
    return eb, ldx, out, _matrix(out, X.dtype, n, d, "out")


def moe_permute(X, plan: MoePlan, out=None):
    """Xs [T K, d]: the tokens' rows X [T, d] in the plan's order. Rows past the last one with an expert are left as
    they were in ``out`` (a new one holds whatever its memory held there). Its gradient is moe_dispatch_backward; no graph
    is recorded, and an X that requires a gradient is refused unless under torch.no_grad."""
    _no_graph("moe_dispatch_backward", X)
    eb, ldx, out, ldo = _permute_out(X, plan, out)
    st = _here(X, plan.buf, out)
    _check(lib().fp_moe_permute(eb, X.data_ptr(), ldx, plan.T, plan.K, X.shape[1], plan.ptrs[3], out.data_ptr(), ldo,
                                st), "fp_moe_permute")
    return out


def moe_dispatch(X, ids, n_experts: int, plan: MoePlan | None = None, out=None):
    """(Xs, plan): moe_sort of ids and moe_permute of X in one call (its gradient: moe_dispatch_backward, as there)."""
    _no_graph("moe_dispatch_backward", X)
    plan = _sort_args(ids, n_experts, plan)
    eb, ldx, out, ldo = _permute_out(X, plan, out)
    st = _here(X, ids, plan.buf, out)
    _check(lib().fp_moe_dispatch(eb, X.data_ptr(), ldx, X.shape[1], ids.data_ptr(), ids.element_size(), plan.T, plan.K,
                                 plan.E, *plan.ptrs, out.data_ptr(), ldo, plan.ws.data_ptr(), plan.nbytes, st),
           "fp_moe_dispatch")
    return out, plan


def _combine(O, plan, weights, out, name):
    if O.dim() != 2:
        raise ValueError("%s: shape %s, expected two dimensions" % (name, tuple(O.shape)))
    T, K, d = plan.T, plan.K, O.shape[1]
    dt = _float_dt(O.dtype, name)
    ldi = _matrix(O, None, T * K, d, name)
    if weights is not None:
        _vector(weights, torch.float32, (T, K), "weights")
    if out is None:
        out = torch.empty((T, d), dtype=O.dtype, device=O.device)
    ldo = _matrix(out, O.dtype, T, d, "out")
    st = _here(O, plan.buf, weights, out)
    _check(lib().fp_moe_combine(dt, O.data_ptr(), ldi, T * K, plan.ptrs[3],
                                0 if weights is None else weights.data_ptr(), T, K, d, out.data_ptr(), ldo, st),
           "fp_moe_combine")
    return out


def moe_combine(O, plan: MoePlan, weights=None, out=None):
    """Y [T, d]: each token's rows of O [T K, d] (the experts' outputs in the plan's order) added with its weights
    (float32 [T, K]; None: all one), in fp32, k ascending. Its gradients are moe_combine_backward (without weights:
    moe_permute); no graph is recorded, and tensors that require a gradient are refused unless under torch.no_grad."""
    _no_graph("moe_combine_backward", O, weights)
    return _combine(O, plan, weights, out, "O")


def moe_dispatch_backward(dXs, plan: MoePlan, out=None):
    """dX [T, d], the gradient of moe_permute and moe_dispatch: each token's rows of dXs [T K, d] added."""
    return _combine(dXs, plan, None, out, "dXs")


def moe_combine_backward(dY, O, plan: MoePlan, weights, dO=None, dw=None):
    """(dO [T K, d], dw [T, K]), the gradients of moe_combine. Rows of dO past the last one with an expert are left as
    they were (a new one holds whatever its memory held there); dw is zero for a slot without an expert."""
    if O.dim() != 2:
        raise ValueError("O: shape %s, expected two dimensions" % (tuple(O.shape),))
    T, K, d = plan.T, plan.K, O.shape[1]
    dt = _float_dt(O.dtype, "O")
    ldi, ldy = _matrix(O, None, T * K, d, "O"), _matrix(dY, O.dtype, T, d, "dY")
    _vector(weights, torch.float32, (T, K), "weights")
    if dO is None:
        dO = torch.empty((T * K, d), dtype=O.dtype, device=O.device)
    ldo = _matrix(dO, O.dtype, T * K, d, "dO")
    if dw is None:
        dw = torch.empty((T, K), dtype=torch.float32, device=O.device)
    else:
        _vector(dw, torch.float32, (T, K), "dw")
    st = _here(dY, O, plan.buf, weights, dO, dw)
    _check(lib().fp_moe_combine_backward(dt, dY.data_ptr(), ldy, O.data_ptr(), ldi, T * K, plan.ptrs[3],
                                         weights.data_ptr(), T, K, d, dO.data_ptr(), ldo, dw.data_ptr(), st),
           "fp_moe_combine_backward")
    return dO, dw


def _expert_scales(We, scale, shape, name: str):
    """Check an expert map and its scales; their addresses and the scales' leading dimension."""
    if (We.d_out, We.d_in) != shape:
        raise ValueError("%s: experts of %d -> %d, expected %d -> %d" % (name, We.d_in, We.d_out, shape[1], shape[0]))
    return We.table.data_ptr(), scale.data_ptr(), _matrix(scale, torch.float32, len(We.weights), shape[0], name + "_scale")


def moe_layer(X, ids, weights, up: PackedExperts, up_scale, down: PackedExperts, down_scale, gate: PackedExperts | None = None,
              gate_scale=None, x_scale=None, out=None, dtype=None):
    """Y [T, d] = sum_k weights[t, k] Down(silu(Gate x_t) * Up x_t) by the experts ids[t, k] (without a gate: silu(Up x_t)),
    for a few tokens (T K at most 1024), in two launches (up to four where an expert has many): the answer of the same layer
    strung together from scaled_linear's products by expert and moe_combine. X [T, d]: float32, float16 or bfloat16, or int8
    with ``x_scale`` (rms_norm_quantize's rows). ids [T, K] (int32 or int64 on the device): an id outside [0, experts) is a
    slot without an expert; weights float32 [T, K]. up, gate: pack_experts of [E, ff, d], down: of [E, d, ff], each with
    float32 scales [E, outputs]. With many small experts the calls for many tokens are faster from about 64 tokens on. Y is in
    ``out``'s type, ``dtype``, X's, or bfloat16 for int8 X. It has no gradient: tensors that require one are refused unless
    under torch.no_grad."""
    for t in (X, weights, x_scale, up_scale, down_scale, gate_scale):
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("a tensor requires a gradient, which this layer does not have: train through moe_dispatch and "
                             "moe_combine, or detach the tensor")
    if X.dim() != 2:
        raise ValueError("X: shape %s, expected two dimensions" % (tuple(X.shape),))
    T, d = X.shape
    if X.dtype is torch.int8:
        if x_scale is None:
            raise ValueError("x_scale: int8 rows have scales")
        _vector(x_scale, torch.float32, (T,), "x_scale")
        x_dt = FP_I8
    else:
        if x_scale is not None:
            raise ValueError("x_scale: %s rows have none" % X.dtype)
        x_dt = _float_dt(X.dtype, "X")
    ldx = _matrix(X, None, T, d, "X")
    if ids.dim() != 2 or ids.shape[0] != T or ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError("ids: %s %s, expected contiguous int32 or int64 (%d, K)" % (ids.dtype, tuple(ids.shape), T))
    K, E, ff = ids.shape[1], len(up.weights), up.d_out
    _vector(weights, torch.float32, (T, K), "weights")
    if (gate is None) != (gate_scale is None):
        raise ValueError("gate and gate_scale come together")
    if len(down.weights) != E or (gate is not None and len(gate.weights) != E):
        raise ValueError("maps of different numbers of experts")
    u, us, ldu = _expert_scales(up, up_scale, (ff, d), "up")
    dn, ds, ldd = _expert_scales(down, down_scale, (d, ff), "down")
    g, gs, ldg = (0, 0, ff) if gate is None else _expert_scales(gate, gate_scale, (ff, d), "gate")
    if out is None:
        dtype = dtype or (torch.bfloat16 if x_dt == FP_I8 else X.dtype)
        _float_dt(dtype, "out")
        out = torch.empty((T, d), dtype=dtype, device=X.device)
    ldy = _matrix(out, None, T, d, "out")
    y_dt = _float_dt(out.dtype, "out")
    st = _here(X, x_scale, ids, weights, up.table, up_scale, down.table, down_scale, gate and gate.table, gate_scale, out)
    nbytes = lib().fp_moe_layer_workspace(T, K, d, ff)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    _check(lib().fp_moe_layer(x_dt, X.data_ptr(), ldx, 0 if x_scale is None else x_scale.data_ptr(), ids.data_ptr(),
                              ids.element_size(), weights.data_ptr(), T, K, E, g, gs, ldg, u, us, ldu, dn, ds, ldd, d, ff,
                              y_dt, out.data_ptr(), ldy, ws.data_ptr(), nbytes, st), "fp_moe_layer")
    return out


# ------------------------------------------------------- log probabilities --
class TokenLogprobs:
    """What token_logprobs says of T rows of logits: ``logprob`` and ``entropy`` float32 [T], ``top_logprobs`` float32 and
    ``top_ids`` int32 [T, top], and ``max`` and ``logsum`` float32 [T], which the gradient reads. A program that asks at every
    step may keep one."""

    def __init__(self, T: int, top: int = 0, device=None):
        if T < 0 or top < 0:
            raise ValueError("TokenLogprobs: T=%d top=%d" % (T, top))
        self.T, self.top = T, top
        buf = torch.empty(T * (4 + 2 * top), dtype=torch.float32, device=device or _dev())
        self.logprob, self.entropy, self.max, self.logsum = (buf[i * T:(i + 1) * T] for i in range(4))
        self.top_logprobs = buf[4 * T:(4 + top) * T].view(T, top)
        self.top_ids = buf[(4 + top) * T:].view(torch.int32).view(T, top)
        self.buf = buf
        self.ptrs = tuple(t.data_ptr() for t in (self.logprob, self.entropy, self.max, self.logsum)) + (
            (self.top_logprobs.data_ptr(), self.top_ids.data_ptr()) if top else (0, 0))


def _logit_args(logits, tokens):
    if logits.dim() != 2:
        raise ValueError("logits: shape %s, expected two dimensions" % (tuple(logits.shape),))
    T, V = logits.shape
    dt = _float_dt(logits.dtype, "logits")
    if tokens.dtype not in (torch.int32, torch.int64):
        raise ValueError("tokens: %s, expected int32 or int64" % tokens.dtype)
    _vector(tokens, tokens.dtype, (T,), "tokens")
    return T, V, dt, _matrix(logits, None, T, V, "logits")


def token_logprobs(logits, tokens, temperature: float = 1.0, top: int = 0, out: TokenLogprobs | None = None) -> TokenLogprobs:
    """Of every row of logits [T, V] (float32, float16 or bfloat16), divided by the temperature: the log probability of
    tokens[t] (int32 or int64 on the device; one outside [0, V) is padding and gets 0), the entropy, and the ``top`` most
    probable tokens (at most 32; equal logits by their index). Logits of -infinity are tokens that cannot come; a row of
    these alone has log probability -infinity and entropy 0, one with a NaN or +infinity NaN and top ids -1. The gradient
    is token_logprobs_backward; no graph is recorded, and logits that require a gradient are refused unless under
    torch.no_grad."""
    _no_graph("token_logprobs_backward", logits)
    T, V, dt, ldx = _logit_args(logits, tokens)
    if out is None:
        out = TokenLogprobs(T, top, logits.device)
    elif (out.T, out.top) != (T, top):
        raise ValueError("out: for T=%d top=%d, the call has T=%d top=%d" % (out.T, out.top, T, top))
    st = _here(logits, tokens, out.buf)
    nbytes = lib().fp_token_logprobs_workspace(dt, T, V, top)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=logits.device) if nbytes else None
    _check(lib().fp_token_logprobs(dt, logits.data_ptr(), ldx, T, V, tokens.data_ptr(), tokens.element_size(), temperature,
                                   top, *out.ptrs, ws.data_ptr() if nbytes else 0, nbytes, st), "fp_token_logprobs")
    return out


def token_logprobs_backward(dlogprob, dentropy, logits, tokens, lp: TokenLogprobs, temperature: float = 1.0, out=None):
    """dlogits [T, V] in the logits' type, from the gradients of lp.logprob and lp.entropy (float32 [T]; None: zero), lp
    being what token_logprobs said of the same logits, tokens and temperature. ``out`` may be the logits themselves.
    A row with a NaN or +infinity has a gradient of NaN throughout."""
    T, V, dt, ldx = _logit_args(logits, tokens)
    for g, name in ((dlogprob, "dlogprob"), (dentropy, "dentropy")):
        if g is not None:
            _vector(g, torch.float32, (T,), name)
    if lp.T != T:
        raise ValueError("lp: for T=%d, the call has T=%d" % (lp.T, T))
    if out is None:
        out = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
    lddx = _matrix(out, logits.dtype, T, V, "out")
    st = _here(dlogprob, dentropy, logits, tokens, lp.buf, out)
    _check(lib().fp_token_logprobs_backward(dt, logits.data_ptr(), ldx, T, V, tokens.data_ptr(), tokens.element_size(),
                                            temperature, 0 if dlogprob is None else dlogprob.data_ptr(),
                                            0 if dentropy is None else dentropy.data_ptr(), lp.ptrs[2], lp.ptrs[3],
                                            lp.ptrs[1], out.data_ptr(), lddx, st), "fp_token_logprobs_backward")
    return out


# ----------------------------------------------------------------------- eq --
def eq_table(r, E=None):
    n = r.numel()
    E = torch.empty(1 << n, dtype=torch.int64, device=_dev()) if E is None else E
    _check(lib().fp_eq_table(_ptr(r) if n else None, n, _ptr(E), _stream()), "fp_eq_table")
    return E


def eq_table_batched(rs, Es=None):
    k = len(rs)
    if Es is None:
        Es = [torch.empty(1 << r.numel(), dtype=torch.int64, device=_dev()) for r in rs]
    descs = (_EqDesc * k)(*[_EqDesc(r.data_ptr() if r.numel() else None, r.numel(), E.data_ptr())
                            for r, E in zip(rs, Es)])
    _check(lib().fp_eq_table_batched(k, descs, None, 0, _stream()), "fp_eq_table_batched")
    return Es


# -------------------------------------------------------------------- folds --
def _dt(M):
    if M.dtype == torch.int8:
        return FP_I8
    if M.dtype == torch.int32:
        return FP_I32
    raise TypeError(M.dtype)


def fold_matrix(M, E, cols_pad: int | None = None, rows: int | None = None, out=None):
    rows = M.shape[0] if rows is None else rows
    cols = M.shape[1]
    cols_pad = cols if cols_pad is None else cols_pad
    out = torch.empty(cols_pad, dtype=torch.int64, device=M.device) if out is None else out
    need = lib().fp_fold_matrix_workspace(_dt(M), rows, cols)
    p, nb = _ws_fold.get(need)
    _check(lib().fp_fold_matrix(_dt(M), _ptr(M), _ld(M), rows, cols, _ptr(E), _ptr(out), cols_pad, p, nb,
                                _stream()), "fp_fold_matrix")
    return out


def fold_matrix_batched(jobs):
    """jobs: list of (M, E, cols_pad, out); all M of one dtype."""
    k = len(jobs)
    dt = _dt(jobs[0][0])
    descs = (_FoldDesc * k)(*[_fold_desc(f) for f in jobs])
    need = lib().fp_fold_matrix_batched_workspace(dt, k, descs)
    p, nb = _ws_fold.get(need)
    _check(lib().fp_fold_matrix_batched(dt, k, descs, p, nb, _stream()), "fp_fold_matrix_batched")
    return [j[3] for j in jobs]


def fold_weights_prepare(M, Mt=None, colsum=None):
    """Transposed copy Mt [cols, ldt] (ldt = rows rounded up to 16) and column
    sums [cols] int32 of an int8 matrix M [rows, cols], for fold_matrix_multi."""
    rows, cols = M.shape
    ldt = max(16, (rows + 15) // 16 * 16)
    Mt = torch.empty((cols, ldt), dtype=torch.int8, device=M.device) if Mt is None else Mt
    colsum = torch.empty(cols, dtype=torch.int32, device=M.device) if colsum is None else colsum
    assert Mt.dtype == torch.int8 and Mt.shape[0] == cols and Mt.stride(1) == 1
    _check(lib().fp_fold_weights_prepare(_ptr(M) if M.numel() else None, _ld(M), rows, cols,
                                         _ptr(Mt) if Mt.numel() else None, Mt.stride(0), _ptr(colsum), _stream()),
           "fp_fold_weights_prepare")
    return Mt, colsum


def fold_matrix_multi(Mt, colsum, rows: int, E, cols_pad: int | None = None, out=None):
    """out[j, k] = sum_t E[j, t] M[t, k] for every row j of E [R, >= rows]
    (int64 field tensor), from fold_weights_prepare's Mt and colsum."""
    cols = Mt.shape[0]
    R = E.shape[0]
    cols_pad = cols if cols_pad is None else cols_pad
    out = torch.empty((R, cols_pad), dtype=torch.int64, device=Mt.device) if out is None else out
    assert E.dtype == torch.int64 and E.stride(1) == 1 and out.stride(1) == 1
    lde = E.stride(0) if R > 1 else max(E.stride(0), rows)
    ldo = out.stride(0) if R > 1 else max(out.stride(0), cols_pad)
    need = lib().fp_fold_matrix_multi_workspace(rows, cols, R)
    p, nb = _ws_multi.get(need)
    _check(lib().fp_fold_matrix_multi(_ptr(Mt) if Mt.numel() else None, Mt.stride(0), _ptr(colsum), rows, cols, R,
                                      _ptr(E) if E.numel() else None, lde, _ptr(out) if out.numel() else None, ldo,
                                      cols_pad, p, nb, _stream()), "fp_fold_matrix_multi")
    return out


# --------------------------------------------------------------- commitment --
SALT_BYTES, DIGEST_BYTES = 16, 32


def commit_rows(na: int, nb: int, logn: int) -> int:
    """Rows of 2^logn elements that hold na + nb limbs, three per element."""
    elems = (na + nb + 2) // 3
    return max(1, (elems + (1 << logn) - 1) >> logn)


def commit_pack(A, B, logn: int, rows: int | None = None, out=None):
    """Limbs of the int8 tensors A then B, three per field element in 20-bit
    slots, as [rows, 2^logn] (zero past the limbs)."""
    na, nb = A.numel(), B.numel()
    rows = commit_rows(na, nb, logn) if rows is None else rows
    dev = A.device if na else B.device
    out = torch.empty((rows, 1 << logn), dtype=torch.int64, device=dev) if out is None else out
    assert out.is_contiguous() and A.is_contiguous() and B.is_contiguous()
    _check(lib().fp_commit_pack(_ptr(A) if na else None, na, _ptr(B) if nb else None, nb, logn, rows, _ptr(out),
                                _stream()), "fp_commit_pack")
    return out


def rs_encode(msg, code=None):
    """Rate-1/2 Reed-Solomon codewords [rows, 2n] of the rows of msg [rows, n]."""
    rows, n = msg.shape
    logn = n.bit_length() - 1
    assert 1 << logn == n and msg.stride(1) == 1
    code = torch.empty((rows, 2 * n), dtype=torch.int64, device=msg.device) if code is None else code
    need = lib().fp_rs_encode_workspace(rows, logn)
    p, nbytes = _ws_rs.get(need)
    _check(lib().fp_rs_encode(_ptr(msg), msg.stride(0) if rows > 1 else n, rows, logn, _ptr(code),
                              code.stride(0) if rows > 1 else 2 * n, p, nbytes, _stream()), "fp_rs_encode")
    return code


def merkle_commit(code, salts, tree=None):
    """Salted BLAKE2b-256 Merkle tree over the columns of code [rows, W]
    (W a power of 2); salts: uint8 [W, 16]. Returns the tree as uint8
    [2W - 1, 32]: the W leaves, then each level up, the root last."""
    rows, W = code.shape
    logw = W.bit_length() - 1
    assert 1 << logw == W and salts.shape == (W, SALT_BYTES) and salts.is_contiguous()
    tree = torch.empty((2 * W - 1, DIGEST_BYTES), dtype=torch.uint8, device=code.device) if tree is None else tree
    _check(lib().fp_merkle_commit(_ptr(code), code.stride(0) if rows > 1 else W, rows, logw, _ptr(salts),
                                  _ptr(tree), _stream()), "fp_merkle_commit")
    return tree


# ------------------------------------------------------------------- lookup --
def lookup_tree(keys, L: int, gamma, tree=None):
    """Product tree [2^(L+1) - 1] of the leaves gamma - key (int8 keys, padded
    with 0 to 2^L), levels from the leaves up; gamma: device int64 [1]."""
    n = keys.numel()
    _need(keys, torch.int8, n, "keys")
    assert 0 <= L <= 30 and n <= (1 << L), "keys must fit the 2^L leaves"
    _need(gamma, torch.int64, 1, "gamma")
    tree = torch.empty((2 << L) - 1, dtype=torch.int64, device=gamma.device) if tree is None else tree
    _need(tree, torch.int64, (2 << L) - 1, "tree")
    _check(lib().fp_lookup_tree(_ptr(keys) if n else None, n, L, _ptr(gamma), _ptr(tree), _stream()),
           "fp_lookup_tree")
    return tree


CLAMP_SCALE, CLAMP_OFFSET, CLAMP_BITS = 1 << 16, (1 << 15) + (128 << 16), 16


def lookup_tree_pairs(A, B, L: int, gamma, scale: int = CLAMP_SCALE, offset: int = CLAMP_OFFSET, tree=None):
    """Product tree [2^(L+1) - 1] of the leaves gamma - (A + scale B + offset) of two field tables of 2^L
    entries (by default the clamp's keys of Q = A and Y = B)."""
    n = A.numel()
    _need(A, torch.int64, n, "A")
    _need(B, torch.int64, n, "B")
    assert n <= (1 << L) and B.numel() == n
    _need(gamma, torch.int64, 1, "gamma")
    tree = torch.empty((2 << L) - 1, dtype=torch.int64, device=A.device) if tree is None else tree
    _need(tree, torch.int64, (2 << L) - 1, "tree")
    _check(lib().fp_lookup_tree_pairs(_ptr(A), _ptr(B), n, scale % P, offset % P, L, _ptr(gamma), _ptr(tree),
                                      _stream()), "fp_lookup_tree_pairs")
    return tree


def lookup_counts_field(A, lo: int = -(1 << 15), bits: int = CLAMP_BITS, counts=None):
    """Multiplicities [2^bits + 1] of the field values A read as signed integers over [lo, lo + 2^bits) (the
    last entry: values outside)."""
    n = A.numel()
    _need(A, torch.int64, n, "A")
    counts = torch.empty((1 << bits) + 1, dtype=torch.int32, device=A.device) if counts is None else counts
    _need(counts, torch.int32, (1 << bits) + 1, "counts")
    _check(lib().fp_lookup_counts_field(_ptr(A), n, lo, bits, _ptr(counts), _stream()), "fp_lookup_counts_field")
    return counts


def lookup_counts(keys, L: int, s: int, counts=None):
    """Multiplicities [2^s + 1] (int32 holding uint32) of the table values
    -2^(s-1) + i among the padded keys; the last entry counts keys outside."""
    n = keys.numel()
    dev = keys.device if n else _dev()
    _need(keys, torch.int8, n, "keys")
    assert 1 <= s <= 8, "s outside [1, 8]"
    counts = torch.empty((1 << s) + 1, dtype=torch.int32, device=dev) if counts is None else counts
    _need(counts, torch.int32, (1 << s) + 1, "counts")
    _check(lib().fp_lookup_counts(_ptr(keys) if n else None, n, L, s, _ptr(counts), _stream()), "fp_lookup_counts")
    return counts


def sumcheck3_prove(E, V, r, rounds=None, finals=None):
    """Degree-3 sum-check of sum_x E[x] V[2x] V[2x+1]: rounds [m, 4], finals [3]."""
    m = r.numel()
    dev = E.device
    rounds = torch.empty((max(m, 1), 4), dtype=torch.int64, device=dev) if rounds is None else rounds
    finals = torch.empty(3, dtype=torch.int64, device=dev) if finals is None else finals
    _need(E, torch.int64, 1 << m, "E")
    _need(V, torch.int64, 2 << m, "V")
    _need(r, torch.int64, m, "r")
    _need(rounds, torch.int64, 4 * m, "rounds")
    _need(finals, torch.int64, 3, "finals")
    need = lib().fp_sumcheck3_workspace(m)
    p, nbytes = _ws_lookup.get(need)
    _check(lib().fp_sumcheck3_prove(_ptr(E), _ptr(V), m, _ptr(r) if m else None, _ptr(rounds), _ptr(finals), p,
                                    nbytes, _stream()), "fp_sumcheck3_prove")
    return rounds[:m], finals


def lookup_prove(tree, L: int, chal, rounds=None, finals=None):
    """The product tree's proof: rounds [L(L-1)/2, 4] and finals [L, 3], levels
    from the root down; chal: device int64 [L(L+1)/2]."""
    dev = tree.device
    nr = L * (L - 1) // 2
    rounds = torch.empty((max(nr, 1), 4), dtype=torch.int64, device=dev) if rounds is None else rounds
    finals = torch.empty((L, 3), dtype=torch.int64, device=dev) if finals is None else finals
    _need(tree, torch.int64, (2 << L) - 1, "tree")
    _need(chal, torch.int64, L * (L + 1) // 2, "chal")
    _need(rounds, torch.int64, 4 * nr, "rounds")
    _need(finals, torch.int64, 3 * L, "finals")
    need = lib().fp_lookup_prove_workspace(L)
    p, nbytes = _ws_lookup.get(need)
    _check(lib().fp_lookup_prove(_ptr(tree), L, _ptr(chal), _ptr(rounds), _ptr(finals), p, nbytes, _stream()),
           "fp_lookup_prove")
    return rounds[:nr], finals


# ---------------------------------------------- soundness-faithful challenges --
def fs_init(state, msg: bytes):
    """state (device uint8 [32], 8-byte aligned) <- BLAKE2b-256(msg), msg <= 128 bytes."""
    _check(lib().fp_fs_init(_ptr(state), msg, len(msg), _stream()), "fp_fs_init")
    return state


def fs_absorb(state, data):
    """state <- BLAKE2b-256(state || data), data a device int64 tensor of words."""
    _check(lib().fp_fs_absorb(_ptr(state), _ptr(data) if data.numel() else None, data.numel(), _stream()),
           "fp_fs_absorb")
    return state


def fs_challenges(state, k: int, out=None):
    """k extension challenges [k, 2] read from the state."""
    out = torch.empty((max(k, 1), 2), dtype=torch.int64, device=state.device) if out is None else out
    _check(lib().fp_fs_challenges(_ptr(state), k, _ptr(out), _stream()), "fp_fs_challenges")
    return out[:k]


def eq_table_ext(r, E0=None, E1=None):
    """(E0, E1): eq over the extension at r [n, 2]."""
    n = r.shape[0]
    dev = r.device
    E0 = torch.empty(1 << n, dtype=torch.int64, device=dev) if E0 is None else E0
    E1 = torch.empty(1 << n, dtype=torch.int64, device=dev) if E1 is None else E1
    _check(lib().fp_eq_table_ext(_ptr(r) if n else None, n, _ptr(E0), _ptr(E1), _stream()), "fp_eq_table_ext")
    return E0, E1


def ext_claim_combine(c4, c0=None):
    c0 = torch.empty(2, dtype=torch.int64, device=c4.device) if c0 is None else c0
    _check(lib().fp_ext_claim_combine(_ptr(c4), _ptr(c0), _stream()), "fp_ext_claim_combine")
    return c0


def sumcheck_ext_fs(A0, A1, B0, B1, state, rounds=None, r=None, finals=None):
    """Extension sum-check with the transcript: rounds [n, 3, 2], r [n, 2], finals [2, 2]."""
    n = A0.numel().bit_length() - 1
    dev = A0.device
    rounds = torch.empty((max(n, 1), 3, 2), dtype=torch.int64, device=dev) if rounds is None else rounds
    r = torch.empty((max(n, 1), 2), dtype=torch.int64, device=dev) if r is None else r
    finals = torch.empty((2, 2), dtype=torch.int64, device=dev) if finals is None else finals
    _check(lib().fp_sumcheck_ext_fs(_ptr(A0), _ptr(A1), _ptr(B0), _ptr(B1), n, _ptr(state), _ptr(rounds), _ptr(r),
                                    _ptr(finals), _stream()), "fp_sumcheck_ext_fs")
    return rounds[:n], r[:n], finals


def sumcheck_ext_fs_multi(A0s, A1s, B0s, B1s, state, rho=None, rounds=None, r=None, finals=None):
    """Extension sum-check of sum_j rho_j sum_k A_j[k] B_j[k] (A_j = A0s[j] + u A1s[j], 1..8 pairs of int64
    [2^n] tables; rho device [n_pairs, 2] or None) with the transcript: rounds [n, 3, 2], r [n, 2],
    finals [n_pairs, 2, 2]."""
    k = len(A0s)
    assert 1 <= k <= 8 and len(A1s) == len(B0s) == len(B1s) == k
    N = A0s[0].numel()
    n = N.bit_length() - 1
    assert N == 1 << n
    for t in list(A0s) + list(A1s) + list(B0s) + list(B1s):
        _need(t, torch.int64, N, "sum-check table")
    dev = A0s[0].device
    rounds = torch.empty((max(n, 1), 3, 2), dtype=torch.int64, device=dev) if rounds is None else rounds
    r = torch.empty((max(n, 1), 2), dtype=torch.int64, device=dev) if r is None else r
    finals = torch.empty((k, 2, 2), dtype=torch.int64, device=dev) if finals is None else finals
    _need(rounds, torch.int64, 6 * n, "rounds")
    _need(r, torch.int64, 2 * n, "r")
    _need(finals, torch.int64, 4 * k, "finals")
    assert state.is_contiguous() and state.numel() * state.element_size() >= 32, "state: 32 bytes"
    if rho is not None:
        _need(rho, torch.int64, 2 * k, "rho")
    arr = lambda ts: (ctypes.c_void_p * k)(*[t.data_ptr() for t in ts])
    p, nb = _ws_scx.get(lib().fp_sumcheck_ext_fs_multi_workspace(k, n))
    _check(lib().fp_sumcheck_ext_fs_multi(k, arr(A0s), arr(A1s), arr(B0s), arr(B1s), _ptr(rho), n, _ptr(state),
                                          _ptr(rounds), _ptr(r), _ptr(finals), p, nb, _stream()),
           "fp_sumcheck_ext_fs_multi")
    return rounds[:n], r[:n], finals


def commit_tables(maps, n_t: int, s: int, msg):
    """Each map's Q (before the clamp), R and Y as zero-padded [2^n_t, 2^n_o] field tables in whole rows of
    msg [rows, 2^L]; maps: (Z int32 [T, d_out], n_o, row_q, row_r, row_y)."""
    rows, cols = msg.shape
    L = cols.bit_length() - 1
    assert 1 << L == cols and msg.is_contiguous() and msg.dtype == torch.int64
    descs = []
    for Z, n_o, rq, rr, ry in maps:
        T, d_out = Z.shape
        _need(Z, torch.int32, T * d_out, "Z")
        descs.append(_TableDesc(_ptr(Z) if Z.numel() else None, max(d_out, 1), T, d_out, n_o, rq, rr, ry))
    arr = (_TableDesc * len(descs))(*descs)
    _check(lib().fp_commit_tables(len(descs), arr, n_t, s, L, _ptr(msg), cols, rows, _stream()), "fp_commit_tables")
    return msg


def commit_fold_ext(msg, r_prox, claims, U):
    """Folded rows over the extension of msg [rows, 2^L]: U [1 + len(claims), 2, 2^L] receives the proximity row
    (row weights eq(r_prox, i); r_prox [n_prox, 2]) and each claim's row; claims: (row0, z1 [n1, 2], z2 [n2, 2])
    with 2^(n1 + n2) rows from row0, sorted and disjoint."""
    rows, cols = msg.shape
    L = cols.bit_length() - 1
    assert 1 << L == cols and msg.is_contiguous() and msg.dtype == torch.int64
    _need(U, torch.int64, (1 + len(claims)) * 2 * cols, "U")
    cs = []
    for row0, z1, z2 in claims:
        n1, n2 = z1.shape[0], z2.shape[0]
        for z in (z1, z2):
            assert z.dtype == torch.int64 and (z.numel() == 0 or z.is_contiguous())
        cs.append(_OpenClaim(row0, 1 << (n1 + n2), _ptr(z1) if n1 else None, n1, _ptr(z2) if n2 else None, n2))
    arr = (_OpenClaim * max(1, len(cs)))(*cs)
    n_prox = r_prox.shape[0]
    assert r_prox.dtype == torch.int64 and r_prox.is_contiguous()
    p, nb = _ws_open.get(lib().fp_commit_fold_ext_workspace(rows))
    _check(lib().fp_commit_fold_ext(_ptr(msg), cols, rows, L, _ptr(r_prox) if n_prox else None, n_prox, len(cs), arr,
                                    _ptr(U), p, nb, _stream()), "fp_commit_fold_ext")
    return U


def merkle_open(code, salts, tree, chal, cols=None, col_salts=None, paths=None, idx=None):
    """Columns j = chal[q, 0] mod W of code [rows, W] with their salts and Merkle paths: cols [nq, rows] int64,
    col_salts [nq, 16] uint8, paths [nq, log2 W, 32] uint8, idx [nq] int32."""
    rows, W = code.shape
    logw = W.bit_length() - 1
    nq = chal.shape[0]
    assert 1 << logw == W and code.is_contiguous() and chal.dtype == torch.int64 and chal.is_contiguous()
    _need(salts, torch.uint8, W * SALT_BYTES, "salts")
    _need(tree, torch.uint8, (2 * W - 1) * DIGEST_BYTES, "tree")
    dev = code.device
    cols = torch.empty((nq, rows), dtype=torch.int64, device=dev) if cols is None else cols
    col_salts = torch.empty((nq, SALT_BYTES), dtype=torch.uint8, device=dev) if col_salts is None else col_salts
    paths = torch.empty((nq, logw, DIGEST_BYTES), dtype=torch.uint8, device=dev) if paths is None else paths
    idx = torch.empty(nq, dtype=torch.int32, device=dev) if idx is None else idx
    _need(cols, torch.int64, nq * rows, "cols")
    _need(col_salts, torch.uint8, nq * SALT_BYTES, "col_salts")
    _need(paths, torch.uint8, nq * logw * DIGEST_BYTES, "paths")
    _need(idx, torch.int32, nq, "idx")
    _check(lib().fp_merkle_open(_ptr(code), W, rows, logw, _ptr(salts), _ptr(tree), _ptr(chal), nq, _ptr(cols),
                                _ptr(col_salts), _ptr(paths), _ptr(idx), _stream()), "fp_merkle_open")
    return cols, col_salts, paths, idx


def mle_eval(M, r_rows, r_cols, out=None):
    rows, cols = M.shape
    out = torch.empty(1, dtype=torch.int64, device=M.device) if out is None else out
    nr, nc = r_rows.numel(), r_cols.numel()
    need = lib().fp_mle_eval_workspace(_dt(M), rows, cols, nr, nc)
    p, nb = _ws_mle.get(need)
    _check(lib().fp_mle_eval(_dt(M), _ptr(M), _ld(M), rows, cols, _ptr(r_rows) if nr else None, nr,
                             _ptr(r_cols) if nc else None, nc, _ptr(out), p, nb, _stream()), "fp_mle_eval")
    return out


# ---------------------------------------------------------------- sum-check --
def sumcheck_prove(As, Bs, r, rho=None, rounds=None, finals=None, claim0=None):
    k = len(As)
    n = r.numel()
    dev = r.device
    rounds = torch.empty((n, 3), dtype=torch.int64, device=dev) if rounds is None else rounds
    finals = torch.empty((k, 2), dtype=torch.int64, device=dev) if finals is None else finals
    claim0 = torch.empty(1, dtype=torch.int64, device=dev) if claim0 is None else claim0
    pa = (ctypes.c_void_p * k)(*[a.data_ptr() for a in As])
    pb = (ctypes.c_void_p * k)(*[b.data_ptr() for b in Bs])
    need = lib().fp_sumcheck_workspace(k, n)
    p, nb = _ws_sc.get(need)
    _check(lib().fp_sumcheck_prove(k, pa, pb, _ptr(rho), n, _ptr(r), _ptr(rounds), _ptr(finals), _ptr(claim0),
                                   p, nb, _stream()), "fp_sumcheck_prove")
    return rounds, finals, claim0


def sumcheck_prove_multi(A, B, r, rounds=None, finals=None, claim0=None):
    n_inst, m = A.shape
    n = r.shape[1]
    assert m == 1 << n
    dev = A.device
    rounds = torch.empty((n_inst, n, 3), dtype=torch.int64, device=dev) if rounds is None else rounds
    finals = torch.empty((n_inst, 2), dtype=torch.int64, device=dev) if finals is None else finals
    claim0 = torch.empty(n_inst, dtype=torch.int64, device=dev) if claim0 is None else claim0
    _check(lib().fp_sumcheck_prove_multi(n_inst, n, _ptr(A), _ptr(B), _ptr(r), _ptr(rounds), _ptr(finals),
                                         _ptr(claim0), _stream()), "fp_sumcheck_prove_multi")
    return rounds, finals, claim0


def combine_claims(g_last, x_last, rho, out=None):
    """out = sum_j rho[j] g_j(x_j); g_last[j]: device view of 3 values, x_last[j]: view of 1."""
    k = len(g_last)
    out = torch.empty(1, dtype=torch.int64, device=rho.device) if out is None else out
    pg = (ctypes.c_void_p * k)(*[g.data_ptr() for g in g_last])
    px = (ctypes.c_void_p * k)(*[x.data_ptr() for x in x_last])
    _check(lib().fp_combine_claims(k, pg, px, _ptr(rho), _ptr(out), _stream()), "fp_combine_claims")
    return out


def claim_eval_batched(jobs):
    """jobs: list of (M, E_rows, E_cols, out); out_j = sum E_rows[t] E_cols[c] M[t, c]."""
    k = len(jobs)
    dt = _dt(jobs[0][0])
    descs = (_ClaimDesc * k)(*[_ClaimDesc(M.data_ptr(), _ld(M), M.shape[0], M.shape[1], Er.data_ptr(),
                                          Ec.data_ptr(), out.data_ptr()) for (M, Er, Ec, out) in jobs])
    need = lib().fp_claim_eval_batched_workspace(dt, k, descs)
    p, nb = _ws_claim.get(need)
    _check(lib().fp_claim_eval_batched(dt, k, descs, p, nb, _stream()), "fp_claim_eval_batched")
    return [j[3] for j in jobs]


def fold_claim_batched(fold_jobs, claim_jobs):
    """One pass over fold jobs (M, E, cols_pad, out) of one dtype and claim jobs
    (M, E_rows, E_cols, out) of one dtype; outputs as fold_matrix_batched and
    claim_eval_batched."""
    nf, nc = len(fold_jobs), len(claim_jobs)
    fdt = _dt(fold_jobs[0][0]) if nf else FP_I8
    cdt = _dt(claim_jobs[0][0]) if nc else FP_I32
    fd = (_FoldDesc * max(nf, 1))(*[_fold_desc(f) for f in fold_jobs])
    cd = (_ClaimDesc * max(nc, 1))(*[_ClaimDesc(M.data_ptr(), _ld(M), M.shape[0], M.shape[1], Er.data_ptr(),
                                                Ec.data_ptr(), out.data_ptr()) for (M, Er, Ec, out) in claim_jobs])
    need = lib().fp_fold_claim_batched_workspace(fdt, nf, fd, cdt, nc, cd)
    p, nb = _ws_fold.get(need)
    _check(lib().fp_fold_claim_batched(fdt, nf, fd, cdt, nc, cd, p, nb, _stream()), "fp_fold_claim_batched")
    return [j[3] for j in fold_jobs], [j[3] for j in claim_jobs]


def linear_combine(vals, rho, out=None):
    k = len(vals)
    out = torch.empty(1, dtype=torch.int64, device=rho.device) if out is None else out
    pv = (ctypes.c_void_p * k)(*[v.data_ptr() for v in vals])
    _check(lib().fp_linear_combine(k, pv, _ptr(rho), _ptr(out), _stream()), "fp_linear_combine")
    return out
