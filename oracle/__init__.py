"""CPU oracle for the quantized message-passing layer -- TEST INFRASTRUCTURE.

Only the tests, the smoke check and the benchmark's CPU-baseline leg use this
package.  The CUDA library never imports, links or calls it, and it never
imports the CUDA library.

The loops live in plain C (gq_oracle.c, built with -ffp-contract=off and
OpenMP over output rows); dense products use numpy's float64 matmul as the
library primitive.  All values are float64 except the quantizer, whose fp32
arithmetic is part of its specification.

Routines follow:
  AdaQP (arXiv 2306.01381) Sec. 2.1 weighted-sum layer, Sec. 2.3 Eqn 4-6
      (stochastic integer quantization / de-quantization), Sec. 3.1 (only
      boundary messages are quantized);
  Sancus (IJCAI 2023) Sec. 2: normalized adjacency D~^-1/2 (A+I) D~^-1/2;
  Tango (arXiv 2308.00890) Sec. 2.1, Fig. 1: GAT forward/backward steps;
  AdaQP Sec. 4.2 (Problem 11): per-message variance weight beta_k, and
      the width choice of Problems 10-12 on one device;
  Tango Sec. 3.2 (Eq. 4): relative quantization error Error_X and the
      bit-count rule built on it;
  Tango Sec. 3.3: the SpMM's edge values quantized at 8 bits (one AdaQP
      Eqn 4 vector per destination and head).

Parity status: every routine is pinned by tests/test_oracle_*.py against the
Tango worked example, closed forms, dense brute force or finite differences,
except the single printed head-2 value of dD in the Tango example, whose
inputs the page does not print (parity unpinned for that number only).
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_SRC = os.path.join(_HERE, "gq_oracle.c")
_BUILD = os.path.join(_HERE, "_build")
_LIB_PATH = os.path.join(_BUILD, "libgq_oracle.so")
_lock = threading.Lock()
_lib = None

COEF_GCN, COEF_SAGE, COEF_ONE = 0, 1, 2


def build(force: bool = False) -> str:
    """Compile the C oracle (gcc, portable C, no target-specific flags)."""
    os.makedirs(_BUILD, exist_ok=True)
    if (not force and os.path.exists(_LIB_PATH)
            and os.path.getmtime(_LIB_PATH) >= os.path.getmtime(_SRC)):
        return _LIB_PATH
    tmp = _LIB_PATH + f".tmp{os.getpid()}"
    cmd = ["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-fno-fast-math", "-fopenmp",
           "-fPIC", "-shared", _SRC, "-o", tmp, "-lm"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, _LIB_PATH)
    return _LIB_PATH


def _L():
    global _lib
    with _lock:
        if _lib is None:
            lib = ctypes.CDLL(build())
            P, I64, I, U64, D = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                 ctypes.c_uint64, ctypes.c_double)
            sig = {
                "orc_fmix32": ([ctypes.c_uint32], ctypes.c_uint32),
                "orc_hash": ([U64, ctypes.c_uint32, ctypes.c_uint32], ctypes.c_uint32),
                "orc_uniform": ([U64, ctypes.c_uint32, ctypes.c_uint32], ctypes.c_float),
                "orc_payload_bytes": ([I, I], I64),
                "orc_header_offset": ([I, I], I64),
                "orc_pitch": ([I, I], I64),
                "orc_quantize": ([P, I64, I, I64, P, I, U64, P], None),
                "orc_quantize_rows": ([P, I64, I, I64, P, I, U64, P], None),
                "orc_spmm_rows": ([I64, P, P, I, I, I64, P, I64, P, P, I, P], I),
                "orc_dequant": ([P, I64, I, I, P, P, I64], None),
                "orc_codes": ([P, I64, I, I, P], None),
                "orc_degree_norms": ([I64, P, P, P, P, P], None),
                "orc_spmm": ([I64, P, P, I, P, I, P], None),
                "orc_spmm_t": ([I64, P, P, I, P, I, P], None),
                "orc_head_proj": ([I64, I, I, P, P, P], None),
                "orc_edge_softmax": ([I64, P, P, P, P, I, D, P, P], None),
                "orc_edge_spmm": ([I64, P, P, P, I, P, I, P], None),
                "orc_edge_spmm_t": ([I64, P, P, P, I, P, I, P], None),
                "orc_sddmm_dot": ([I64, P, P, P, P, I, I, P], None),
                "orc_edge_softmax_bwd": ([I64, P, P, P, P, I, D, P, P, P], None),
                "orc_edge_segment_sums": ([I64, P, P, P, I, P, P], None),
                "orc_beta": ([I64, P, P, I, P, I, P], None),
                "orc_quant_error": ([P, I64, I, P, P, I, D], D),
                "orc_quantize_edge_values": ([I64, P, P, I, U64, P, P], None),
                "orc_assign_bits": ([P, P, I64, I, D, D, P], None),
                "orc_dequant_edge_values": ([I64, P, P, P, I, P], None),
            }
            for name, (args, res) in sig.items():
                f = getattr(lib, name)
                f.argtypes = args
                f.restype = res
            _lib = lib
    return _lib


def _p(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _c(a, dtype):
    return np.ascontiguousarray(np.asarray(a), dtype=dtype)


def num_threads() -> int:
    """OpenMP threads the oracle's parallel loops use."""
    n = os.environ.get("OMP_NUM_THREADS")
    if n:
        return int(n)
    return len(os.sched_getaffinity(0))


# --------------------------------------------------------------------------
# quantization (AdaQP Sec. 2.3)
# --------------------------------------------------------------------------

def pitch(d: int, bits: int) -> int:
    return int(_L().orc_pitch(d, bits))


def header_offset(d: int, bits: int) -> int:
    return int(_L().orc_header_offset(d, bits))


def uniform(seed: int, row: int, col: int) -> float:
    return float(_L().orc_uniform(seed, row, col))


def fmix32(h: int) -> int:
    return int(_L().orc_fmix32(h))


def hash32(seed: int, row: int, col: int) -> int:
    return int(_L().orc_hash(seed, row, col))


def quantize(X, mask, bits: int, seed: int, out: np.ndarray | None = None) -> np.ndarray:
    """Packed rows (n x pitch bytes).  Rows with mask 0 are left as in `out`
    (zeros when `out` is None)."""
    X = _c(X, np.float32)
    n, d = X.shape
    m = None if mask is None else _c(mask, np.uint8)
    if out is None:
        out = np.zeros((n, pitch(d, bits)), dtype=np.uint8)
    _L().orc_quantize(_p(X), n, d, d, _p(m), bits, seed & 0xFFFFFFFFFFFFFFFF, _p(out))
    return out


def quantize_rows(X, ids, bits: int, seed: int) -> np.ndarray:
    """The quantizer on a list of rows: row k of X is node ids[k], whose id
    keys its noise, so the bytes equal rows ids[k] of quantize() on the
    whole matrix.  Returns len(ids) x pitch bytes."""
    X = _c(X, np.float32)
    k, d = X.shape
    ids = _c(ids, np.int64)
    assert ids.shape == (k,)
    out = np.zeros((k, pitch(d, bits)), dtype=np.uint8)
    _L().orc_quantize_rows(_p(X), k, d, d, _p(ids), bits, seed & 0xFFFFFFFFFFFFFFFF, _p(out))
    return out


def dequant(packed, d: int, bits: int, mask=None) -> np.ndarray:
    packed = _c(packed, np.uint8)
    n = packed.shape[0]
    m = None if mask is None else _c(mask, np.uint8)
    Y = np.zeros((n, d), dtype=np.float32)
    _L().orc_dequant(_p(packed), n, d, bits, _p(m), _p(Y), d)
    return Y


def codes(packed, d: int, bits: int) -> np.ndarray:
    packed = _c(packed, np.uint8)
    n = packed.shape[0]
    Q = np.zeros((n, d), dtype=np.int32)
    _L().orc_codes(_p(packed), n, d, bits, _p(Q))
    return Q


def header(packed, d: int, bits: int):
    """(S, mn) per row as float32 arrays."""
    h = header_offset(d, bits)
    packed = _c(packed, np.uint8)
    S = packed[:, h:h + 4].copy().view(np.float32).reshape(-1)
    mn = packed[:, h + 4:h + 8].copy().view(np.float32).reshape(-1)
    return S, mn


def messages(X, packed, mask, d: int, bits: int) -> np.ndarray:
    """The message rows an aggregation reads (AdaQP Sec. 3.1): de-quantized
    rows where the node is marginal, the full-precision row otherwise.
    bits >= 32 means no quantization.  Returns float64."""
    M = np.array(X, dtype=np.float32, copy=True)
    if bits < 32:
        deq = dequant(packed, d, bits)
        sel = np.ones(M.shape[0], bool) if mask is None else np.asarray(mask).astype(bool)
        M[sel] = deq[sel]
    return M.astype(np.float64)


def quantize_mixed(X, rbits, seed: int):
    """Mixed bit-widths per row: row r with width rbits[r] in {2, 4, 8} is
    quantized at that width (the same bytes quantize() gives row r) and laid
    at byte roff[r]; other rows take no bytes.  Returns (packed, roff)."""
    X = _c(X, np.float32)
    n, d = X.shape
    rbits = np.asarray(rbits).astype(np.int64)
    sizes = np.array([pitch(d, int(b)) if b in (2, 4, 8) else 0 for b in rbits], np.int64)
    roff = np.zeros(n + 1, np.int64)
    roff[1:] = np.cumsum(sizes)
    packed = np.zeros(int(roff[-1]), np.uint8)
    for b in (2, 4, 8):
        sel = rbits == b
        if sel.any():
            rows = quantize(X, sel.astype(np.uint8), b, seed)
            for r in np.nonzero(sel)[0]:
                packed[roff[r]:roff[r + 1]] = rows[r]
    return packed, roff


def messages_mixed(X, packed, roff, rbits, d: int) -> np.ndarray:
    """The message rows an aggregation reads from a mixed buffer: row r
    de-quantized at its width rbits[r], or X[r] for a full-precision row."""
    M = np.array(X, dtype=np.float32, copy=True)
    packed = np.asarray(packed, np.uint8)
    for r, b in enumerate(np.asarray(rbits).astype(np.int64)):
        if b in (2, 4, 8):
            M[r] = dequant(packed[roff[r]:roff[r + 1]][None, :], d, int(b))[0]
    return M.astype(np.float64)


# --------------------------------------------------------------------------
# graph normalization and aggregation
# --------------------------------------------------------------------------

def degree_norms(rowptr, col):
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    n = rowptr.shape[0] - 1
    a, b, c = (np.zeros(n, np.float32) for _ in range(3))
    _L().orc_degree_norms(n, _p(rowptr), _p(col), _p(a), _p(b), _p(c))
    return a, b, c


def spmm(rowptr, col, coef: int, M, transpose: bool = False) -> np.ndarray:
    """Y = A^ M (transpose=False) or A^T M (transpose=True), float64."""
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    M = _c(M, np.float64)
    n = rowptr.shape[0] - 1
    d = M.shape[1]
    Y = np.zeros((n, d), dtype=np.float64)
    f = _L().orc_spmm_t if transpose else _L().orc_spmm
    f(n, _p(rowptr), _p(col), coef, _p(M), d, _p(Y))
    return Y


def spmm_rows(rowptr, col, coef: int, rows, ids, M, transpose: bool = False) -> np.ndarray:
    """spmm() evaluated at the output rows `rows` only (ascending node ids),
    coefficients from the degrees of the whole graph.  M[i] is the message
    row of node ids[i] (ids ascending); every node an output row reads must
    be listed.  Returns len(rows) x d, float64."""
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    rows = _c(rows, np.int64)
    ids = _c(ids, np.int64)
    M = _c(M, np.float64)
    n = rowptr.shape[0] - 1
    d = M.shape[1]
    assert M.shape[0] == ids.shape[0]
    assert np.all(np.diff(rows) > 0) and np.all(np.diff(ids) > 0)
    Y = np.zeros((rows.shape[0], d), dtype=np.float64)
    rc = _L().orc_spmm_rows(n, _p(rowptr), _p(col), coef, 1 if transpose else 0, rows.shape[0], _p(rows),
                            ids.shape[0], _p(ids), _p(M), d, _p(Y))
    if rc != 0:
        raise ValueError("spmm_rows: a message row the output rows read is not among ids")
    return Y


# --------------------------------------------------------------------------
# message-level quantization metrics (AdaQP Sec. 4.2; Tango Sec. 3.2)
# --------------------------------------------------------------------------

def beta(rowptr, col, coef: int, X) -> np.ndarray:
    """AdaQP's variance weight of every message row (Problem 11):
    beta_k = sum_{v: k->v} a_{k,v}^2 * d * (max X[k] - min X[k])^2 / 6."""
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    X = _c(X, np.float32)
    n, d = X.shape
    out = np.zeros(n, np.float64)
    _L().orc_beta(n, _p(rowptr), _p(col), coef, _p(X), d, _p(out))
    return out


def quant_error(X, packed, mask, bits: int, eps: float = 5e-4) -> float:
    """Tango's relative quantization error Error_X of the tensor X against
    its quantized rows (Eq. 4), with |X| + |Xq| + eps as denominator."""
    X = _c(X, np.float32)
    n, d = X.shape
    packed = _c(packed, np.uint8)
    m = None if mask is None else _c(mask, np.uint8)
    return float(_L().orc_quant_error(_p(X), n, d, _p(packed), _p(m), bits, eps))


def assign_bits(beta, d: int, lam: float, gamma: float, mask=None) -> np.ndarray:
    """AdaQP Sec. 4.2 Problems 10-12 on one device: per row, the width in
    {2, 4, 8} minimizing lam * beta / (2^b - 1)^2 + (1 - lam) * gamma * d * b
    (fp64, ties to the fewer bits); rows with mask 0 get 0 (full
    precision).  uint8 per row, the rbits of quantize_mixed."""
    beta = _c(beta, np.float32)
    n = beta.shape[0]
    m = None if mask is None else _c(mask, np.uint8)
    out = np.zeros(n, np.uint8)
    _L().orc_assign_bits(_p(beta), _p(m), n, d, float(lam), float(gamma), _p(out))
    return out


def bits_for_error(X, mask, seed: int, threshold: float = 0.3, eps: float = 5e-4, choices=(2, 4, 8)) -> int:
    """Tango's rule: the fewest bits whose Error_X stays below the threshold
    (the largest choice if none does)."""
    for b in choices:
        if quant_error(X, quantize(X, mask, b, seed), mask, b, eps) < threshold:
            return b
    return choices[-1]


# --------------------------------------------------------------------------
# dense products
# --------------------------------------------------------------------------

def bf16_round(x) -> np.ndarray:
    """Round float32 values to bfloat16 (nearest, ties to even), returned as
    float32.  Inputs are first rounded to float32."""
    f = np.ascontiguousarray(x, dtype=np.float32)
    b = f.view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    return (b & 0xFFFFFFFF).astype(np.uint32).view(np.float32).reshape(f.shape)


def gemm(A, B, bf16: bool) -> np.ndarray:
    """A @ B in float64; with bf16=True both operands are first rounded to
    bfloat16 (the tensor-core input precision)."""
    if bf16:
        A, B = bf16_round(A), bf16_round(B)
    return np.asarray(A, np.float64) @ np.asarray(B, np.float64)


# --------------------------------------------------------------------------
# GCN / GraphSAGE layer (AdaQP Sec. 2.1; Sancus Sec. 2)
# --------------------------------------------------------------------------

def gcn_layer_fwd(rowptr, col, coef, H_in, W, mask, bits, seed, relu: bool, bf16: bool = True):
    """Aggregate first, then update:  A = sum_u a_uv m_u,  Z = A W,
    H_out = relu(Z).  Messages of marginal rows are quantized (bits < 32)."""
    H_in = _c(H_in, np.float32)
    d = H_in.shape[1]
    packed = quantize(H_in, mask, bits, seed) if bits < 32 else None
    M = messages(H_in, packed, mask, d, bits)
    A = spmm(rowptr, col, coef, M)
    Z = gemm(A, W, bf16)
    H_out = np.maximum(Z, 0.0) if relu else Z
    return dict(packed=packed, A=A, Z=Z, H_out=H_out)


def gcn_layer_bwd(rowptr, col, coef, dH_out, A, Z, W, mask, bits, seed, relu: bool,
                  bf16: bool = True, need_dinput: bool = True):
    """dZ = dH_out * relu'(Z); dW = A^T dZ; dA = dZ W^T; the rows of dA of
    marginal nodes travel quantized (bits < 32); dH_in = A^T-aggregation of
    those messages.  The quantizer is the identity in backward (its codes
    are treated as constants)."""
    dZ = np.asarray(dH_out, np.float64) * ((np.asarray(Z) > 0) if relu else 1.0)
    dW = gemm(np.asarray(A).T, dZ, bf16)
    out = dict(dZ=dZ, dW=dW)
    if need_dinput:
        dA = gemm(dZ, np.asarray(W).T, bf16).astype(np.float32)
        d = dA.shape[1]
        packed = quantize(dA, mask, bits, seed) if bits < 32 else None
        M = messages(dA, packed, mask, d, bits)
        out.update(dA=dA, packed=packed, dH_in=spmm(rowptr, col, coef, M, transpose=True))
    return out


# --------------------------------------------------------------------------
# GAT (Tango Sec. 2.1, Fig. 1)
# --------------------------------------------------------------------------

def head_proj(Hp, a, heads: int) -> np.ndarray:
    Hp = _c(Hp, np.float64)
    a = _c(a, np.float64)
    n, d = Hp.shape
    out = np.zeros((n, heads), np.float64)
    _L().orc_head_proj(n, heads, d // heads, _p(Hp), _p(a), _p(out))
    return out


def edge_softmax(rowptr, col, S, D, slope: float):
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    S = _c(S, np.float64)
    D = _c(D, np.float64)
    n, heads = D.shape
    E = int(rowptr[-1])
    Epre = np.zeros((E, heads), np.float64)
    alpha = np.zeros((E, heads), np.float64)
    _L().orc_edge_softmax(n, _p(rowptr), _p(col), _p(S), _p(D), heads, slope, _p(Epre), _p(alpha))
    return Epre, alpha


def edge_spmm(rowptr, col, alpha, M, transpose: bool = False) -> np.ndarray:
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    alpha = _c(alpha, np.float64)
    M = _c(M, np.float64)
    n = rowptr.shape[0] - 1
    heads = alpha.shape[1]
    d = M.shape[1]
    out = np.zeros((n, d), np.float64)
    f = _L().orc_edge_spmm_t if transpose else _L().orc_edge_spmm
    f(n, _p(rowptr), _p(col), _p(alpha), heads, _p(M), d, _p(out))
    return out


def quantize_edge_values(rowptr, alpha, seed: int):
    """Tango Sec. 3.3: the SpMM's edge values alpha (E x heads, CSR edge
    order) quantized at 8 bits, one AdaQP Eqn 4 vector per (destination,
    head) segment, u hashed from (seed, edge id, head).  Returns (codes
    uint8 E x heads, hdr float32 n x heads x 2 holding {S, Z})."""
    rowptr = _c(rowptr, np.int32)
    alpha = _c(alpha, np.float32)
    n = rowptr.shape[0] - 1
    E, heads = alpha.shape
    codes = np.zeros((E, heads), np.uint8)
    hdr = np.zeros((n, heads, 2), np.float32)
    _L().orc_quantize_edge_values(n, _p(rowptr), _p(alpha), heads, seed & 0xFFFFFFFFFFFFFFFF, _p(codes), _p(hdr))
    return codes, hdr


def dequant_edge_values(rowptr, codes, hdr) -> np.ndarray:
    """AdaQP Eqn 5 per segment: fmaf(q, S[v,k], Z[v,k]), float32 E x heads."""
    rowptr = _c(rowptr, np.int32)
    codes = _c(codes, np.uint8)
    hdr = _c(hdr, np.float32)
    n = rowptr.shape[0] - 1
    out = np.zeros(codes.shape, np.float32)
    _L().orc_dequant_edge_values(n, _p(rowptr), _p(codes), _p(hdr), codes.shape[1], _p(out))
    return out


def sddmm_dot(rowptr, col, dOut, M, heads: int) -> np.ndarray:
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    dOut = _c(dOut, np.float64)
    M = _c(M, np.float64)
    n = rowptr.shape[0] - 1
    d = M.shape[1]
    E = int(rowptr[-1])
    out = np.zeros((E, heads), np.float64)
    _L().orc_sddmm_dot(n, _p(rowptr), _p(col), _p(dOut), _p(M), heads, d, _p(out))
    return out


def edge_softmax_bwd(rowptr, alpha, dalpha, Epre, slope: float):
    rowptr = _c(rowptr, np.int32)
    alpha = _c(alpha, np.float64)
    dalpha = _c(dalpha, np.float64)
    Ep = None if Epre is None else _c(Epre, np.float64)
    n = rowptr.shape[0] - 1
    E, heads = alpha.shape
    P = np.zeros((n, heads), np.float64)
    dE = np.zeros((E, heads), np.float64)
    dEpre = np.zeros((E, heads), np.float64)
    _L().orc_edge_softmax_bwd(n, _p(rowptr), _p(alpha), _p(dalpha), _p(Ep), heads, slope,
                              _p(P), _p(dE), _p(dEpre))
    return P, dE, dEpre


def edge_segment_sums(rowptr, col, X):
    rowptr = _c(rowptr, np.int32)
    col = _c(col, np.int32)
    X = _c(X, np.float64)
    n = rowptr.shape[0] - 1
    heads = X.shape[1]
    dD = np.zeros((n, heads), np.float64)
    dS = np.zeros((n, heads), np.float64)
    _L().orc_edge_segment_sums(n, _p(rowptr), _p(col), _p(X), heads, _p(dD), _p(dS))
    return dD, dS


# The layer draws the attention values' noise from seed ^ ALPHA_SEED_TAG, so
# that it is independent of the messages' noise drawn with the same seed (a
# fixed choice of this implementation; any constant with that property would
# do).
ALPHA_SEED_TAG = 0x5851F42D4C957F2D


def gat_layer_fwd(rowptr, col, H, W, a_src, a_dst, heads, slope, mask=None, bits=32, seed=0,
                  bf16: bool = True, alpha_bits: int = 32):
    """Tango Fig. 1a: H' = H W (step 1); S, D head projections (step 2);
    SDDMM add + LeakyReLU (step 3); edge softmax (step 4); SpMM (step 5).
    With bits < 32 the H' rows of marginal nodes are the quantized messages;
    with alpha_bits = 8 the SpMM weights are the attention values quantized
    per destination and head (Tango Sec. 3.3), returned as ahat."""
    Hp = gemm(H, W, bf16)
    S = head_proj(Hp, a_src, heads)
    D = head_proj(Hp, a_dst, heads)
    Epre, alpha = edge_softmax(rowptr, col, S, D, slope)
    Hp32 = Hp.astype(np.float32)
    d = Hp.shape[1]
    packed = quantize(Hp32, mask, bits, seed) if bits < 32 else None
    M = messages(Hp32, packed, mask, d, bits) if bits < 32 else Hp
    ahat = alpha
    if alpha_bits == 8:
        acode, ahdr = quantize_edge_values(rowptr, alpha.astype(np.float32), seed ^ ALPHA_SEED_TAG)
        ahat = dequant_edge_values(rowptr, acode, ahdr).astype(np.float64)
    out = edge_spmm(rowptr, col, ahat, M)
    return dict(Hp=Hp, S=S, D=D, Epre=Epre, alpha=alpha, packed=packed, M=M, out=out, ahat=ahat)


def gat_layer_bwd(rowptr, col, dOut, H, M, Hp, Epre, alpha, W, a_src, a_dst, heads, slope,
                  mask=None, bits=32, seed=0, bf16: bool = True, ahat=None):
    """Tango Fig. 1b.  M = the forward messages (H' rows, de-quantized where
    marginal); ahat = the forward's SpMM weights when they were quantized
    (the transposed SpMM uses them; the softmax derivative uses alpha).  dalpha by SDDMM dot; softmax derivative; LeakyReLU'; dD by
    in-edge sums, dS by out-edge sums; dM = transposed edge SpMM of dOut
    (whose marginal rows travel quantized when bits < 32); then
    dH' = dM + dS a_src + dD a_dst, da_src/da_dst, dW = H^T dH', dH = dH' W^T."""
    dOut = np.asarray(dOut, np.float64)
    n, d = dOut.shape
    F = d // heads
    dalpha = sddmm_dot(rowptr, col, dOut, M, heads)
    P, dE, dEpre = edge_softmax_bwd(rowptr, alpha, dalpha, Epre, slope)
    dD, dS = edge_segment_sums(rowptr, col, dEpre)
    dOut32 = dOut.astype(np.float32)
    packed = quantize(dOut32, mask, bits, seed) if bits < 32 else None
    Mb = messages(dOut32, packed, mask, d, bits) if bits < 32 else dOut
    dM = edge_spmm(rowptr, col, alpha if ahat is None else ahat, Mb, transpose=True)
    a_src = np.asarray(a_src, np.float64).reshape(heads, F)
    a_dst = np.asarray(a_dst, np.float64).reshape(heads, F)
    dHp = dM + np.repeat(dS, F, axis=1) * a_src.reshape(1, d) + np.repeat(dD, F, axis=1) * a_dst.reshape(1, d)
    Hp = np.asarray(Hp, np.float64)
    da_src = (dS[:, :, None] * Hp.reshape(n, heads, F)).sum(axis=0)
    da_dst = (dD[:, :, None] * Hp.reshape(n, heads, F)).sum(axis=0)
    dW = gemm(np.asarray(H).T, dHp, bf16)
    dH = gemm(dHp, np.asarray(W).T, bf16)
    return dict(dalpha=dalpha, P=P, dE=dE, dEpre=dEpre, dD=dD, dS=dS, dM=dM, dHp=dHp,
                da_src=da_src, da_dst=da_dst, dW=dW, dH=dH, packed=packed)


# --------------------------------------------------------------------------
# what stands between and behind the layers of a training step: dropout,
# layer normalization, the class head's cross entropy (no page describes
# them; the formulas are written out in each docstring)
# --------------------------------------------------------------------------

def _fmix32_array(h: np.ndarray) -> np.ndarray:
    h = h.astype(np.uint32)
    with np.errstate(over="ignore"):
        h = h ^ (h >> np.uint32(16))
        h = h * np.uint32(0x85EBCA6B)
        h = h ^ (h >> np.uint32(13))
        h = h * np.uint32(0xC2B2AE35)
        return h ^ (h >> np.uint32(16))


def noise_codes(seed: int, n: int, d: int) -> np.ndarray:
    """The 23-bit noise codes (u = code * 2^-23) of rows 0..n-1, columns 0..d-1."""
    key = np.uint32(fmix32((seed ^ (seed >> 32)) & 0xFFFFFFFF))
    rows = _fmix32_array(np.arange(n, dtype=np.uint32) ^ key)
    with np.errstate(over="ignore"):
        cols = np.arange(d, dtype=np.uint32) * np.uint32(0x9E3779B9)
        return _fmix32_array(rows[:, None] + cols[None, :]) >> np.uint32(9)


def kept(seed: int, n: int, d: int, p: float) -> np.ndarray:
    """[u >= p] as booleans; u has 23 bits, so u >= p is code >= p 2^23."""
    return noise_codes(seed, n, d).astype(np.float64) >= p * 2.0 ** 23


def dropout(X, p: float, seed: int) -> np.ndarray:
    """x / (1 - p) where kept, else 0."""
    X = np.asarray(X, np.float64)
    if p == 0.0:
        return X.copy()
    keep = kept(seed, *X.shape, p)
    return np.where(keep, X / (1.0 - p) if p < 1.0 else 0.0, 0.0)


def layer_norm_fwd(X, gamma=None, beta=None, eps: float = 1e-5, relu: bool = False, p: float = 0.0, seed: int = 0):
    """mean = (1/d) sum x; rstd = 1/sqrt((1/d) sum (x - mean)^2 + eps);
    z = (x - mean) rstd gamma + beta; Y = drop(relu(z)).  Also [z > 0]."""
    X = np.asarray(X, np.float64)
    d = X.shape[1]
    mean = X.sum(1) / d
    xc = X - mean[:, None]
    rstd = 1.0 / np.sqrt((xc * xc).sum(1) / d + eps)
    z = xc * rstd[:, None] * (1.0 if gamma is None else np.asarray(gamma, np.float64))
    z = z + (0.0 if beta is None else np.asarray(beta, np.float64))
    y = np.maximum(z, 0.0) if relu else z
    return dict(Y=dropout(y, p, seed), mean=mean, rstd=rstd, z=z, on=z > 0)


def layer_norm_bwd(dY, X, mean, rstd, gamma=None, on=None, p: float = 0.0, seed: int = 0):
    """dz = drop'(dY) where `on` (everywhere when None); dgamma = sum_rows
    dz xhat; dbeta = sum_rows dz; g = dz gamma;
    dX = rstd (g - mean_j g - xhat mean_j(g xhat))."""
    X, dz = np.asarray(X, np.float64), dropout(dY, p, seed)
    if on is not None:
        dz = np.where(on, dz, 0.0)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xhat = (X - np.asarray(mean, np.float64)[:, None]) * rstd
    g = dz * (1.0 if gamma is None else np.asarray(gamma, np.float64))
    dX = rstd * (g - g.mean(1, keepdims=True) - xhat * (g * xhat).mean(1, keepdims=True))
    return dict(dX=dX, dgamma=(dz * xhat).sum(0), dbeta=dz.sum(0), xhat=xhat, dz=dz, g=g)


def linear_xent(X, W, labels, weight=None, scale: float = 1.0):
    """Z = X W^T; for a row with 0 <= label < C: lse = log sum_c exp(z_c),
    loss = lse - z_label, G = weight scale (softmax(z) - onehot(label));
    other rows: lse = loss = 0 and G = 0.  dX = G W, dW = G^T X (rows
    without a label do not enter)."""
    X, W, labels = np.asarray(X, np.float64), np.asarray(W, np.float64), np.asarray(labels)
    n, C = X.shape[0], W.shape[0]
    at = np.nonzero((labels >= 0) & (labels < C))[0]
    lse, loss = np.zeros(n), np.zeros(n)
    Z = X[at] @ W.T
    top = Z.max(1, keepdims=True) if at.size else np.zeros((0, 1))
    E = np.exp(Z - top)
    s = E.sum(1)
    lse[at] = np.log(s) + top[:, 0]
    loss[at] = lse[at] - Z[np.arange(at.size), labels[at]]
    G = E / s[:, None]
    G[np.arange(at.size), labels[at]] -= 1.0
    G *= scale * (np.ones(at.size) if weight is None else np.asarray(weight, np.float64)[at])[:, None]
    dX = np.zeros(X.shape)
    dX[at] = G @ W
    absdX = np.zeros(X.shape)
    absdX[at] = np.abs(G) @ np.abs(W)
    return dict(loss=loss, lse=lse, dX=dX, dW=G.T @ X[at], rows=at, absdX=absdX, absdW=np.abs(G).T @ np.abs(X[at]),
                absZ=(np.abs(X[at]) @ np.abs(W).T).max(1) if at.size else np.zeros(0))
