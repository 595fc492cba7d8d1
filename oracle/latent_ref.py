"""fp64 definitions of the 8-bit latent cache and of latent attention over a
shared prefix and a sequence's own rows (include/mla.h: mla_set_cache_dtype,
mla_latent_attn). Plain loops and tables; none of the CUDA path's code."""
from __future__ import annotations

import math

import numpy as np

K_MIN, K_MAX = -64, 7


def e4m3_value(code: int) -> float:
    """The value of one E4M3 (OCP) code: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    e, f = (code >> 3) & 15, code & 7
    if e == 15 and f == 7:
        return math.nan
    v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
    return -v if code & 128 else v


E4M3 = np.array([e4m3_value(c) for c in range(256)])


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest code (ties to the even code, saturating at 448); NaN for NaN and infinities. uint8."""
    pos = E4M3[:127]
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448.0, 126, code).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def scale_exponent(latent: np.ndarray) -> int:
    fine = np.abs(latent[np.isfinite(latent)])
    amax = float(fine.max()) if fine.size else 0.0
    if amax == 0.0:
        return 0
    for k in range(K_MIN, K_MAX):
        if amax <= 448.0 * 2.0 ** k:
            return k
    return K_MAX


def quantise_row(latent: np.ndarray):
    """(codes uint8 [r_kv], k) of one latent row: values E4M3[codes] * 2**k."""
    k = scale_exponent(latent)
    return e4m3_round(np.asarray(latent, np.float64) * 2.0 ** -k), k


def block_layout(block_size: int, r_kv: int, d_r: int, esz: int):
    """(offset of the rotary plane, of the scales, bytes of a block)."""
    pe = block_size * r_kv
    sc = pe + block_size * d_r * esz
    return pe, sc, -(-(sc + 4 * block_size) // 128) * 128


def latent_attention(q_abs, q_pe, latent, k_pe, scale, sink=None):
    """One sequence: q_abs [H, r], q_pe [H, d], keys latent [L, r], k_pe [L, d] (fp64).
    Returns (o [H, r], lse [H], p [H, L] normalised). No keys: o 0, lse -inf (the sink's)."""
    H, L = q_abs.shape[0], latent.shape[0]
    s = (q_abs @ latent.T + q_pe @ k_pe.T) * scale if L else np.zeros((H, 0))
    z = np.full(H, -np.inf) if sink is None else np.asarray(sink, np.float64)
    m = np.maximum(s.max(1) if L else np.full(H, -np.inf), z)
    safe = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - safe[:, None])
    den = e.sum(1) + np.exp(z - safe)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.where(den > 0, safe + np.log(den), -np.inf)
        p = np.where(den[:, None] > 0, e / den[:, None], 0.0)
    return p @ latent if L else np.zeros((H, latent.shape[1])), lse, p
