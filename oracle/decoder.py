"""Plain definitions, in fp64, of the operators between a decoder layer's
linears (include/qaff.h: rmsnorm, rmsnorm_w4a8, kv_cache_append_affine,
kv_cache_read_affine, paged_attention_affine).  Test infrastructure: numpy
loops over rows, no code shared with the HIP path.  Half-precision arrays are
raw 16-bit patterns with a dtype tag, as everywhere in the oracle."""
from __future__ import annotations

import numpy as np

import oracle


def _store(v, dtype: str) -> np.ndarray:
    return oracle.f64_to_bf16(v) if dtype == "bf16" else oracle.f64_to_f16(v)


def rmsnorm(x, resid, weight, eps: float, act: str, w_dtype: str):
    """(h bits, n f64): h = x + resid stored in the activation type (x without resid), n = h / rms(h) * weight."""
    h = x if resid is None else _store(oracle.to_f64(x, act) + oracle.to_f64(resid, act), act)
    hv = oracle.to_f64(h, act)
    rms = np.sqrt((hv * hv).mean(axis=1, keepdims=True) + eps)
    return h, hv / rms * oracle.to_f64(weight, w_dtype)


def quantize_rows(x, act: str, G: int, bits: int):
    """(codes words u32, scales bits, biases bits) of cache rows x [..., D]: each row as quantize_pack_affine has it."""
    D = x.shape[-1]
    N = x.size // D
    w, s, b = oracle.quantize_pack_affine(np.ascontiguousarray(x).reshape(N, D), act, N, D, G, bits, act)
    lead = x.shape[:-1]
    return w.reshape(*lead, -1), s.reshape(*lead, -1), b.reshape(*lead, -1)


def codes(packed, bits: int) -> np.ndarray:
    """Codes of packed words [..., W], lowest column in the low bits: int64 [..., W * 32 / bits]."""
    p = np.ascontiguousarray(packed).view(np.uint32)
    out = np.empty((*p.shape, 32 // bits), np.int64)
    for i in range(32 // bits):
        out[..., i] = (p >> np.uint32(bits * i)) & np.uint32(2**bits - 1)
    return out.reshape(*p.shape[:-1], -1)


def values(packed, scales, biases, dtype: str, G: int, bits: int) -> np.ndarray:
    """code * scale + bias, fp64."""
    c = codes(packed, bits).astype(np.float64)
    return c * np.repeat(oracle.to_f64(scales, dtype), G, -1) + np.repeat(oracle.to_f64(biases, dtype), G, -1)


def paged_attention(q, k, v, dtype: str, G: int, bits: int, table, lens, scale: float, window: int = 0):
    """q bits [B, H, D]; k, v triples over [pages, kv_heads, page_size, ...]; returns (out f64 [B, H, D], bound).

    `bound` is how far a kernel may be off before its output's rounding, when
    it multiplies integer codes by 16-bit rounded weights and sums in fp32:
      - each weight p*s rounded to 11 bits:    2^-11 * sum p s code
      - a logit off by delta changes p by a factor within 1 +- 2 delta (for
        delta < 1/2), the output by 2 delta * sum p |v|, twice (numerator and
        denominator).  The logit is a sum of D products q * (offset + code)
        with an offset of at most 1024, in fp32: off by at most
        4 sqrt(D) u sum |q| (1024 + code) s, u = 2^-24 (the probabilistic
        bound of a sum of D rounded terms with a factor 4), and q itself is
        held to 2^-24 of its row's largest.
      - the value sum, over the same offset, off by 4 sqrt(n) u (1024 + code).
      - weights relative to the largest p and s end in a grain of 2^-30.
    """
    B, H, D = q.shape
    pages, kvh, size = k[0].shape[:3]
    qf = oracle.to_f64(q, dtype)
    out, bound = np.zeros((B, H, D)), np.zeros((B, H, D))
    u = 2.0**-24
    for b in range(B):
        n = min(int(lens[b]), table.shape[1] * size)
        first = max(0, n - window) if window else 0
        at = [(int(table[b, t // size]), t % size) for t in range(first, n)]
        at = [(p, o) for p, o in at if 0 <= p < pages]
        if not at:
            continue
        pg, off = np.array(at).T
        for j in range(kvh):
            kt, vt = [tuple(a[pg, j, off] for a in t) for t in (k, v)]
            kv_, vv = values(*kt, dtype, G, bits), values(*vt, dtype, G, bits)
            ks, vs = [np.repeat(oracle.to_f64(t[1], dtype), G, -1) for t in (kt, vt)]
            kc, vc = codes(kt[0], bits), codes(vt[0], bits)
            for h in range(j * (H // kvh), (j + 1) * (H // kvh)):
                z = scale * (kv_ @ qf[b, h])
                p = np.exp(z - z.max())
                p /= p.sum()
                out[b, h] = p @ vv
                delta = abs(scale) * (4 * np.sqrt(D) * u * ((1024 + kc) * np.abs(ks)) @ np.abs(qf[b, h])
                                      + u * np.abs(qf[b, h]).max() * np.abs(kv_).sum(1)).max()
                bound[b, h] = (2.0**-11 * (p @ (np.abs(vs) * vc)) + 4 * min(delta, 1.0) * (p @ np.abs(vv))
                               + 4 * np.sqrt(len(at)) * u * (p @ (np.abs(vs) * (1024 + vc)))
                               + 2.0**-30 * np.abs(vs).max() * vc.sum(0))
    return out, bound
