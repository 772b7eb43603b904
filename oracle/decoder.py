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

    `bound` is a wide one, for any kernel that multiplies integer codes, a
    constant of up to 1024 added to them, by 16-bit rounded weights and sums
    in fp32 (attention_bound is the one of the kernel's own roundings):
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


LAMBDA = 6.0  # see attention_bound


def attention_bound(q, k, v, dtype: str, G: int, bits: int, table, lens, scale: float, window: int = 0, leave_out=()):
    """As paged_attention, with a bound from the kernel's own roundings.

    `leave_out`: positions counted from a sequence's first (0, 1, ...) or last
    (-1, -2, ...) seen token that are left out of the sums, a mistake planted
    for tests of what the bound can tell.

    With u = 2^-24 (half a step of fp32; 2 u where the matrix cores may cut
    instead of rounding), code, s and b a row's codes, scales and biases, per
    token t, group g, head and column:
      logit   z = c (sum_g s C_g + b Q_g), C_g = sum code q, Q_g = sum q over
              the group.  C_g: G sums of at most S = sum code |q|, 2 u each.
              Q_g: G sums, in four lanes, of at most a lane's part of sum |q|, u
              each, 2 u for adding the lanes', u for the pieces it is cut into,
              and 2^-32 of the row's largest |q|; the same error for every token.  sum b Q_g: 3 D/G sums, 2 u.  The sum over the
              groups: D/G roundings.  q itself is held to 2^-33 of the row's
              largest.  c: three roundings, the same for every token.
      weight  p = 2^(z - ref): u of the argument's size (the distance from the
              largest logit, and 64), 2 u for the power.
      sums    each weight p s rounded to 11 bits, 2^-11 relative, or 2^-28 of
              the group's largest p s; products with code summed, 2 u for
              each 8 tokens; sum p b and sum p a rounding a token and lane.
    An error d of a token's logit moves the output by p d (v - out).  Errors
    of one number that all tokens share are taken in full.  The many
    independent ones are added as LAMBDA times the root of their squares'
    sum: of independent errors of mean zero within +- c_i, a sum passes
    LAMBDA sqrt(sum c_i^2) with probability below 2 exp(-LAMBDA^2 / 2) =
    3e-8, and far less where they fill their ranges evenly (a variance of
    c_i^2 / 3).  The 11-bit roundings take the plain sum where that is less.
    """
    B, H, D = q.shape
    pages, kvh, size = k[0].shape[:3]
    NG, u, lam = D // G, 2.0**-24, LAMBDA
    qf = oracle.to_f64(q, dtype)
    out, bound = np.zeros((B, H, D)), np.zeros((B, H, D))
    root = lambda x: np.sqrt((x * x).sum(0))
    for b in range(B):
        n = min(int(lens[b]), table.shape[1] * size)
        first = max(0, n - window) if window else 0
        skip = {first + i if i >= 0 else n + i for i in leave_out}
        at = [(int(table[b, t // size]), t % size) for t in range(first, n) if t not in skip]
        at = [(p, o) for p, o in at if 0 <= p < pages]
        if not at:
            continue
        pg, off = np.array(at).T
        n = len(at)
        for j in range(kvh):
            kt, vt = [tuple(a[pg, j, off] for a in t) for t in (k, v)]
            kd, vd = values(*kt, dtype, G, bits), values(*vt, dtype, G, bits)
            kc, vc = codes(kt[0], bits).astype(np.float64), codes(vt[0], bits).astype(np.float64)
            ks, kb, vs, vb = [oracle.to_f64(x, dtype) for x in (kt[1], kt[2], vt[1], vt[2])]  # [n, NG]
            va, vb = np.repeat(np.abs(vs), G, 1) * vc, np.repeat(np.abs(vb), G, 1)
            for h in range(j * (H // kvh), (j + 1) * (H // kvh)):
                qg, c = qf[b, h].reshape(NG, G), abs(scale)
                z = scale * (kd @ qf[b, h])
                p = np.exp(z - z.max())
                p /= p.sum()
                out[b, h] = o = p @ vd
                # logits
                most = np.abs(qg).max()
                C, S = [np.einsum("tgi,gi->tg", kc.reshape(n, NG, G), x) for x in (qg, np.abs(qg))]
                Q = np.abs(qg.sum(1))
                terms = (np.abs(kb) * Q).sum(1)
                own = c * np.sqrt(((np.sqrt(G) * 2 * u * np.abs(ks) * S)**2).sum(1) + 3 * NG * (2 * u * terms)**2
                                  + NG * (u * (terms + (np.abs(ks * C)).sum(1)))**2)
                own = own + np.log(2) * u * ((z.max() - z) / np.log(2) + 64) + 2 * u
                own = lam * own + c * 2.0**-33 * most * (np.repeat(np.abs(ks), G, 1) * kc).sum(1)
                e_q = (lam * np.sqrt(G) / 4 + 3) * u * np.abs(qg).sum(1) + 2.0**-32 * most
                far = vd - o
                err = root((p * own)[:, None] * np.abs(far))
                err += c * e_q @ np.abs((p[:, None] * kb).T @ far) + 3 * u * np.abs((p * z) @ far)
                err *= np.exp(min(own.max(), 1.0))
                # sums
                w = p[:, None] * va
                err += 2.0**-11 * (1 + 2.0**-10) * np.minimum(w.sum(0), lam * root(w))
                err += 2.0**-28 * np.repeat((p[:, None] * np.abs(vs)).max(0), G) * np.minimum(vc.sum(0), lam * root(vc))
                steps = n / 8 + 32
                err += lam * np.sqrt(steps) * 2 * u * w.sum(0)
                err += lam * np.sqrt(2 * steps) * u * (p @ vb + np.abs(o)) + 32 * u * (w.sum(0) + p @ vb)
                bound[b, h] = err
    return out, bound
