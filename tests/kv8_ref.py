"""The 8-bit paged KV cache's operators in 64 bits, written from their definitions (NumPy, loops over
sequences and pages), and the error bounds that their kernels are held to."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _values():
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if b & 128 else x)
    return np.array(v)


E4M3 = _values()
_POS = E4M3[:127]  # 0 .. 448


def encode(x):
    """float64 -> E4M3 codes: nearest, ties to the even code, saturating; NaN -> 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    hi = np.searchsorted(_POS, a, side="left").clip(max=126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = np.abs(_POS[hi] - a), np.abs(a - _POS[lo])
    with np.errstate(invalid="ignore"):
        up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (a >= 448.0)
    code = np.where(up, hi, lo).astype(np.uint8)
    code = np.where(a >= 448.0, np.uint8(126), code)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), code).astype(np.uint8)


def need_scale(amax):
    """Least 2^e with amax <= 448 * 2^e, e clamped to [-100, 120]."""
    if not amax > 0:
        return 2.0 ** -100
    for e in range(-100, 121):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 120


def rows_of(n_rows, S, cu):
    return [(s * (n_rows // S), n_rows // S) if cu is None else (cu[s], cu[s + 1] - cu[s]) for s in range(S)]


def append(k, k_scale, x, table, kv_len, shares, page):
    """In place on codes uint8 [P][H][page][D] and scales; x float64 [T][H][D]."""
    for s, (r0, n) in enumerate(shares):
        L = int(kv_len[s])
        for h in range(k.shape[1]):
            pos = max(0, L - n)
            while pos < L:
                a, p = pos % page, int(table[s][pos // page])
                m = min(page - a, L - pos)
                new = x[r0 + pos - (L - n):r0 + pos - (L - n) + m, h]
                fin = np.abs(new[~np.isnan(new)])
                need = need_scale(fin.max() if fin.size else 0.0)
                old = float(k_scale[p, h])
                sc = max(old, need) if a > 0 else need
                if a > 0 and sc > old:
                    k[p, h, :a] = encode(E4M3[k[p, h, :a]] * (old / sc))
                k[p, h, a:a + m] = encode(new / sc)
                k_scale[p, h] = sc
                pos += m


def gather(k, k_scale, table_row, lo, hi, page):
    """float64 [hi - lo][H][D] of tokens lo .. hi - 1."""
    j = np.arange(lo, hi)
    p = np.asarray(table_row)[j // page]
    return E4M3[k[p, :, j % page]] * k_scale[p][:, :, None].astype(np.float64)


def attention(q, cache, table, kv_len, shares, page, causal, window, scale):
    """out, lse in float64, and what the bounds need: A = sum p |v| per channel, the largest sum of |products|
    of a visible logit, and the largest |logit|.  q float64 [T][H][D]; cache (k, v, k_scale, v_scale)."""
    k, v, ks, vs = cache
    T, H, D = q.shape
    G = H // k.shape[1]
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    A, B, Z = np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H))
    for s, (r0, n) in enumerate(shares):
        L = int(kv_len[s])
        if L == 0:
            continue
        for i in range(n):
            pos = L - n + i
            hi = min(L, pos + 1) if causal else L
            lo = max(0, pos - window + 1) if window > 0 else 0
            if hi <= lo:
                continue
            K, V = gather(k, ks, table[s], lo, hi, page), gather(v, vs, table[s], lo, hi, page)
            for h in range(H):
                z = scale * (K[:, h // G] @ q[r0 + i, h])
                m = z.max()
                e = np.exp(z - m)
                w = e / e.sum()
                out[r0 + i, h] = w @ V[:, h // G]
                lse[r0 + i, h] = m + math.log(e.sum())
                A[r0 + i, h] = w @ np.abs(V[:, h // G])
                big = np.abs(q[r0 + i, h]).max()
                B[r0 + i, h] = scale * (np.abs(K[:, h // G]) @ np.abs(q[r0 + i, h])).max()
                # the query's own rounding (2^-25 of the row's largest value, in each channel)
                B[r0 + i, h] += scale * big * np.abs(K[:, h // G]).sum(axis=1).max() / 2 / (D + 8)
                Z[r0 + i, h] = np.abs(z).max()
    return out, lse, A, B, Z


def attention_bounds(out, lse, A, B, Z, D, tokens, dtype):
    """How far the kernel's outputs may be off.

    A logit: D + 8 fp32 roundings of terms that sum to at most B, and a few of the logit itself in the exponent
    (2^-22 of it and of the block scale's logarithm, at most 128).  A weight: its logit's error, 2^-11 as the fp16
    operand, 2^-21 for the exponential.  The sums: one fp32 rounding (of up to a whole step, 2^-23) a token.  The
    output: half a step of its type."""
    logit = (D + 8) * 2.0 ** -24 * B + 2.0 ** -22 * (Z * 1.5 + 128)
    weight = np.expm1(logit) + 2.0 ** -21
    both = 2 * weight + 2.0 ** -11 + tokens * 2.0 ** -23
    finite = np.where(np.isfinite(lse), lse, 0.0)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return (both[..., None] * A + HALF_STEP[dtype] * (np.abs(out) + both[..., None] * A) + tiny,
            logit + 2.0 ** -21 + tokens * 2.0 ** -23 + 2.0 ** -22 * np.abs(finite))
