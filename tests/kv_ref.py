"""The cache operators and the attention over the cache in float64, from
their definitions: position by position, on the CPU, no code of the library.
NumPy only; e4m3 codes are uint8 and bfloat16 bits uint16."""
import numpy as np

E_MIN, E_MAX = -100, 119


def e4m3_table():
    """Value of each of the 256 codes."""
    c = np.arange(256)
    m, e = c & 7, (c >> 3) & 15
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c >= 128, -v, v)


E4M3 = e4m3_table()


def exponent(most):
    """Least e in [E_MIN, E_MAX] with most <= 448 * 2^e."""
    for e in range(E_MIN, E_MAX + 1):
        if most <= 448 * 2.0 ** e:
            return e
    return E_MAX


def quantise(row):
    """A float64 row -> (e4m3 codes, exponent): one rounding, ties to the even code."""
    fin = np.abs(row[np.isfinite(row)])
    e = exponent(fin.max() if fin.size else 0.0)
    pos = E4M3[:127]  # codes 0 .. 126: 0 .. 448
    codes = np.empty(row.shape, np.uint8)
    for i, x in enumerate(row):
        if not np.isfinite(x):
            codes[i] = 0x7F
            continue
        y = min(abs(x) * 2.0 ** -e, 448.0)
        k = int(np.searchsorted(pos, y))  # pos[k - 1] < y <= pos[k]
        if k and (y - pos[k - 1] < pos[k] - y or (y - pos[k - 1] == pos[k] - y and (k - 1) % 2 == 0)):
            k -= 1
        codes[i] = k | (0x80 if np.signbit(x) else 0)
    return codes, e


def bf16_bits(x):
    """float32 -> bfloat16 bits, to nearest even."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def cache_value(pages, exps):
    """Pages (codes uint8 with exponents, or bfloat16 bits) -> float64."""
    if exps is None:
        return bf16_value(pages)
    return E4M3[pages] * 2.0 ** exps.astype(np.float64)[..., None]


def tokens_of(value, table, ptable, prefix, page_size, b, n):
    """Positions 0 .. n - 1 of sequence b: [n, Hkv, D]."""
    out = np.empty((n,) + (value.shape[1], value.shape[3]))
    for p in range(n):
        t = p if p < prefix else p - prefix
        ids = ptable if p < prefix else table[b]
        out[p] = value[ids[t // page_size], :, t % page_size]
    return out


def attend(q, kval, vval, table, kv_len, ptable, prefix, gammas, page_size, scale):
    """Per query of B, N, Hq: out [.., D] and lse in float64, and what bounds a
    single-precision evaluation's error: weight [.., D] = sum_j w_j |v_jd|,
    size = max_j scale * sum_d |q_d k_jd|."""
    B, N, Hq, D = q.shape
    G = Hq // kval.shape[1]
    out, lse = np.zeros(q.shape), np.full((B, N, Hq), -np.inf)
    weight, size = np.zeros(q.shape), np.zeros((B, N, Hq))
    for b in range(B):
        held = int(kv_len[b]) + int(gammas[b]) + 1
        k = tokens_of(kval, table, ptable, prefix, page_size, b, held)
        v = tokens_of(vval, table, ptable, prefix, page_size, b, held)
        for i in range(int(gammas[b]) + 1):
            sees = int(kv_len[b]) + i + 1
            for h in range(Hq):
                with np.errstate(invalid="ignore", over="ignore"):
                    kk, vv = k[:sees, h // G], v[:sees, h // G]
                    z = scale * (kk @ q[b, i, h])
                    m = z.max()
                    e = np.exp(z - m)
                    s = e.sum()
                    out[b, i, h] = (e / s) @ vv
                    lse[b, i, h] = m + np.log(s)
                    weight[b, i, h] = (e / s) @ np.abs(vv)
                    size[b, i, h] = scale * (np.abs(kk) @ np.abs(q[b, i, h])).max()
    return out, lse, weight, size
