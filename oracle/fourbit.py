"""float64 oracle of the 4-bit layers and the 4-bit key/value cache (NumPy), from the definitions in
include/ifq.h; every entry is placed and found by its address formula, one entry at a time."""
import numpy as np

BF16_MAX = np.float32(3.3895313892515355e38)


def bf16_bits(x):
    """Nearest-even bf16 bit patterns (uint16) of finite float32 values."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def _half_even(num, den, rest=0):
    """rint((num + rest) / den) half-even for den > 0 (0 where den == 0), from extended-precision quotients;
    rest: what num's rounding left out, which decides where num / den is a half."""
    num, den = np.longdouble(num), np.longdouble(den)
    q = num / np.where(den > 0, den, 1)
    half = (q - np.floor(q) == 0.5) & (np.longdouble(rest) != 0)
    n = np.where(half, np.floor(q) + (np.longdouble(rest) > 0), np.rint(q))
    return np.where(den > 0, n, 0)


# ------------------------------------------------------------------ 4-bit layers
def w4_quantize(R, group):
    """R float32 [rows][cols] -> (q int8 [rows][cols], scale bf16 bits [rows][cols/group])."""
    rows, cols = R.shape
    w = np.where(np.isfinite(R), R, np.float32(0)).reshape(rows, cols // group, group)
    with np.errstate(under="ignore"):
        s = bf16_bits(np.abs(w).max(axis=2) * (np.float32(1) / np.float32(7)))
    q = np.clip(_half_even(w, bf16_value(s).astype(np.float64)[..., None]), -7, 7)
    return q.astype(np.int8).reshape(rows, cols), s


def w4_code_place(r, k, cols):
    """Byte offset and bit of entry (r, k) in the codes."""
    word = 2 * ((k % 64) // 32) + (r % 16) // 8
    at = ((r // 16) * (cols // 64) + k // 64) * 512 + (4 * (r % 8) + (k % 32) // 8) * 16 + 4 * word
    bit = 4 * ((k % 8) // 2) + 16 * (k % 2)
    return at + bit // 8, bit % 8


def w4_scale_place(r, j, groups):
    return ((r // 16) * groups + j) * 16 + 2 * (r % 8) + (r % 16) // 8


def w4_pack(q, s):
    """(q, scale bits) -> codes uint8 [rt][cols/64][512], scales uint16 [rt][groups][16]."""
    rows, cols = q.shape
    groups, rt = s.shape[1], (rows + 15) // 16
    codes = np.zeros(rt * cols * 8, dtype=np.uint8)
    full = np.zeros((rt * 16, cols), dtype=np.int64)
    full[:rows] = q
    r, k = np.meshgrid(np.arange(rt * 16), np.arange(cols), indexing="ij")
    at, bit = w4_code_place(r, k, cols)
    np.add.at(codes, at.ravel(), ((full + 8) << bit).ravel().astype(np.uint8))
    scales = np.zeros(rt * groups * 16, dtype=np.uint16)
    r, j = np.meshgrid(np.arange(rows), np.arange(groups), indexing="ij")
    scales[w4_scale_place(r, j, groups)] = s
    return codes.reshape(rt, cols // 64, 512), scales.reshape(rt, groups, 16)


def w4_values(q, s, group):
    """float64 s q."""
    return q.astype(np.float64) * np.repeat(bf16_value(s).astype(np.float64), group, axis=1)


# ------------------------------------------------------------------ 4-bit cache
def kv4_quantize(x):
    """x float32 [..., dim] (one plane each) -> (n uint8, s bits, m bits)."""
    x = np.clip(np.where(np.isfinite(x), x, np.float32(0)), -BF16_MAX, BF16_MAX)
    lo, hi = x.min(axis=-1), x.max(axis=-1)
    m = bf16_bits(lo)
    with np.errstate(under="ignore"):
        s = bf16_bits(hi * (np.float32(1) / np.float32(15)) - lo * (np.float32(1) / np.float32(15)))
    a, b = np.longdouble(x), -np.longdouble(bf16_value(m)[..., None])
    num = a + b
    rest = (a - (num - (num - a))) + (b - (num - a))   # a + b = num + rest exactly
    n = np.clip(_half_even(num, bf16_value(s).astype(np.float64)[..., None], rest), 0, 15)
    return n.astype(np.uint8), s, m


def kv4_values(n, s, m):
    """float64 s n + m."""
    return bf16_value(s).astype(np.float64)[..., None] * n + bf16_value(m).astype(np.float64)[..., None]


def kv4_key_place(r, d):
    word = 2 * ((d % 64) // 32) + r // 8
    bit = 4 * ((d % 8) // 2) + 16 * (d % 2)
    return (d // 64) * 512 + (4 * (r % 8) + (d % 32) // 8) * 16 + 4 * word + bit // 8, bit % 8


def kv4_value_place(r, d, D):
    word = 2 * ((d % 64) // 32) + r // 8
    bit = 4 * (d % 4) + 16 * (r % 2)
    return 8 * D + (d // 64) * 512 + (4 * ((d % 32) // 4) + (r % 8) // 2) * 16 + 4 * word + bit // 8, bit % 8


def kv4_put(record, r, key, value):
    """Writes token r (0..15) of a record (uint8 [32 dim + 256]) in place; key, value: (n [2][dim], s [2], m [2])."""
    dim = key[0].shape[1]
    D = 2 * dim
    d = np.arange(D)
    for (n, s, m), place, par in ((key, kv4_key_place(r, d), 16 * D), (value, kv4_value_place(r, d, D), 16 * D + 128)):
        for at, bit, code in zip(place[0], place[1], n.reshape(-1)):
            record[at] = (record[at] & ~(15 << bit) & 255) | (int(code) << int(bit))
        record[par + 8 * r:par + 8 * r + 8] = np.array([s[0], m[0], s[1], m[1]], dtype=np.uint16).view(np.uint8)


def kv4_get(records, dim):
    """Records uint8 [T][32 dim + 256] -> per token (codes, s, m) of keys and values: n [16 T][2][dim], bits [16 T][2]."""
    T, D = records.shape[0], 2 * dim
    r, d = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    out = []
    for (at, bit), par in ((kv4_key_place(r, d), 16 * D), (kv4_value_place(r, d, D), 16 * D + 128)):
        n = (records[:, at] >> bit) & 15
        p = np.ascontiguousarray(records[:, par:par + 128]).view(np.uint16).reshape(T * 16, 2, 2)
        out.append((n.reshape(T * 16, 2, dim).astype(np.uint8), p[..., 0].copy(), p[..., 1].copy()))
    return out


def kv4_attention(q, k, v, first, scale):
    """q float64 [rows][D]; k, v: (n, s, m) of a head's tokens; row i sees keys 0 .. first + i.  Returns (o, bound):
    bound is the first-order error of o from a two-term fp16 split of q, weights held as one fp16 term and
    float32 sums, without o's own rounding."""
    rows, D = q.shape
    T = k[0].shape[0]
    if T == 0:
        return np.zeros((rows, D)), np.zeros((rows, D))

    def parts(x):
        n, s, m = x
        sv, mv = bf16_value(s).astype(np.float64)[..., None], bf16_value(m).astype(np.float64)[..., None]
        val = sv * n + mv
        return val.reshape(T, D), (np.abs(sv * n) + np.abs(mv)).reshape(T, D)

    kv, ka = parts(k)
    vv, va = parts(v)
    s = scale * (q @ kv.T)
    # |q - (two fp16 terms)| <= 2^-22 |q| or, where the second term is subnormal, 2^-36 of the row's largest (the
    # entries are scaled to below 2^11 or 2^15, subnormal steps are 2^-24); D products and the parameters'
    # terms are added in float32
    ds = abs(scale) * ((np.abs(q) @ ka.T) * (2.0 ** -21 + (D / 16 + 8) * 2.0 ** -22) +
                       2.0 ** -34 * np.abs(q).max(axis=1, keepdims=True) * ka.sum(axis=1)) + 2.0 ** -22 * np.abs(s)
    seen = np.arange(T)[None, :] <= first + np.arange(rows)[:, None]
    o, bound = np.zeros((rows, D)), np.zeros((rows, D))
    for i in range(rows):
        if not seen[i].any():
            continue
        si, di = s[i, seen[i]], ds[i, seen[i]]
        p = np.exp(si - si.max())
        p /= p.sum()
        o[i] = p @ vv[seen[i]]
        # a score off by d moves a weight by the factor exp(2 d) at most (its own and the sum's); the weights'
        # rounding to fp16 2^-11, or 2^-25 of 2^9 / cap where subnormal, the cap at most 8 times the largest scale;
        # float32 sums over the keys, exp2 and the joins of partial results
        rel = np.expm1(2 * di.max()) + 2.0 ** -11 + (len(si) / 16 + 64) * 2.0 ** -22
        flush = 2.0 ** -31 * 15 * len(si) * bf16_value(v[1][:len(si)]).max() / np.exp(si - si.max()).sum()
        bound[i] = rel * (p @ va[seen[i]]) + flush
    return o, bound
