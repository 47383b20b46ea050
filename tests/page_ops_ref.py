"""Plain 64-bit forms of the block-scaled FP8 cache, of the pages' bounds, of the
selection and of attention over a set of tokens, from the definitions in
include/nvfp4kv.h, and the readers of both caches' records."""
import numpy as np
import torch

from layout import nvfp4_planes

E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
_MAG = E4M3[:127]                                    # 0 .. 448, ascending by code
_MID = (_MAG[1:] + _MAG[:-1]) / 2
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_codes(x):
    """Nearest codes, ties to the even one, saturating."""
    a = np.abs(x)
    lo = np.searchsorted(_MID, a, "left")            # (a midpoint: the code under it)
    hi = np.searchsorted(_MID, a, "right")
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def scale_exp(amax):
    if not amax > 0:
        return -100
    f, x = np.frexp(np.float64(amax))                # amax = f 2^x, f in [0.5, 1): 448 = 0.875 * 2^9
    return int(np.clip(x - 9 if f <= 0.875 else x - 8, -100, 100))


class BlockRef:
    """Codes and exponents [2 (K, V)][pages][kv heads]..., filled as fp8bkv_append does."""

    def __init__(self, pages, hkv):
        self.code = np.zeros((2, pages, hkv, 16, 128), np.uint8)
        self.exp = np.full((2, pages, hkv), -100)

    def append(self, rows, table, length):
        """rows: (k, v) [C][hkv][128] in 64 bits, the last C of `length` tokens."""
        C = len(rows[0])
        pos = length - C
        while pos < length:
            page, first = pos // 16, pos % 16
            n = min(16 - first, length - pos)
            p = table[page]
            for i in range(2):
                x = rows[i][pos - (length - C):][:n]
                for h in range(x.shape[1]):
                    e = scale_exp(np.abs(x[:, h]).max())
                    if first:
                        old = int(self.exp[i, p, h])
                        if e > old:
                            c = self.code[i, p, h, :first]
                            self.code[i, p, h, :first] = e4m3_codes(E4M3[c] * 2.0 ** (old - e))
                        e = max(e, old)
                    self.exp[i, p, h] = e
                    self.code[i, p, h, first:first + n] = e4m3_codes(x[:, h] / 2.0 ** e)
            pos += n

    def values(self, i, table, length):
        """[length][hkv][128]"""
        p = np.asarray(table[:-(-length // 16)], int)
        v = E4M3[self.code[i, p]] * (2.0 ** self.exp[i, p].astype(float))[..., None, None]
        return v.transpose(0, 2, 1, 3).reshape(-1, v.shape[1], 128)[:length]


def block_planes(pool):
    """Codes [2][pages][hkv][16][128] and scales [2][pages][hkv] of block-scaled records."""
    n, h, _ = pool.shape
    t, c = np.meshgrid(np.arange(16), np.arange(128), indexing="ij")
    f = (t // 2) % 2 + 4 * ((t // 4) % 2)
    k = t * 128 + ((c // 16 + t % 2) % 8) * 16 + c % 16
    v = 2048 + (t // 2) * 256 + ((c // 8 + f) % 16) * 16 + 2 * (c % 8) + t % 2
    codes = np.stack([pool[:, :, k.ravel()], pool[:, :, v.ravel()]]).reshape(2, n, h, 16, 128)
    return codes, pool[:, :, 4096:4104].copy().view(np.float32).transpose(2, 0, 1)


def block_pool(ref, fill=0):
    """Records that hold what a BlockRef does."""
    n, h = ref.code.shape[1:3]
    pool = np.full((n, h, 4128), fill, np.uint8)
    t, c = np.meshgrid(np.arange(16), np.arange(128), indexing="ij")
    f = (t // 2) % 2 + 4 * ((t // 4) % 2)
    pool[:, :, (t * 128 + ((c // 16 + t % 2) % 8) * 16 + c % 16).ravel()] = ref.code[0].reshape(n, h, -1)
    pool[:, :, (2048 + (t // 2) * 256 + ((c // 8 + f) % 16) * 16 + 2 * (c % 8) + t % 2).ravel()] = \
        ref.code[1].reshape(n, h, -1)
    s = np.ascontiguousarray((2.0 ** ref.exp.astype(float)).astype(np.float32).transpose(1, 2, 0))
    pool[:, :, 4096:4104] = s.view(np.uint8)
    return pool


def nvfp4_values(pool):
    """K and V [pages][hkv][16][128] in 64 bits of NVFP4 records (before the tensor scale)."""
    kd, ks, vd, vs = nvfp4_planes(pool)
    out = []
    for d, s in ((kd, ks), (vd, vs)):
        code = np.stack([d & 15, d >> 4], -1).reshape(*d.shape[:-1], 128)
        out.append(E2M1[code] * np.repeat(E4M3[s], 16, -1))
    return out


def bounds(k):
    """(lo, hi int8 [128], step) of the keys [tokens][128] of a page."""
    k = k.astype(np.float32)
    u = np.abs(k).max()
    if u == 0:
        return np.zeros(128, np.int8), np.zeros(128, np.int8), np.float32(0)
    r = np.float32(127) / u
    hi = np.minimum(np.ceil(k.max(0) * r), 127)
    lo = np.maximum(np.floor(k.min(0) * r), -127)
    return lo.astype(np.int8), hi.astype(np.int8), u / np.float32(127)


def select(q, ints, steps, n, budget, first, last):
    """The list of one query token and kv head: q [group][128] fp32, ints [P][2][128], steps [P]."""
    P = -(-n // 16) if n > 0 else 0
    if P <= budget:
        return list(range(P)) + [-1] * (budget - P)
    q = q.astype(np.float32)
    top = np.abs(q).max()
    w = np.rint(q * (np.float32(127) / top)).astype(np.int64) if top > 0 else np.zeros(q.shape, np.int64)
    i = ints[:P].astype(np.int64)
    best = np.maximum(w[:, None] * i[None, :, 0], w[:, None] * i[None, :, 1]).sum(-1).max(0)
    score = (best.astype(np.float32) * steps[:P]).astype(np.float64)
    score[:first] = np.inf
    score[P - last:] = np.inf
    return sorted(np.lexsort((np.arange(P), -score))[:budget].tolist())


def attend(q, k, v, sm_scale, out_eps, q_eps=0.0):
    """Attention of q [rows][128] over k, v [tokens][128] in 64 bits, and how far the
    kernels may be off it.  Their roundings: scores in fp32 (eight matrix
    instructions of exact products, each sum off by 2^-22 of its terms' magnitudes
    at most: 2^-18 of sum |q k|), with q_eps also q itself to fp16 (q_eps of each
    element, 2^-25 in log2 units where it is subnormal); a score off by d puts its
    weight and the sum of weights off by e^d - 1 each; weights to fp16 (2^-11; 2^-25
    below 2^-14, the largest being at least 1); sums of up to 256 terms a lane in
    fp32, above and below the line (2^-15); the output's own type."""
    if len(k) == 0:
        return np.zeros((len(q), 128)), np.full((len(q), 128), 1e-300)
    s = sm_scale * (q @ k.T)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    o = w @ v
    d = (2.0 ** -18 + q_eps) * sm_scale * (np.abs(q) @ np.abs(k).T).max(-1)
    if q_eps:
        d = d + 2.0 ** -25 * np.log(2) * np.abs(k).sum(-1).max()
    rel = 2 * np.expm1(d) + 2.0 ** -11 + 2.0 ** -15
    bound = rel[:, None] * (w @ np.abs(v)) + 2.0 ** -25 * np.abs(v).sum(0) + out_eps * np.abs(o)
    return o, bound * (1 + 2.0 ** -8) + 1e-300


def check(got, want, bound, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - want) / bound
    assert (off <= 1).all(), f"{what}: {off.max():.3g} times the bound at {np.unravel_index(off.argmax(), off.shape)}"
