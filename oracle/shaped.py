"""Reference of the rules on logits, of MXFP4 and of the statistics of shaped rows, in fp64
NumPy from the definitions (test infrastructure only)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_codes(x: np.ndarray):
    """(codes 0..15 [R, K], scale bytes [R, K/32]) of x [R, K]: OCP MXFP4, ties to the even
    code; a block with a NaN or an infinity has scale 0xFF and codes 0."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    _, ex = np.frexp(top)                                   # top = f * 2^ex, f in [0.5, 1)
    e = np.where(top > 0, np.maximum(ex - 1 - 2, -127), -127).astype(np.int64)
    a = np.abs(b) / np.exp2(e.astype(np.float64))[..., None]
    dist = np.abs(a[..., None] - E2M1)
    near = dist == dist.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1) & (near.sum(-1) > 1), even.argmax(-1), near.argmax(-1))
    code = code + 8 * np.signbit(b)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(R, K).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    R, K = codes.shape
    return (v.reshape(R, K // 32, 32) * s[..., None]).reshape(R, K)


def unpack_bits(words: np.ndarray, V: int) -> np.ndarray:
    """bool [rows, V] of int32 / uint32 bitmap rows."""
    w = np.ascontiguousarray(words).view(np.uint32).astype(np.uint64)
    v = np.arange(V)
    return ((w[:, v // 32] >> (v % 32).astype(np.uint64)) & np.uint64(1)).astype(bool)


def pack_bits(bits: np.ndarray) -> np.ndarray:
    rows, V = bits.shape
    words = (V + 31) // 32
    full = np.zeros((rows, words * 32), dtype=np.uint64)
    full[:, :V] = bits
    w = (full.reshape(rows, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def shape_logits(z, seq, pos, V, bias=None, counts=None, repetition=None, presence=None,
                 frequency=None, allow=None, allow_id=None):
    """Rules on logits z [n, V] (fp64) of rows of sequences seq [n] at flat positions pos [n]."""
    z = z.copy()
    if counts is not None:
        c = counts[seq].astype(np.float64)
        th = (np.ones(counts.shape[0]) if repetition is None else repetition.astype(np.float64))[seq][:, None]
        pr = (np.zeros(counts.shape[0]) if presence is None else presence.astype(np.float64))[seq][:, None]
        fr = (np.zeros(counts.shape[0]) if frequency is None else frequency.astype(np.float64))[seq][:, None]
        cut = np.where(z > 0, z / th, z * th) - pr - fr * c
        z = np.where(c > 0, cut, z)
    if bias is not None:
        z = z + (bias.astype(np.float64)[seq] if bias.ndim == 2 else bias.astype(np.float64))
    if allow is not None:
        ids = allow_id.reshape(-1)[pos] if allow_id is not None else \
            (np.zeros_like(seq) if allow.shape[0] == 1 else seq)
        ok = unpack_bits(allow, V)[np.maximum(ids, 0)] | (ids < 0)[:, None]
        z = np.where(ok, z, -np.inf)
    return z


def row_stats(z):
    """tok, lse, conf, entropy, margin of logits [n, V]."""
    n, V = z.shape
    m = z.max(-1) if n else np.zeros(0)
    empty = np.isneginf(m)
    x = np.where(np.isneginf(z), -np.inf, z - np.where(empty, 0.0, m)[:, None])
    p = np.exp(x)
    s = np.where(empty, 1.0, p.sum(-1))
    t = np.where(p > 0, p * np.where(np.isfinite(x), x, 0.0), 0.0).sum(-1)
    tok = np.where(empty, -1, z.argmax(-1) if n else 0)
    second = np.partition(z, V - 2, axis=-1)[:, V - 2] if V > 1 else np.full(n, -np.inf)
    with np.errstate(invalid="ignore"):
        drop = np.where(np.isneginf(second), 0.0, np.exp(second - m))
    return dict(tok=tok.astype(np.int64), lse=np.where(empty, -np.inf, m + np.log(s)),
                conf=np.where(empty, 0.0, 1 / s), entropy=np.where(empty, np.inf, np.log(s) - t / s),
                margin=np.where(empty, 0.0, (1 - drop) / s))
