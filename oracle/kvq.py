"""CPU oracle of the 4-bit latent cache: quantisation, the packed row and the
attention over it, written as definitions in float64 (test infrastructure;
shares no code with the CUDA path).

Quantisation takes the nearest number of an explicit list of candidates;
visibility is decided node by node and position by position.
"""
from __future__ import annotations

import numpy as np

ROW = 416
ERR_SLOT, ERR_NONFINITE = 0x4, 0x200


def e4m3_value(byte: int) -> float:
    """Magnitude of the low seven bits."""
    e, m = (byte >> 3) & 15, byte & 7
    return (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9


SCALES = np.array([e4m3_value(i) for i in range(127)])  # what a write may choose


def quantise_block(x, exponent: int):
    """(16 codes, scale byte) of 16 latents (float64 holding bf16 or fp32 values)."""
    x = np.asarray(x, np.float64)
    v = np.where(np.isnan(x), 0.0, x) * 2.0 ** -exponent
    a = np.abs(v).max()
    # nearest scale to a / 7: distances of 7 s from a, exact in float64; the even byte wins a tie
    with np.errstate(invalid="ignore"):
        d = np.abs(7.0 * SCALES - min(a, 7 * 448.0))
    best = np.flatnonzero(d == d.min())
    byte = int(best[0]) if len(best) == 1 or best[0] % 2 == 0 else int(best[1])
    s = SCALES[byte]
    codes = []
    for t in v:
        if s == 0:
            codes.append(8)
            continue
        t = max(min(t, 1e6), -1e6)
        q = np.arange(-7, 8)
        d = np.abs(q * s - t)
        best = q[d == d.min()]
        codes.append(8 + int(best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]))
    return codes, byte


def pack_row(kv_c, k_pe_bits, exponent: int = 0) -> np.ndarray:
    """The 416 bytes of one row; k_pe_bits: 64 bf16 bit patterns (uint16)."""
    row = np.zeros(ROW, np.uint8)
    words = [0] * 64
    for i in range(32):
        codes, row[256 + i] = quantise_block(kv_c[16 * i:16 * i + 16], exponent)
        for j, c in enumerate(codes):
            e = 16 * i + j
            t, odd = (e % 8) // 2, e % 2
            words[e // 8] |= c << (4 * t + 16 * odd)
    for w, v in enumerate(words):
        for k in range(4):
            row[4 * w + k] = (v >> (8 * k)) & 255
    row[288:] = np.ascontiguousarray(k_pe_bits, np.uint16).view(np.uint8)
    return row


def unpack_row(row, exponent: int = 0):
    """(512 latents, 64 rope values) float64 that a row stands for."""
    lat = np.zeros(512)
    for e in range(512):
        w = 4 * (e // 8)
        word = int(row[w]) | int(row[w + 1]) << 8 | int(row[w + 2]) << 16 | int(row[w + 3]) << 24
        code = word >> (4 * ((e % 8) // 2) + 16 * (e % 2)) & 15
        lat[e] = (code - 8) * e4m3_value(int(row[256 + e // 16])) * 2.0 ** exponent
    bits = np.ascontiguousarray(row[288:]).view(np.uint16).astype(np.uint32) << 16
    return lat, bits.view(np.float32).astype(np.float64)


def unpack_rows(rows, exponent: int = 0):
    """unpack_row of many rows at once."""
    rows = np.asarray(rows)
    word = np.ascontiguousarray(rows[:, :256]).view("<u4").astype(np.int64)
    lat = np.stack([(word >> (4 * (e // 2) + 16 * (e % 2)) & 15) - 8 for e in range(8)], -1).reshape(len(rows), 512)
    scale = np.array([e4m3_value(i) for i in range(128)])[rows[:, 256:288] & 127]
    bits = np.ascontiguousarray(rows[:, 288:]).view("<u2").astype(np.uint32) << 16
    return (lat * np.repeat(scale, 16, 1) * 2.0 ** exponent, bits.view(np.float32).astype(np.float64))


def node_chain(parent, i):
    """Node i and its ancestors, deepest first."""
    up = [i]
    while parent[up[-1]] >= 0:
        up.append(int(parent[up[-1]]))
    return up


def visible(parent, i: int, P: int, window: int = 0, sinks: int = 0):
    """Logical positions that node i sees, in order."""
    chain = node_chain(parent, i)
    depth = {t: len(node_chain(parent, t)) - 1 for t in chain}
    here = P + depth[i]

    def keep(place):
        return window == 0 or place < sinks or here - place < window

    seen = [j for j in range(P) if keep(j)]
    return seen + sorted(P + t for t in chain if keep(P + depth[t]))


def attention(lat, rope, q_lat, q_pe, scale, parent, P, H, window=0, sinks=0):
    """out [Q, H, 512], lse [Q, H] of one sequence, and what bounds their
    rounding: sum of weights times |latents| [Q, H, 512], and the largest sum
    of magnitudes behind a score [Q, H].  lat [N][512], rope [N][64] in logical
    order, float64."""
    Q = len(parent)
    out, lse = np.zeros((Q, H, 512)), np.zeros((Q, H))
    mag, smag = np.zeros((Q, H, 512)), np.zeros((Q, H))
    for i in range(Q):
        pos = visible(parent, i, P, window, sinks)
        s = scale * (q_lat[i] @ lat[pos].T + q_pe[i] @ rope[pos].T)
        m = s.max(1, keepdims=True)
        w = np.exp(s - m)
        z = w.sum(1, keepdims=True)
        out[i], lse[i] = (w / z) @ lat[pos], (m + np.log(z))[:, 0]
        mag[i] = (w / z) @ np.abs(lat[pos])
        smag[i] = scale * (np.abs(q_lat[i]) @ np.abs(lat[pos]).T + np.abs(q_pe[i]) @ np.abs(rope[pos]).T).max(1)
    return out, lse, mag, smag
