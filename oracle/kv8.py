"""CPU oracle of the paged 8-bit latent cache and of a step's page tables, written as
definitions in float64 and plain Python (test infrastructure; shares no code with the
CUDA path).

Quantisation takes the nearest number of an explicit list of candidates; a block's
scale is found by trying them; the tables are built request by request.  Which
positions a node sees and the attention itself are those of the 4-bit cache's oracle.
"""
from __future__ import annotations

import numpy as np

from .kvq import attention, node_chain, visible  # noqa: F401  (the same definitions)

ROW, KMAX = 640, 15


def e4m3_value(code: int) -> float:
    e, m = (code >> 3) & 15, code & 7
    v = float("nan") if code & 127 == 127 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
    return -v if code & 128 else v


VALUES = np.array([e4m3_value(i) for i in range(256)])
POSITIVE = VALUES[:127]


def nearest_code(x: float) -> int:
    """Code of the e4m3 number nearest x: ties to the even code, at most 448, NaN to 0."""
    if np.isnan(x):
        return 0
    a = min(abs(x), 448.0)
    d = np.abs(POSITIVE - a)
    best = np.flatnonzero(d == d.min())
    code = int(best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1])
    return code | (128 if np.signbit(x) else 0)


def nearest_codes(x) -> np.ndarray:
    """nearest_code of many numbers: the midpoints between neighbours decide."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    mid = (POSITIVE[1:] + POSITIVE[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    return (code + np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def bf16_bits(x) -> np.ndarray:
    """Nearest bf16 bit patterns (ties to even) of float64 numbers that fp32 holds."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    nan = np.isnan(np.asarray(x, np.float64))
    return np.where(nan, 0x7fff, (u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def needed(row, exponent: int) -> int:
    """The least k in 0..15 with every finite |x| <= 448 * 2^(exponent + k); 15 where there is none."""
    a = np.abs(np.asarray(row, np.float64))
    a = a[np.isfinite(a)].max(initial=0.0)
    for k in range(KMAX + 1):
        if a <= 448.0 * 2.0 ** (exponent + k):
            return k
    return KMAX


def pack_row(kv_c, k_pe, unit: float) -> np.ndarray:
    row = np.zeros(ROW, np.uint8)
    with np.errstate(over="ignore"):
        row[:512] = nearest_codes(np.asarray(kv_c, np.float64) / unit)
        row[512:] = bf16_bits(np.asarray(k_pe, np.float64) / unit).view(np.uint8)
    return row


def unpack_rows(rows, k, exponent: int = 0):
    """(latents, rope keys) float64 that rows stand for; k: scale of each row's block."""
    rows, unit = np.asarray(rows), 2.0 ** (exponent + np.asarray(k, np.float64))[:, None]
    return VALUES[rows[:, :512]] * unit, bf16_value(np.ascontiguousarray(rows[:, 512:]).view(np.uint16)) * unit


def write(rows, words, block: int, exponent: int, kv_c, k_pe, slots):
    """A write into host copies: rows [n][640] uint8, words [blocks] scale words.  Returns which rows of the pool
    have a defined value afterwards only if they had one before: those of grown blocks are requantised."""
    rows, words = rows.copy(), words.copy()
    need = {}
    for x, s in zip(kv_c, slots):
        if 0 <= s < len(rows):
            need[s // block] = max(need.get(s // block, 0), needed(x, exponent))
    for b, k in need.items():
        had = int(words[b])
        now = max(had, k + 1)
        words[b] = now
        d = now - had
        if had and d:
            a = rows[b * block:(b + 1) * block]
            v = VALUES[a[:, :512]]
            c = nearest_codes(np.where(np.isnan(v), 0, v) / 2.0 ** d)
            a[:, :512] = np.where(np.isnan(v), a[:, :512], c)
            r = bf16_value(np.ascontiguousarray(a[:, 512:]).view(np.uint16))
            a[:, 512:] = bf16_bits(r / 2.0 ** d).view(np.uint8).reshape(len(a), 128)
    for x, r, s in zip(kv_c, k_pe, slots):
        if 0 <= s < len(rows):
            rows[s] = pack_row(x, r, 2.0 ** (exponent + int(words[s // block]) - 1))
    return rows, words


def tables(page, Q, prefix, new, table, held, ring, state, num_pages, slots_len=None, words=None, block=1):
    """One call of the page tables on host lists.  Returns a dict of what it leaves behind."""
    table, held, ring = [list(r) for r in table], list(held), list(ring)
    head, tail = int(state[0]), int(state[1])
    words = None if words is None else list(words)
    slots, ptr, idx = [], [0], []
    taken, returned = [], []
    for b, p in enumerate(prefix):
        n = 0 if p < 0 else Q if new is None else new[b]
        length = p + n if p >= 0 else 0
        need = 0
        while need * page < length:
            need += 1
        while held[b] < need:
            id_ = ring[head % len(ring)]
            head += 1
            table[b][held[b]] = id_
            taken.append(id_)
            held[b] += 1
        for j in range(need, held[b]):
            returned.append(table[b][j])
            table[b][j] = -1
        held[b] = need
        at = [table[b][i // page] * page + i % page for i in range(length)]
        idx += at
        ptr.append(len(idx))
        if new is None:
            slots += at[p:] if p >= 0 else [-1] * Q
        elif p >= 0:
            slots += at[p:]
    for id_ in returned:
        ring[tail % len(ring)] = id_
        tail += 1
    if words is not None:
        for id_ in taken:
            for k in range(id_ * page // block, min((id_ + 1) * page // block + 1, len(words))):
                if id_ * page <= k * block and (k + 1) * block <= (id_ + 1) * page:
                    words[k] = 0
    if slots_len is not None:
        slots += [-1] * (slots_len - len(slots))
    return dict(table=table, held=held, ring=ring, state=[head, tail, 0], slots=slots, ptr=ptr, idx=idx, words=words)
