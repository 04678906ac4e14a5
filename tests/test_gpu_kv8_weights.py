"""What the 8-bit cache's attention keeps of small softmax weights: tokens behind one that
towers over them, and tokens of blocks whose scales differ, on both kernels.

Tolerance (derived, per element; as in test_gpu_kv8.py but for the small weights).  A weight
w_j enters as w_j 2^k_j relative to a unit that follows the tiles: T, the largest of a row
in a tile, is at least 2^F units, F = log2 n + d - 14 in the kernel for few rows (tiles of
128 tokens) and log2 n + d - 8 in that for many (64), for n tokens (counted as a power of
two) whose k_j differ by d at most.  Rounding it to f16 and cutting it into three bytes is
off by 2^-11 + 2^-9 of it, or, where it is small, by 2^-25 + LAST units, which are
    (2^-25 + LAST) 2^-F T / 2^k_j
in softmax weights.  LAST is half a step of the third byte: 2^-17, or 2^-23 in the kernel for
few rows, which keeps it times 2^6.  What is more than 2^40 below the row's largest so far may
be off by 2^-64 of that.  No weight is off by more than itself: below half a step it becomes
0, above that it is more than the error.
"""
import dataclasses

import numpy as np
import pytest

from mla_tree_verify_absorbed_gb300 import api
from oracle import kv8 as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


EXPONENT, SCALE = -6, 0.0721688
HEADS = [16, 33, 96]  # few rows in one group and in two, many


@dataclasses.dataclass
class Case:
    rows: np.ndarray    # the pool, slot = position
    words: np.ndarray
    block: int
    q: np.ndarray       # [H][576]

    def values(self):
        k = np.repeat(self.words.astype(np.int64) - 1, self.block)[:len(self.rows)]
        return (*O.unpack_rows(self.rows, k, EXPONENT), k)


def make(H, score, k, block, x, seed=0, size=2.0 ** -9):
    """Positions whose scores are about score[j] (natural units) for every head and whose latents are x [n][512] as
    far as blocks with scales k [blocks] hold them."""
    r = np.random.default_rng(seed)
    n = len(score)
    unit = 2.0 ** (EXPONENT + np.repeat(k, block)[:n])[:, None]
    rows = np.zeros((n, 640), np.uint8)
    rows[:, :512] = O.nearest_codes(x / unit)
    rope = np.repeat(np.asarray(score, np.float64)[:, None] / (SCALE * 64), 64, 1)
    rows[:, 512:] = O.bf16_bits(rope / unit).view(np.uint8).reshape(n, 128)
    q = np.ones((H, 576))
    q[:, :512] = r.standard_normal((H, 512)) * size
    return Case(rows, np.asarray(k, np.int32) + 1, block, torch.from_numpy(q).to(torch.bfloat16).double().numpy())


def oracle(c, H):
    """out, lse, and what they may be off by."""
    lat, rope, k = c.values()
    n = len(lat)
    tile, loss, last = (64, 8, 2.0 ** -17) if H > 64 else (128, 14, 2.0 ** -23)
    s = SCALE * (c.q[:, :512] @ lat.T + c.q[:, 512:] @ rope.T)
    smag = SCALE * (np.abs(c.q[:, :512]) @ np.abs(lat).T + np.abs(c.q[:, 512:]) @ np.abs(rope).T)
    top = s.max(-1, keepdims=True)
    w = np.exp(s - top)
    l = w.sum(-1, keepdims=True)
    w /= l
    out, mag, lse = w @ lat, w @ np.abs(lat), (top + np.log(l))[:, 0]
    # a query element of 0 is exact
    ds = (1096 * 2.0 ** -24 * smag
          + 2.0 ** -16.8 * SCALE * np.abs(c.q).max(-1)[:, None] * ((c.q[:, :512] != 0) @ np.abs(lat).T)).max(-1)
    dw = np.expm1(2 * ds + 2.0 ** -21) + 2.0 ** -11 + 2.0 ** -9 + 3 * n * 2.0 ** -24
    off = np.zeros_like(w)
    for a in range(0, n, tile):
        at = slice(a, a + tile)
        F = float(np.ceil(np.log2(len(k[at]))) + k[at].max() - k[at].min() - loss)
        T = (w[:, at] * 2.0 ** k[at]).max(-1, keepdims=True)
        off[:, at] = (2.0 ** -25 + last) * 2.0 ** -F * T / 2.0 ** k[at]
    off = np.minimum(off + 2.0 ** -64 * (w * 2.0 ** k).max(-1, keepdims=True) / 2.0 ** k, w)
    tol = 2.0 ** -8 * np.abs(out) + 1.01 * dw[:, None] * mag + off @ np.abs(lat)
    # the tolerance can tell a lost part from what is there
    assert np.median(tol) <= 0.1 * np.median(np.abs(out)), (np.median(tol), np.median(np.abs(out)))
    return out, tol, lse, ds + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse)


def check(c, H, copies):
    """The case as one sequence, cut into pieces, and as one of many, most of them whole in a piece."""
    n = len(c.rows)
    out, tol, lse, ltol = oracle(c, H)
    cache = api.BlockCache(torch.from_numpy(c.rows).cuda(), torch.from_numpy(c.words).cuda(), c.block, EXPONENT)
    q = torch.from_numpy(c.q).to(torch.bfloat16).cuda()
    for B in (1, copies):
        i32 = dict(dtype=torch.int32, device="cuda")
        ki = api.Kv8Inputs(B=B, Q=1, H=H, scale=SCALE, q_lat=q[:, :512].expand(B, 1, H, 512).contiguous(),
                           q_pe=q[:, 512:].expand(B, 1, H, 64).contiguous(), cache=cache,
                           prefix_lens=torch.full((B,), n - 1, **i32), page_size=1,
                           kv_indptr=torch.arange(B + 1, **i32) * n, kv_indices=torch.arange(n, **i32).repeat(B))
        ws = api.alloc_workspace(api.kv8_workspace_size(ki))
        o, l = api.kv8_attn(ki, workspace=ws)
        assert api.kv8_check(ws) == 0
        for b in {0, 1 % B, B // 3, B // 2, B - 1}:
            got, gl = o[b, 0].double().cpu().numpy(), l[b, 0].double().cpu().numpy()
            bad = ~(np.abs(got - out) <= tol)
            assert not bad.any(), (B, b, bad.mean(), np.argwhere(bad)[:3], np.abs(got - out).max(), np.abs(out).max())
            assert (np.abs(gl - lse) <= ltol).all(), (B, b, np.abs(gl - lse).max(), ltol.min())


def latents(n, seed=1):
    """Values around 1/2, not around 0: a mean over many is as large as they are."""
    return 0.5 + 0.25 * np.random.default_rng(seed).standard_normal((n, 512))


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("at", [0, 1400, 2899])
@pytest.mark.parametrize("bits", [6, 12, 18, 24, 30, 38])
def test_tail_of_a_needle_without_latents(bits, at, H):
    # one token 2^bits above all others, which alone have latents
    n = 2900
    x, score = latents(n), np.zeros(n)
    x[at], score[at] = 0, bits * np.log(2)
    check(make(H, score, [0] * -(-n // 64), 64, x), H, 400)


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("block", [1, 64])
@pytest.mark.parametrize("k,bits", [(3, 12), (8, 16), (15, 9), (15, 16), (15, 24)])
def test_tail_of_a_needle_in_a_coarse_block(k, bits, block, H):
    # the needle's block has the larger unit, as one large neighbour makes it; its own latents are small
    n = 2900
    x, score = latents(n), np.zeros(n)
    x[0], score[0] = x[0] / 8, bits * np.log(2)
    kk = np.zeros(-(-n // block), int)
    kk[0] = k
    check(make(H, score, kk, block, x), H, 400)


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("period,bits", [(64, 9), (128, 9), (128, 20), (128, 33), (256, 20), (256, 33), (200, 9), (200, 13)])
def test_heights_that_come_and_go(period, bits, H):
    # every second period of tokens is 2^bits above the others and without latents: the unit falls and rises
    n = 1600
    high = np.arange(n) // period % 2 == 0
    x = latents(n)
    x[high] = 0
    check(make(H, np.where(high, bits * np.log(2), 0.0), [0] * -(-n // 16), 16, x), H, 400)


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("block,spread", [(1, 2), (1, 7), (1, 8), (1, 15), (2, 15), (3, 11), (64, 15), (128, 15), (1000, 15)])
def test_scales_that_differ(block, spread, H):
    # values of one size in blocks of very different units, scores that vary a little: what small codes stand for
    # counts as much as what large ones do
    n = 1500
    r = np.random.default_rng(5)
    k = r.integers(0, spread + 1, -(-n // block))
    k[0], k[-1] = spread, 0
    # in a block of scale k the latents are at least 2^(k - 6): the smallest code stands for 2^(k - 15)
    size = 2.0 ** (np.minimum(np.repeat(k, block)[:n], 6) - 6)
    check(make(H, r.standard_normal(n), k, block, latents(n) * size[:, None]), H, 400)


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("d", [8, 10, 13, 15])
def test_a_coarse_token_in_every_tile(d, H):
    # one token of each 32 in a unit 2^d times the others', with a larger weight and without latents
    n = 1500
    k, score, x = np.zeros(n, int), np.zeros(n), latents(n)
    k[::32], x[::32] = d, 0
    score[::32] = np.log(2) * np.arange(len(score[::32])) % 9
    check(make(H, score, k, 1, x), H, 400)


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("bits", [60, 90, 126])
def test_heights_beyond_what_is_followed(bits, H):
    # full codes in coarse blocks, far above a long tail: nothing overflows on the way down, and what is above comes out
    n = 2000
    x, score, k = latents(n), np.zeros(n), np.zeros(n, int)
    x[5:200], score[5:200], k[5:200] = 448 * 2.0 ** (EXPONENT + 15), bits * np.log(2), 15
    check(make(H, score, k, 1, x, size=0), H, 400)


@pytest.mark.parametrize("H", HEADS)
def test_heads_that_move_beside_heads_that_do_not(H):
    # every second head's scores are 32 times as wide
    n = 1500
    r = np.random.default_rng(7)
    score = 0.5 * r.standard_normal(n)
    c = make(H, score, [0] * -(-n // 64), 64, latents(n))
    c2 = dataclasses.replace(c, q=c.q.copy())
    c2.q[1::2] *= 32
    check(c, H, 400)
    check(c2, H, 400)
