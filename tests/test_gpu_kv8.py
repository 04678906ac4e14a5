"""The paged 8-bit latent cache on the GPU: written rows, scales and read-back bit for
bit, the attention against the float64 oracle, masks, tables, streams and graphs.

Tolerance of the attention (derived, per element).  Codes enter the products exactly
and everything accumulates in fp32, so against float64:
  * a query element is off by at most 2^-9 where its row's largest is scaled to at
    least 224, so a score by 2^-16.8 * max|q| * sum |code| unit * scale, and by
    (2 * 512 + 64 + 8) * 2^-24 * sum |q||k| * scale from its additions (two terms per
    latent product; the units and the argument of exp)  =: ds together;
  * a weight by a factor 1 +- (2 ds + 2^-21): numerator and normaliser, and the
    hardware exponential's 2^-22 in each; rounding it to f16 and cutting it into three
    bytes adds 2^-11 + 2^-9, and 2^-24 of the largest weight times 2^k where it falls
    below what the bytes reach;
  * the sums over n tokens (three terms each) by 3 n * 2^-24 of the sums of magnitudes;
  * the result's rounding to bf16 by 2^-8 of the value.
lse: ds + 2^-21 + n * 2^-24 from the normaliser, and fp32 rounding 2^-22 |lse|.
"""
import dataclasses
import time

import numpy as np
import pytest

from mla_tree_verify_absorbed_gb300 import api
from oracle import kv8 as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SLOT, NONFINITE, PREFIX, INDPTR, PARENT, PAGES, CAPACITY, TIMEOUT = 0x4, 0x200, 0x1, 0x2, 0x8, 0x10, 0x20, 0x40


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
def latents(kind, n, dtype, seed, exponent=0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, 512)) * 2.0 ** (exponent + 7)
    if kind == "sizes":  # rows of very different sizes: blocks grow
        x *= 2.0 ** r.integers(-3, 9, (n, 1))
    elif kind == "ties":  # midpoints of neighbouring codes
        x = (O.POSITIVE[1:] + O.POSITIVE[:-1])[r.integers(0, 126, (n, 512))] / 2 * r.choice([-1, 1], (n, 512))
        x *= 2.0 ** exponent
    elif kind == "borders":  # largest magnitudes at the border between two scales, and the bf16 number above it
        x = r.uniform(-1, 1, (n, 512))
        k = r.integers(0, 15, n)
        x[np.arange(n), r.integers(0, 512, n)] = 448.0 * 2.0 ** k * r.choice([-1.0, 1.0, 1 + 2.0 ** -7], n)
        x *= 2.0 ** exponent
    elif kind == "huge":
        x *= 2.0 ** r.integers(8, 40, (n, 1))
    elif kind == "tiny":
        x *= 2.0 ** r.integers(-20, -6, (n, 1))
    elif kind == "zeros":
        x[:, :256] = 0
        x[0] = -0.0
    t = torch.from_numpy(x).to(torch.float32).to(dtype)
    k = torch.from_numpy(r.standard_normal((n, 64))).to(torch.float32).to(dtype)
    return t, k


def check_write(cache, t, k, at, status=0):
    """Writes on the device and in the oracle: the same bytes and words."""
    rows, words = cache.rows.cpu().numpy(), cache.scales.cpu().numpy().astype(np.int64)
    want, want_words = O.write(rows, words, cache.block, cache.exponent, t.double().numpy(), k.double().numpy(), list(at))
    ws = api.kv8_write(cache, t.cuda(), k.cuda(), i32(at))
    assert api.kv8_check(ws) == status
    assert np.array_equal(cache.scales.cpu().numpy(), want_words)
    got = cache.rows.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind,exponent,block", [("normal", -7, 8), ("sizes", -7, 8), ("sizes", 3, 5), ("sizes", -32, 1),
                                                 ("sizes", 32, 64), ("ties", 0, 16), ("borders", 0, 4),
                                                 ("borders", -9, 1), ("huge", 0, 16), ("tiny", -7, 8), ("zeros", 1, 7)])
def test_writes_are_the_oracles_bytes(kind, exponent, block, dtype):
    # three writes into one cache: empty blocks, blocks that hold rows and grow, rows that are written over
    slots = 70
    cache = api.kv8_alloc(slots, block, exponent)
    for step in range(3):
        n = 23
        t, k = latents(kind, n, dtype, 11 + step, exponent)
        if step == 1:
            t = t / 8
        at = np.random.default_rng(5 + step).permutation(slots)[:n]
        at[3] = at[n - 1] = -1
        check_write(cache, t, k, at)
    rows, words = cache.rows.cpu().numpy(), cache.scales.cpu().numpy()
    keep = at >= 0
    lat, rope = O.unpack_rows(rows[at[keep]], np.maximum(words[at[keep] // block] - 1, 0), exponent)
    for name, dt in (("bf16", torch.bfloat16), ("fp32", torch.float32)):
        c0, r0 = torch.full((n, 512), 5.0, dtype=dt).cuda(), torch.full((n, 64), 6.0, dtype=dt).cuda()
        c, r, ws = api.kv8_read(cache, i32(at), kv_c=c0, k_pe=r0)
        assert api.kv8_check(ws) == 0
        assert np.array_equal(c.double().cpu().numpy()[keep], lat)
        assert np.array_equal(r.double().cpu().numpy()[keep], rope)
        assert (c.float().cpu().numpy()[~keep] == 5).all() and (r.float().cpu().numpy()[~keep] == 6).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 2, 7, 64, 127, 128, 129, 255, 256, 257, 2433, 9001])
def test_rows_of_any_count_with_strides(n, dtype):
    # one wide array holds kv_c and k_pe; cache rows 672 bytes apart; the last block is not whole; sizes differ
    slots, block = n + 3, 13
    t, k = latents("sizes", min(n, 50), dtype, 12, -7)
    rep = -(-n // 50)
    wide = torch.full((n, 704), 9.0, dtype=dtype)
    wide[:, :512] = t.repeat(rep, 1)[:n]
    wide[:, 640:] = k.repeat(rep, 1)[:n]
    pool = torch.zeros((slots, 672), dtype=torch.uint8, device="cuda")
    pool[:, 640:] = 7
    cache = api.BlockCache(pool[:, :640], torch.zeros(-(-slots // block), dtype=torch.int32, device="cuda"), block, -7)
    for step in range(2):  # the second time some blocks hold rows already
        at = np.random.default_rng(n + step).permutation(slots)[:n]
        rows, words = cache.rows.cpu().numpy(), cache.scales.cpu().numpy().astype(np.int64)
        x = wide[:, :512].double().numpy() * 4.0 ** step
        want, ww = O.write(rows, words, block, -7, x, wide[:, 640:].double().numpy(), list(at))
        w = wide.clone()
        w[:, :512] *= 4.0 ** step
        w = w.cuda()
        assert api.kv8_check(api.kv8_write(cache, w[:, :512], w[:, 640:], i32(at))) == 0
        assert np.array_equal(cache.scales.cpu().numpy(), ww) and np.array_equal(cache.rows.cpu().numpy(), want)
    assert bool((pool[:, 640:] == 7).all())
    back = torch.full((n, 704), 3.0, dtype=dtype, device="cuda")
    api.kv8_read(cache, i32(at), kv_c=back[:, :512], k_pe=back[:, 640:])
    lat, rope = O.unpack_rows(want[at], ww[at // block] - 1, -7)
    assert np.array_equal(back[:, :512].double().cpu().numpy(), lat)
    assert np.array_equal(back[:, 640:].double().cpu().numpy(), rope)
    assert bool((back[:, 512:640] == 3).all())


@pytest.mark.parametrize("n", [300, 40])
def test_many_rows_of_one_block_grow_it_once(n):
    # every row of the call goes to one block that holds rows already, and each needs more than the one before
    cache = api.kv8_alloc(800, 800, -7)
    t, k = latents("normal", 100, torch.float32, 3, -7)
    check_write(cache, t, k, range(700, 800))
    t, k = latents("normal", n, torch.float32, 4, -7)
    check_write(cache, t * 2.0 ** (torch.arange(n)[:, None] % 12), k, np.random.default_rng(0).permutation(700)[:n])
    # codes that fall off the lower end, and rope keys that do not
    assert cache.scales.tolist()[0] > 10


def test_a_block_that_was_empty_keeps_its_other_bytes():
    cache = api.kv8_alloc(64, 16, 0)
    cache.rows.fill_(0x7f)
    t, k = latents("huge", 3, torch.bfloat16, 2)
    check_write(cache, t, k, [17, 30, 50])
    assert bool((cache.rows[[16, 18, 31, 48, 63]] == 0x7f).all()) and cache.scales.tolist()[0] == 0


def test_words_that_nobody_wrote():
    # any 32 bits in a word read as some scale: nothing is written outside the rows
    cache = api.kv8_alloc(64, 16, 0)
    cache.scales.copy_(torch.tensor([-1, 2 ** 31 - 1, 200, 17], dtype=torch.int32))
    t, k = latents("normal", 8, torch.bfloat16, 2)
    at = i32(range(0, 64, 8))
    assert api.kv8_check(api.kv8_write(cache, t.cuda(), k.cuda(), at)) == 0
    assert set(cache.scales.tolist()) <= set(range(1, 17))
    c, _, _ = api.kv8_read(cache, at)
    assert bool(torch.isfinite(c.float()).all())


def test_read_of_any_bytes():
    rng = np.random.default_rng(2)
    rows = rng.integers(0, 256, (300, 640), dtype=np.uint8)
    rows[:, :512][rows[:, :512] & 127 == 127] = 5  # NaN would not compare
    rows[:, 513::2] &= 0xbf
    words = rng.integers(0, 17, 38).astype(np.int32)
    at = rng.integers(0, 300, 500)  # slots named several times
    for exponent in (0, -32, 32, 5):
        cache = api.BlockCache(torch.from_numpy(rows).cuda(), i32(words), 8, exponent)
        lat, rope = O.unpack_rows(rows[at], np.maximum(words[at // 8] - 1, 0), exponent)
        for name in ("bf16", "fp32"):
            c, r, ws = api.kv8_read(cache, i32(at), name)
            assert api.kv8_check(ws) == 0
            assert np.array_equal(c.double().cpu().numpy(), lat)
            fits = np.abs(rope) < 3e38  # a rope key times 2^47 may leave the type
            fits &= (np.abs(rope) > 1e-37) | (rope == 0)
            assert np.array_equal(r.double().cpu().numpy()[fits], rope[fits])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [4, 600])
def test_write_of_infinities_and_nan(dtype, n):
    t, k = latents("normal", n, dtype, 13)
    t[1, 20], t[1, 40], t[2, 511], t[2, 500] = float("inf"), float("nan"), float("-inf"), float("nan")
    k[3, 7], k[3, 8] = float("nan"), float("inf")
    cache = api.kv8_alloc(n, 1)
    ws = api.kv8_write(cache, t.cuda(), k.cuda(), i32(range(n)))
    assert api.kv8_check(ws) == NONFINITE
    c, r, _ = api.kv8_read(cache, i32(range(n)), "fp32")
    k1, k2 = cache.scales[1].item() - 1, cache.scales[2].item() - 1
    assert k1 <= 2 and float(c[1, 20]) == 448 * 2.0 ** k1 and float(c[1, 40]) == 0
    assert float(c[2, 511]) == -448 * 2.0 ** k2
    assert bool(torch.isnan(r[3, 7])) and float(r[3, 8]) == float("inf")
    # only rope keys are not finite: no error
    assert api.kv8_check(api.kv8_write(cache, t[3:4].cuda(), k[3:4].cuda(), i32([0]))) == 0


@pytest.mark.parametrize("pad", [0, 400])
def test_slots_outside_the_pool(pad):
    t, k = latents("normal", 5 + pad, torch.bfloat16, 14)
    pool = torch.full((12, 640), 1, dtype=torch.uint8, device="cuda")
    cache = api.BlockCache(pool[2:10], torch.zeros(2, dtype=torch.int32, device="cuda"), 4)
    at = [3, 8, -2, 0, 2 ** 31 - 1] + [-1] * pad
    check_write(cache, t, k, at, SLOT)
    assert bool((pool[[0, 1, 10, 11]] == 1).all())
    c, r = torch.full((5 + pad, 512), 2.0, device="cuda"), torch.full((5 + pad, 64), 2.0, device="cuda")
    _, _, ws = api.kv8_read(cache, i32(at), kv_c=c, k_pe=r)
    assert api.kv8_check(ws) == SLOT
    assert bool((c[[1, 2, 4]] == 2).all()) and bool((r[[1, 2, 4]] == 2).all()) and bool((c[[0, 3]] != 2).any())
    # the next call on the workspace starts without the error
    api.kv8_read(cache, i32([0] * (5 + pad)), kv_c=c, k_pe=r, workspace=ws)
    assert api.kv8_check(ws) == 0


def test_rows_beyond_32_bit_offsets():
    # slot 7,000,000 lies 4.5 GB into the pool
    n = 7_000_001
    cache = api.BlockCache(torch.empty((n, 640), dtype=torch.uint8, device="cuda"),
                           torch.zeros(-(-n // 64), dtype=torch.int32, device="cuda"), 64, -7)
    t, k = latents("normal", 3, torch.bfloat16, 15, -7)
    at = [n - 1, 5_200_000, 0]
    api.kv8_write(cache, t.cuda(), k.cuda(), i32(at))
    words = cache.scales.cpu().numpy()
    want = np.stack([O.pack_row(a, b, 2.0 ** (words[s // 64] - 8)) for a, b, s in
                     zip(t.double().numpy(), k.double().numpy(), at)])
    assert np.array_equal(cache.rows[torch.tensor(at).cuda()].cpu().numpy(), want)
    c, _, ws = api.kv8_read(cache, i32(at), "fp32")
    assert api.kv8_check(ws) == 0
    kk = words[np.array(at) // 64] - 1
    assert np.array_equal(c.double().cpu().numpy(), O.unpack_rows(want, kk, -7)[0])
    # the attention reads the same rows, with few query rows and with many
    for H in (4, 70):
        p = problem(B=1, Q=1, H=H, lens=[2], seed=3)
        ki = dataclasses.replace(p.ki, cache=cache, kv_indices=i32(at), kv_indptr=i32([0, 3]))
        check_attn(dataclasses.replace(p, ki=ki, rows=want, k=kk, slots=[np.arange(3)]))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class Prob:
    ki: object
    rows: np.ndarray        # host copy of the cache's rows,
    k: np.ndarray           # and the scale of each
    slots: list             # per sequence: pool slot of each position
    lens: list
    parent: np.ndarray


def random_parents(B, Q, seed, kind="tree"):
    r = np.random.default_rng(seed)
    par = np.zeros((B, Q), np.int32)
    for b in range(B):
        for i in range(Q):
            par[b, i] = i - 1 if kind == "chain" else r.integers(-1, i) if kind == "forest" else r.integers(0, max(i, 1))
        par[b, 0] = -1
    return par


def problem(B=1, Q=4, H=8, lens=None, page=1, seed=0, tree="tree", window=0, sinks=0, exponent=-6, q_scale=1.0,
            scale=0.0721688, stride=640, freed=False, block=16, spread=3):
    r = np.random.default_rng(seed)
    need = [0 if v < 0 else v + Q for v in lens]
    slots = []
    if page == 1:
        pool = sum(need) + 9
        idx = r.permutation(pool)[:sum(need)].astype(np.int32)
        ptr = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
        slots = [idx[ptr[b]:ptr[b + 1]].copy() for b in range(B)]
        table = idx if len(idx) else np.zeros(1, np.int32)
    else:
        count = sum(-(-v // page) for v in need) + 2
        pool = count * page
        ids = r.permutation(count).astype(np.int32)
        width = max(max(-(-v // page) for v in need), 1) + 1
        table = np.full((B, width), -1, np.int32)
        at = 0
        for b, v in enumerate(need):
            c = -(-v // page)
            table[b, :c] = ids[at:at + c]
            at += c
            slots.append((table[b, np.arange(v) // page].astype(np.int64) * page + np.arange(v) % page))
    if freed:  # entries that no node sees
        for b, v in enumerate(lens):
            if v < 0:
                continue
            lo = max(0, v - window + 1)
            if page == 1:
                a = ptr[b] + min(sinks, v)
                table[a:max(a, ptr[b] + lo)] = 2 ** 31 - 1 if b % 2 else -5
            else:
                a, z = -(-sinks // page), lo // page
                if z > a:
                    table[b, a:z] = 2 ** 31 - 1 if b % 2 else -1
    # latents of about unit size whatever their block's scale
    words = r.integers(1, 2 + spread, -(-pool // block)).astype(np.int32)
    k = np.repeat(words - 1, block)[:pool]
    unit = 2.0 ** (exponent + k)[:, None]
    gain = np.exp(0.4 * r.standard_normal(512))
    rows = np.zeros((pool, 640), np.uint8)
    x = (r.standard_normal((pool, 512)) * gain * 2.0 ** (exponent + 6) / unit).clip(-448, 448)
    rows[:, :512] = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    rows[:, 512:] = O.bf16_bits(r.standard_normal((pool, 64)) / unit).view(np.uint8).reshape(pool, 128)
    # rows that no position names hold anything
    used = np.zeros(pool, bool)
    for s in slots:
        used[np.asarray(s, np.int64)] = True
    rows[~used] = 0xff
    buf = torch.zeros((pool, stride), dtype=torch.uint8)
    buf[:, :640] = torch.from_numpy(rows)
    parent = random_parents(B, Q, seed + 2, tree)
    q = torch.from_numpy(q_scale * r.standard_normal((B, Q, H, 576))).to(torch.bfloat16)
    kw = dict(kv_indptr=i32(ptr), kv_indices=i32(table)) if page == 1 else dict(block_table=i32(table))
    cache = api.BlockCache(buf.cuda()[:, :640], i32(words), block, exponent)
    ki = api.Kv8Inputs(B=B, Q=Q, H=H, scale=scale, q_lat=q[..., :512].contiguous().cuda(),
                       q_pe=q[..., 512:].contiguous().cuda(), cache=cache, prefix_lens=i32(lens), page_size=page,
                       tree_parent=None if tree == "null" else i32(parent), window=window, sinks=sinks, **kw)
    if tree == "null":
        parent = random_parents(B, Q, 0, "chain")
    return Prob(ki, rows, k, slots, list(lens), parent)


def run(ki, **kw):
    out, lse = api.kv8_attn(ki, **kw)
    torch.cuda.synchronize()
    return out, lse


def compare(p, out, lse):
    ki = p.ki
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, P in enumerate(p.lens):
        if P < 0:
            continue
        k = np.asarray(p.k)[p.slots[b]]
        lat, rope = O.unpack_rows(p.rows[p.slots[b]], k, ki.cache.exponent)
        ql, qp = ki.q_lat[b].double().cpu().numpy(), ki.q_pe[b].double().cpu().numpy()
        o, l, mag, smag = O.attention(lat, rope, ql, qp, ki.scale, p.parent[b], P, ki.H, ki.window, ki.sinks)
        n = P + ki.Q
        qmax = np.maximum(np.abs(ql).max(-1), np.abs(qp).max(-1))
        ds = 1096 * 2.0 ** -24 * smag + 2.0 ** -16.8 * ki.scale * qmax * np.abs(lat).sum(1).max()
        dw = np.expm1(2 * ds + 2.0 ** -21) + 2.0 ** -11 + 2.0 ** -9 + 3 * n * 2.0 ** -24
        # weights below the bytes' range: 2^-24 of the largest weight (at most 1) times 2^k, against their codes
        top = 2.0 ** -24 * (2.0 ** (k.max() - k)[:, None] * np.abs(lat)).sum(0)
        tol = 2.0 ** -8 * np.abs(o) + 1.01 * dw[..., None] * mag + top
        bad = ~(np.abs(out[b] - o) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(out[b] - o).max(), tol.min())
        ltol = ds + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(l)
        bad = ~(np.abs(lse[b] - l) <= ltol)
        assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(lse[b] - l).max(), ltol.min())


def check_attn(p, **kw):
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    ws.fill_(0xee)  # a workspace needs no clearing
    out, lse = run(p.ki, workspace=ws, **kw)
    assert api.kv8_check(ws) == 0
    compare(p, out, lse)
    return out, lse


# shapes with one thing out of the ordinary each: lengths of 0 and 1, tile and page borders, head counts around the
# row groups (32 rows in the kernel for few rows, 128 in the other) and around the choice between the kernels
SHAPES = [
    dict(B=1, Q=1, H=1, lens=[0]),
    dict(B=1, Q=1, H=16, lens=[1]),
    dict(B=1, Q=1, H=17, lens=[126], tree="null"),
    dict(B=1, Q=1, H=32, lens=[127], tree="null"),
    dict(B=1, Q=1, H=33, lens=[128], tree="null"),
    dict(B=1, Q=2, H=32, lens=[255]),
    dict(B=1, Q=1, H=65, lens=[0]),
    dict(B=1, Q=1, H=128, lens=[62], tree="null"),
    dict(B=1, Q=1, H=128, lens=[63], tree="null"),
    dict(B=1, Q=1, H=129, lens=[64], tree="null"),
    dict(B=1, Q=3, H=43, lens=[128]),
    dict(B=1, Q=64, H=5, lens=[0], tree="forest"),
    dict(B=1, Q=64, H=1, lens=[0], tree="forest"),
    dict(B=2, Q=64, H=16, lens=[301, 0], tree="tree"),
    dict(B=3, Q=8, H=16, lens=[700, 0, 1500], tree="forest"),
    dict(B=3, Q=8, H=8, lens=[700, 0, 1500], tree="forest"),
    dict(B=3, Q=5, H=7, lens=[33, 3000, 1], page=16),
    dict(B=3, Q=5, H=20, lens=[33, 3000, 1], page=16),
    dict(B=2, Q=17, H=3, lens=[999, 65], page=100, tree="null"),
    dict(B=4, Q=1, H=16, lens=[5, -1, 257, -1], page=64, tree="null"),
    dict(B=4, Q=1, H=96, lens=[5, -1, 257, -1], page=64, tree="null"),
    dict(B=5, Q=3, H=9, lens=[-1, 60, -1, 61, 62], tree="chain"),
    dict(B=1, Q=4, H=64, lens=[2900], stride=672),
    dict(B=1, Q=4, H=10, lens=[2900], stride=672),
    dict(B=70, Q=1, H=2, lens=[(37 * i) % 400 for i in range(70)], tree="null"),
    dict(B=1, Q=64, H=64, lens=[130], tree="chain"),
    dict(B=1, Q=7, H=8, lens=[2000], page=1 << 13),
    dict(B=1, Q=7, H=18, lens=[2000], page=1 << 13),
]


@pytest.mark.parametrize("kw", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_attention_matches_oracle(kw):
    check_attn(problem(seed=21, **kw))


@pytest.mark.parametrize("H", [8, 40])
@pytest.mark.parametrize("block,spread", [(1, 0), (1, 3), (2, 15), (7, 3), (64, 3), (128, 15), (10 ** 6, 3), (2 ** 31 - 1, 0)])
def test_blocks_and_scales(block, spread, H):
    check_attn(problem(B=2, Q=3, H=H, lens=[500, 1290], seed=22, block=block, spread=spread, exponent=-6 - spread // 2))


@pytest.mark.parametrize("H", [8, 40])
@pytest.mark.parametrize("exponent", [-32, 0, 7, 32])
def test_attention_exponent(exponent, H):
    # latents and scores scale by 2^(exponent + 6), rope keys do not: a scale that keeps the scores moderate
    check_attn(problem(B=2, Q=3, H=H, lens=[200, 77], seed=22, exponent=exponent,
                       scale=0.07 * 2.0 ** -max(exponent + 6, 0)))


@pytest.mark.parametrize("H", [8, 40])
@pytest.mark.parametrize("scale,q_scale", [(1e-6, 1.0), (1.0, 1.0), (8.0, 3.0), (0.07, 100.0), (1e30, 2.0 ** -100),
                                           (1e-20, 2.0 ** 60)])
def test_attention_flat_and_sharp(scale, q_scale, H):
    # flat: a mean over all rows; sharp: the running maximum moves over thousands; queries far from 1
    check_attn(problem(B=2, Q=4, H=H, lens=[1500, 300], seed=23, scale=scale, q_scale=q_scale))


def test_rows_of_queries_of_very_different_sizes():
    p = problem(B=1, Q=2, H=40, lens=[700], seed=26)
    f = 2.0 ** (torch.arange(80, device="cuda").view(1, 2, 40, 1) % 20 - 12)
    p.ki.q_lat.mul_(f)
    p.ki.q_pe.mul_(f)
    p.ki.q_lat[0, 0, 3] = 0
    p.ki.q_lat[0, 1, 7], p.ki.q_pe[0, 1, 7] = 0, 0     # every score 0
    p.ki.q_lat[0, 0, 5, :256] *= 2.0 ** -12            # elements of which one term is left, or none
    check_attn(p)
    q = p.ki
    few = dataclasses.replace(q, H=10, q_lat=q.q_lat[:, :, :10].contiguous(), q_pe=q.q_pe[:, :, :10].contiguous())
    check_attn(dataclasses.replace(p, ki=few))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("H", [8, 40])
def test_queries_that_are_not_finite_make_nan_rows_only_of_their_own(H, value):
    p = problem(B=2, Q=2, H=H, lens=[300, 40], seed=27)
    out, lse = run(p.ki)
    p.ki.q_lat[0, 1, 3, 77] = value
    p.ki.q_pe[1, 0, 5, 9] = value
    o, l = run(p.ki)
    for b, i, h in ((0, 1, 3), (1, 0, 5)):
        assert bool(torch.isnan(o[b, i, h].float()).all()) and bool(torch.isnan(l[b, i, h]))
        o[b, i, h], l[b, i, h] = out[b, i, h], lse[b, i, h]
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("H", [2, 80])
def test_rising_maximum(H):
    # keys sorted by their score against the even heads' query: their maximum rises with every tile, the others' falls
    p = problem(B=1, Q=1, H=H, lens=[1600], seed=24, tree="null", q_scale=2.0)
    lat, rope = O.unpack_rows(p.rows, p.k, -6)
    p.ki.q_lat[0, 0, 0::2], p.ki.q_pe[0, 0, 0::2] = p.ki.q_lat[0, 0, 0].clone(), p.ki.q_pe[0, 0, 0].clone()
    p.ki.q_lat[0, 0, 1::2], p.ki.q_pe[0, 0, 1::2] = -p.ki.q_lat[0, 0, 0], -p.ki.q_pe[0, 0, 0]
    s = lat[p.slots[0]] @ p.ki.q_lat[0, 0, 0].double().cpu().numpy() \
        + rope[p.slots[0]] @ p.ki.q_pe[0, 0, 0].double().cpu().numpy()
    p.slots[0] = p.slots[0][np.argsort(s)]
    p.ki.kv_indices.copy_(i32(p.slots[0]))
    check_attn(p)


@pytest.mark.parametrize("tiles", [2, 3, 5, 8, 11])
def test_some_rows_maxima_move_at_every_tile_and_others_never(tiles):
    for H in (64, 128):
        p = problem(B=1, Q=1, H=H, lens=[128 * tiles - 1], seed=60, tree="null")
        half = H // 2
        p.ki.q_lat[0, 0, half:] = p.ki.q_lat[0, 0, half].clone() * 16
        p.ki.q_pe[0, 0, half:] = p.ki.q_pe[0, 0, half].clone() * 16
        p.ki.q_lat[0, 0, :half] *= 2.0 ** -6
        p.ki.q_pe[0, 0, :half] *= 2.0 ** -6
        lat, rope = O.unpack_rows(p.rows, p.k, -6)
        s = lat[p.slots[0]] @ p.ki.q_lat[0, 0, half].double().cpu().numpy() \
            + rope[p.slots[0]] @ p.ki.q_pe[0, 0, half].double().cpu().numpy()
        p.slots[0] = p.slots[0][np.argsort(s)]
        p.ki.kv_indices.copy_(i32(p.slots[0]))
        for _ in range(3):
            check_attn(p)


@pytest.mark.parametrize("H", [16, 128])
def test_a_needle_over_a_flat_tail(H):
    # one token far above 60,000 that score alike and together weigh as much: their weights must not be lost
    n = 60_000
    p = problem(B=1, Q=1, H=H, lens=[n], seed=28, tree="null", block=1 << 20, spread=0)
    row = p.rows[p.slots[0][0]].copy()
    row[512:] = 0
    rows = np.tile(row, (len(p.rows), 1))
    needle = p.slots[0][3]
    rows[needle, :512] = O.nearest_codes(np.random.default_rng(1).standard_normal(512) * 64)
    rows[needle, 512:] = np.tile(O.bf16_bits(np.array([64.0])), 64).view(np.uint8)
    p.ki.cache.rows.copy_(torch.from_numpy(rows))
    lat, _ = O.unpack_rows(rows[p.slots[0][:4]], np.zeros(4), -6)
    # q_pe makes up the distance: exactly ln(n) above the others' score, more or less
    q = p.ki.q_lat.double().cpu().numpy()[0, 0]
    gap = (np.log(n) / p.ki.scale - q @ (lat[3] - lat[0])) / 64
    p.ki.q_pe.copy_(torch.from_numpy(np.repeat(gap[None, None, :, None], 64, -1)).to(torch.bfloat16))
    check_attn(dataclasses.replace(p, rows=rows))


@pytest.mark.parametrize("rows", [129, 198, 225, 1, 33, 17, 64, 65])
def test_row_groups_with_few_rows_between_full_ones(rows):
    # many sequences of a few row groups, the last of them a fraction of one, so that a worker's pieces alternate
    # between groups that use all rows and groups that leave most out
    n = 24
    check_attn(problem(B=n, Q=1, H=rows, lens=[(97 * i) % 700 for i in range(n)], page=16, seed=25, tree="null"))


WINDOWS = [
    dict(B=1, Q=1, H=4, lens=[500], window=1, sinks=0),
    dict(B=1, Q=1, H=4, lens=[500], window=1, sinks=1),
    dict(B=1, Q=1, H=16, lens=[500], window=64, sinks=4),
    dict(B=1, Q=1, H=16, lens=[511], window=129, sinks=128),
    dict(B=1, Q=1, H=80, lens=[511], window=65, sinks=64),
    dict(B=2, Q=8, H=8, lens=[900, 30], window=100, sinks=70, tree="tree"),
    dict(B=2, Q=64, H=4, lens=[777, 5], window=9, sinks=7, tree="chain"),
    dict(B=2, Q=64, H=1, lens=[777, 5], window=9, sinks=7, tree="chain"),
    dict(B=2, Q=64, H=4, lens=[777, 5], window=9, sinks=40, tree="null"),
    dict(B=1, Q=64, H=3, lens=[0], window=5, sinks=20, tree="forest"),
    dict(B=3, Q=5, H=8, lens=[1000, 1000, 63], window=1 << 30, sinks=3, tree="forest"),
    dict(B=3, Q=5, H=18, lens=[1000, 100, 63], window=333, sinks=1 << 30, tree="forest"),
    dict(B=4, Q=2, H=8, lens=[2000, -1, 64, 640], window=130, sinks=66, page=16, tree="null"),
    dict(B=2, Q=33, H=6, lens=[1999, 450], window=200, sinks=129, page=48, tree="tree"),
    dict(B=3, Q=9, H=7, lens=[0, 500, 61], window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    dict(B=3, Q=9, H=8, lens=[0, 500, 61], window=1, sinks=2 ** 31 - 1),
]


@pytest.mark.parametrize("freed", [False, True], ids=["tables", "freed"])
@pytest.mark.parametrize("kw", WINDOWS, ids=[f"{i}" for i in range(len(WINDOWS))])
def test_window_and_sinks_match_oracle(kw, freed):
    check_attn(problem(seed=31, freed=freed, **kw))


@pytest.mark.parametrize("H", [8, 40])
def test_rows_that_a_node_does_not_see_do_not_reach_it(H):
    # a sibling branch holds the largest rows that a write stores and rope keys that are NaN; tokens before the
    # window, and the pool's other rows, the worst bytes there are
    p = problem(B=2, Q=6, H=H, lens=[400, 90], seed=33, window=50, sinks=3)
    par = np.array([[-1, 0, 0, 1, 2, -1]] * 2, np.int32)
    p.ki.tree_parent.copy_(i32(par))
    p = dataclasses.replace(p, parent=par)
    out, lse = check_attn(p)
    dirty = p.ki.cache.rows.clone()
    for b, P in enumerate(p.lens):
        mine = set(O.visible(par[b], 3, P, 50, 3))
        anyone = {j for i in range(6) for j in O.visible(par[b], i, P, 50, 3)}
        for j in set(range(P + 6)) - mine:
            dirty[int(p.slots[b][j])] = 0xff
            if j in anyone:
                dirty[int(p.slots[b][j]), :512] = 0x7e
    o2, l2 = run(dataclasses.replace(p.ki, cache=dataclasses.replace(p.ki.cache, rows=dirty)))
    assert torch.equal(out[:, 3], o2[:, 3]) and torch.equal(lse[:, 3], l2[:, 3])


@pytest.mark.parametrize("H", [8, 40])
def test_unused_sequences_are_left_as_they_were(H):
    p = problem(B=4, Q=3, H=H, lens=[-1, 200, -1, 65], seed=34)
    out = torch.full((4, 3, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 3, H), 4.0, device="cuda")
    check_attn(p, out=out, lse=lse)
    assert bool((out[[0, 2]] == 3).all()) and bool((lse[[0, 2]] == 4).all())
    p.ki.prefix_lens.fill_(-1)  # all of them unused
    p.ki.kv_indptr.zero_()
    out.fill_(3)
    run(p.ki, out=out, lse=lse)
    assert bool((out == 3).all())


@pytest.mark.parametrize("H", [3, 45])
@pytest.mark.parametrize("gap", [1, 31, 32, 127, 128, 129, 500])
def test_unused_sequences_between_used_ones(gap, H):
    lens = [70] + [-1] * gap + [5] + [-1] * (2 * gap) + [130] + [-1] * gap
    p = problem(B=len(lens), Q=2, H=H, lens=lens, seed=54)
    out = torch.full((len(lens), 2, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    check_attn(p, out=out)
    assert bool((out[torch.tensor(lens, device="cuda") < 0] == 3).all())


@pytest.mark.parametrize("H", [16, 40])
def test_lse_may_be_null_and_streams_and_repeats_agree(H):
    import ctypes
    p = problem(B=2, Q=8, H=H, lens=[1500, 700], seed=35)
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    out, lse = run(p.ki, workspace=ws)
    o2 = torch.zeros_like(out)
    a = p.ki.c_args(o2, None)
    st = api.load().mla_kv8_attn(ctypes.byref(a), ws.data_ptr(), ws.numel(), api._stream(None))
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(out, o2)
    # two calls at once, each with its own workspace
    ss = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for k in range(6):
        st = ss[k % 2]
        st.wait_stream(torch.cuda.current_stream())
        res.append(api.kv8_attn(p.ki, out=torch.zeros_like(out), lse=torch.zeros_like(lse),
                                workspace=api.alloc_workspace(ws.numel()), stream=st))
    torch.cuda.synchronize()
    for o, l in res:
        assert torch.equal(out, o) and torch.equal(lse, l)


@pytest.mark.parametrize("kw", [
    dict(B=1500, Q=1, H=2, lens=[(7 * i) % 300 - 1 for i in range(1500)], tree="null"),  # more than a block's threads
    dict(B=641, Q=2, H=1, lens=[-1] * 640 + [900], page=16),
    dict(B=641, Q=2, H=64, lens=[-1] * 640 + [900], page=16),
    dict(B=2, Q=3, H=700, lens=[700, 90]),                                  # 17 row groups, the last of 52 rows
    dict(B=700, Q=1, H=1, lens=[0] * 700, tree="null", window=1),
], ids=["1500", "last_of_641", "last_of_641_many", "700_heads", "nothing_but_nodes"])
def test_many_sequences_and_heads(kw):
    check_attn(problem(seed=42, **kw))


def test_queries_and_outputs_beyond_32_bit_offsets():
    # 2 sequences x 4 nodes x 2^20 heads: 4.3 billion elements; some heads of each row of nodes against the oracle
    B, Q, H = 2, 4, 1 << 20
    heads = [0, 127, 128, 524_287, 1_000_003, H - 1]
    p = problem(B=B, Q=Q, H=len(heads), lens=[100, 61], seed=56)
    g = torch.Generator(device="cuda").manual_seed(57)
    q = {n: torch.empty((B, Q, H, w), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
         for n, w in (("q_lat", 512), ("q_pe", 64))}
    for n, t in q.items():
        getattr(p.ki, n).copy_(t[:, :, heads])
    ki = dataclasses.replace(p.ki, H=H, **q)
    ws = api.alloc_workspace(api.kv8_workspace_size(ki))
    out, lse = run(ki, workspace=ws)
    assert api.kv8_check(ws) == 0
    compare(p, out[:, :, heads], lse[:, :, heads])
    assert bool((lse != 0).all()) and bool((out.view(torch.int32) != 0).any(-1).all())


def test_outputs_of_few_rows_beyond_32_bit_offsets():
    # 140,000 sequences of one token x 64 heads: 4.6 billion elements, in the kernel for few rows
    B, H = 140_000, 64
    p = problem(B=2, Q=1, H=H, lens=[0, 3], seed=58, tree="null", page=16)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = 3
    table = torch.zeros((B, p.ki.block_table.shape[1]), dtype=torch.int32, device="cuda")
    table[:] = p.ki.block_table[0].clamp(min=0)
    table[-1] = p.ki.block_table[1]
    q = {n: torch.zeros((B, 1, H, w), dtype=torch.bfloat16, device="cuda") for n, w in (("q_lat", 512), ("q_pe", 64))}
    for n, t in q.items():
        t[0], t[-1] = getattr(p.ki, n)[0], getattr(p.ki, n)[1]
    ki = dataclasses.replace(p.ki, B=B, prefix_lens=lens, block_table=table, **q)
    ws = api.alloc_workspace(api.kv8_workspace_size(ki))
    out, lse = run(ki, workspace=ws)
    assert api.kv8_check(ws) == 0
    compare(p, out[[0, -1]], lse[[0, -1]])
    # one token: its latents whatever the queries
    assert bool((out[:-1] == out[0, 0, 0]).all())


@pytest.mark.parametrize("H", [8, 40])
@pytest.mark.parametrize("page", [2, 3, 8, 24, 33, 64, 127, 1000, 4096, 4097])
def test_page_sizes(page, H):
    check_attn(problem(B=3, Q=3, H=H, lens=[1400, 2 * page - 3, 65], page=page, seed=46, block=page))


@pytest.mark.parametrize("H", [8, 40])
@pytest.mark.parametrize("page", [2 ** 31 - 1, 2 ** 30, 2 ** 30 + 1])
def test_a_page_larger_than_the_pool(page, H):
    # page 0 holds every position: slots are positions; the pool ends inside the page, and inside a tile
    p = problem(B=1, Q=2, H=H, lens=[900], seed=47)
    rows = p.rows.copy()
    rows[rows == 0xff] = 0x30
    p.ki.cache.rows.copy_(torch.from_numpy(rows))
    ki = dataclasses.replace(p.ki, page_size=page, block_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    check_attn(dataclasses.replace(p, ki=ki, rows=rows, slots=[np.arange(902)]))


@pytest.mark.parametrize("H", [10, 40])
def test_arrays_aligned_to_16_bytes_only(H):
    p = problem(B=5, Q=4, H=H, lens=[70, 3000, 0, 513, 64], seed=43)
    out, lse = check_attn(p)

    def moved(t):
        m = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape)
        assert m.data_ptr() % 32 == 16
        return m.copy_(t)
    o2 = moved(torch.zeros_like(out))
    l2 = torch.zeros(lse.numel() + 1, device="cuda")[1:].view(lse.shape)
    run(dataclasses.replace(p.ki, q_lat=moved(p.ki.q_lat), q_pe=moved(p.ki.q_pe)), out=o2, lse=l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("H", [3, 70])
@pytest.mark.parametrize("B", [40, 76, 153, 260])
def test_many_cut_row_groups(B, H):
    # more boundaries inside row groups than a warp counts: every one of them is merged, in every call
    p = problem(B=B, Q=1, H=H, lens=[1000 + (337 * i) % 1000 for i in range(B)], tree="null", seed=41)
    out, lse = check_attn(p)
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    for _ in range(20):
        o2, l2 = run(p.ki, workspace=ws.fill_(0xee))
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("H", [20, 70])
def test_short_pieces_one_after_another(H):
    # one tile to a row group
    p = problem(B=600, Q=1, H=H, lens=[(7 * i) % 60 for i in range(600)], tree="null", seed=39)
    out, lse = check_attn(p)
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    other = torch.randn(1 << 16, device="cuda")
    for i in range(40):  # other kernels in between: the next call's code is not in the caches
        other.sort(), other.cumsum(0), (other[:1024, None] * other[None, :1024]) @ other[:1024]
        o2, l2 = run(p.ki, workspace=ws)
        assert torch.equal(out, o2) and torch.equal(lse, l2), i


@pytest.mark.parametrize("H", [8, 40])
@pytest.mark.parametrize("page", [1, 16])
def test_bad_tables_are_reported(page, H):
    def go(**kw):
        ki = dataclasses.replace(p.ki, **kw)
        ws = api.alloc_workspace(api.kv8_workspace_size(ki))
        out = torch.full((3, 4, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((3, 4, H), 4.0, device="cuda")
        run(ki, out=out, lse=lse, workspace=ws)
        return api.kv8_check(ws), out, lse
    p = problem(B=3, Q=4, H=H, lens=[150, 90, 10], page=page, seed=36)
    good, out0, lse0 = go()
    assert good == 0

    def edit(t, i, v):
        t = t.clone()
        t.view(-1)[i] = v
        return t
    e, out, lse = go(prefix_lens=edit(p.ki.prefix_lens, 1, -2))
    assert e & PREFIX and bool((out == 3).all()) and bool((lse == 4).all())
    if page == 1:
        for i, v in ((0, 1), (1, 155), (3, 300), (2, -7)):
            e, out, lse = go(kv_indptr=edit(p.ki.kv_indptr, i, v))
            assert e == INDPTR and bool((out == 3).all()) and bool((lse == 4).all())
        for v in (-1, -2, -2 ** 31, p.ki.cache.rows.shape[0], 2 ** 31 - 1):
            e, out, lse = go(kv_indices=edit(p.ki.kv_indices, 7, v))  # sequence 0
            assert e == SLOT and torch.equal(out[1:], out0[1:]) and torch.equal(lse[1:], lse0[1:])
    else:
        e, out, lse = go(block_table=p.ki.block_table[:, :9].contiguous())
        assert e == PAGES and bool((out == 3).all())
        for v in (-1, -2, -2 ** 31, p.ki.cache.rows.shape[0] // page, 2 ** 31 - 1):
            e, out, lse = go(block_table=edit(p.ki.block_table, 3, v))
            assert e == SLOT and torch.equal(out[1:], out0[1:]) and torch.equal(lse[1:], lse0[1:])
    for i, v in ((0, 0), (2, 2), (3, -2), (1, 77)):
        e, out, lse = go(tree_parent=edit(p.ki.tree_parent, i, v))
        assert e == PARENT and torch.equal(out[1:], out0[1:]) and torch.equal(lse[1:], lse0[1:])


@pytest.mark.parametrize("H", [4, 70])
def test_scores_of_minus_infinity(H):
    # rope keys of -infinity: tokens without weight, and rows that have no others, whole or cut into pieces
    p = problem(B=4, Q=1, H=H, lens=[3000, 200, 5, 2500], seed=49, tree="null")
    p.ki.q_pe[..., 0] = 1.0
    dead = np.concatenate([p.slots[0], p.slots[1][:150], p.slots[2], p.slots[3][:2490]]).astype(np.int64)
    p.ki.cache.rows[torch.from_numpy(dead).cuda(), 512] = 0x80
    p.ki.cache.rows[torch.from_numpy(dead).cuda(), 513] = 0xff
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    out, lse = run(p.ki, workspace=ws)
    assert api.kv8_check(ws) == 0
    for b in (0, 2):
        assert bool((out[b] == 0).all()), b
        assert bool((lse[b] == -float("inf")).all()), b
    compare(dataclasses.replace(p, lens=[-1, 50, -1, 10],
                                slots=[None, p.slots[1][150:], None, p.slots[3][2490:]]), out, lse)


@pytest.mark.parametrize("page,H", [(1, 3), (64, 3), (64, 70)])
def test_long_prefix(page, H):
    # 200,000 tokens, a head that sees them all alike, an ordinary one and a sharp one
    p = problem(B=1, Q=2, H=H, lens=[200_000], page=page, seed=52, block=64)
    for h, f in ((0, 2.0 ** -8), (2, 4.0)):
        p.ki.q_lat[:, :, h] *= f
        p.ki.q_pe[:, :, h] *= f
    heads = [0, 1, 2, H - 1]
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    out, lse = run(p.ki, workspace=ws)
    assert api.kv8_check(ws) == 0
    few = dataclasses.replace(p.ki, H=4, q_lat=p.ki.q_lat[:, :, heads].contiguous(), q_pe=p.ki.q_pe[:, :, heads].contiguous())
    compare(dataclasses.replace(p, ki=few), out[:, :, heads], lse[:, :, heads])
    # what compare() allows the normaliser for its additions exceeds a tile: against the sums of a wave of partial
    # results a lost tile of 64 would show in the flat head
    lat, rope = O.unpack_rows(p.rows[p.slots[0]], p.k[p.slots[0]], -6)
    for i in range(2):
        pos = O.visible(p.parent[0], i, 200_000)
        q = p.ki.q_lat[0, i, 0].double().cpu().numpy(), p.ki.q_pe[0, i, 0].double().cpu().numpy()
        want = np.log(np.exp(p.ki.scale * (lat[pos] @ q[0] + rope[pos] @ q[1])).sum())
        assert abs(float(lse[0, i, 0]) - want) <= 64 / 200_000 / 2


@pytest.mark.parametrize("kw", [
    dict(B=2, Q=16, H=64, lens=[900, 2100]),
    dict(B=1, Q=1, H=16, lens=[0], tree="null"),
    dict(B=1, Q=1, H=128, lens=[200], tree="null"),
    dict(B=300, Q=1, H=20, lens=[(7 * i) % 60 for i in range(300)], tree="null"),
    dict(B=8, Q=2, H=30, lens=[3000] * 8),
], ids=["groups", "one_tile", "four_tiles", "short_pieces", "few_rows"])
def test_timeout_is_reported_and_the_context_recovers(kw):
    p = problem(seed=53, **kw)
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    out, lse = run(p.ki)
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    for _ in range(2):
        t0 = time.monotonic()
        api.kv8_selftest_timeout(p.ki, o2, l2, ws, hold_ns=20_000_000)
        assert api.kv8_check(ws) == TIMEOUT
        assert time.monotonic() - t0 < 10
        o3, l3 = run(p.ki, workspace=ws)
        assert api.kv8_check(ws) == 0
        assert torch.equal(out, o3) and torch.equal(lse, l3)
    compare(p, out, lse)


@pytest.mark.parametrize("H", [16, 40])
def test_captured_call_follows_its_inputs(H):
    p = problem(B=3, Q=4, H=H, lens=[900, 300, 64], page=16, seed=37, window=128, sinks=5)
    rows = p.rows.copy()
    rows[rows == 0xff] = 0x30  # every page is used below
    p.ki.cache.rows.copy_(torch.from_numpy(rows))
    p = dataclasses.replace(p, rows=rows)
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    out, lse = torch.zeros((3, 4, H, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 4, H), device="cuda")
    run(p.ki, out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.kv8_attn(p.ki, out=out, lse=lse, workspace=ws, check=False)
    for lens in ([900, 300, 64], [40, 299, 65], [-1, 0, 500], [700, -1, 1]):
        p.ki.prefix_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        p.ki.block_table.copy_(torch.arange(p.ki.block_table.numel(), device="cuda").view_as(p.ki.block_table)
                               % (p.ki.cache.rows.shape[0] // 16))
        tab = p.ki.block_table.cpu().numpy()
        slots = [tab[b, np.arange(max(0, v + 4)) // 16].astype(np.int64) * 16 + np.arange(max(0, v + 4)) % 16
                 for b, v in enumerate(lens)]
        g.replay()
        torch.cuda.synchronize()
        assert api.kv8_check(ws) == 0
        compare(dataclasses.replace(p, slots=slots, lens=lens), out, lse)


@pytest.mark.parametrize("H", [16, 70])
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_calls_that_follow_each_other_see_each_other(captured, H):
    # rows written (and blocks grown), attended to, read back and written over, one call right behind the other
    p = problem(B=6, Q=4, H=H, lens=[700, 90, 1300, 5, 64, 250], seed=44)
    n = sum(v + 4 for v in p.lens)
    at = p.ki.kv_indices[:n].contiguous()
    both = [latents("normal", n, torch.bfloat16, 45 + i, -6) for i in range(2)]
    both = [(t.cuda() * 4.0 ** i, k.cuda()) for i, (t, k) in enumerate(both)]
    first_rows, first_words = p.ki.cache.rows.clone(), p.ki.cache.scales.clone()
    few = at[:100].contiguous()
    ws = api.alloc_workspace(api.kv8_workspace_size(p.ki))
    ws2 = api.alloc_workspace(api.KV8_WORKSPACE_BYTES)

    def buffers():
        return (torch.zeros((6, 4, H, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((6, 4, H), device="cuda"),
                torch.zeros((n, 512), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda"))

    def step(i, o, sync):
        def s():
            if sync:
                torch.cuda.synchronize()
        if i == 0:  # the cache as it was, with small scales
            p.ki.cache.rows.copy_(first_rows)
            p.ki.cache.scales.copy_(first_words)
            s()
        api.kv8_write(p.ki.cache, *both[i], at, workspace=ws2, check=False)
        s()
        api.kv8_write(p.ki.cache, both[i][0][:100] * 2, both[i][1][:100], few, workspace=ws2, check=False)
        s()
        api.kv8_attn(p.ki, out=o[0], lse=o[1], workspace=ws, check=False)
        s()
        api.kv8_read(p.ki.cache, at, kv_c=o[2], k_pe=o[3], workspace=ws2, check=False)
        s()
    want = [buffers() for _ in range(2)]
    for i in range(2):
        step(i, want[i], True)
    got = [buffers() for _ in range(20)]
    torch.cuda.synchronize()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for i, o in enumerate(got):
                step(i % 2, o, False)
        g.replay()
    else:
        for i, o in enumerate(got):
            step(i % 2, o, False)
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for a, b in zip(o, want[i % 2]):
            assert torch.equal(a, b), i


def test_arrays_made_by_a_call_on_another_stream():
    p = problem(B=4, Q=3, H=8, lens=[-1, 200, 900, 65], seed=38)
    out, lse = run(p.ki)
    at = i32([5, -1, 3])
    p.ki.cache.rows[[5, 3]] = 0x31
    c0, k0, _ = api.kv8_read(p.ki.cache, at)
    out, lse = run(p.ki)
    big = torch.randn(6000, 6000, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        big @ big
        o2, l2 = api.kv8_attn(p.ki, stream=s)
        c, k, ws = api.kv8_read(p.ki.cache, at, stream=s)
        junk = [torch.full((1 << 20,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(40)]
        s.synchronize()
        got = [t.cpu() for t in (o2, l2, c, k)]
        assert api.kv8_check(ws, s) == 0
        del junk
        for a, b in zip(got, (out, lse, c0, k0)):
            assert torch.equal(a, b.cpu())
