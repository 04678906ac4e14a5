"""The 4-bit latent cache on the GPU: written rows and read-back bit for bit,
the attention against the float64 oracle, masks, tables, streams and graphs.

Tolerance of the attention (derived, per element).  Keys and values enter the
products exactly and everything accumulates in fp32, so against float64:
  * a score is off by at most (576 + 8) * 2^-24 * sum |q||k| * scale  =: ds
    (576 additions, the exponent's scaling and the argument of exp);
  * a weight by a factor 1 +- (2 ds + 2^-21): numerator and normaliser, and the
    hardware exponential's 2^-22 in each; rounding it to f16 adds 2^-11, and
    2^-31 of the row's largest weight where it falls below f16's normal range;
  * the sums over n tokens by n * 2^-24 of the sums of magnitudes;
  * the result's rounding to bf16 by 2^-8 of the value.
lse: ds + 2^-21 + n * 2^-24 from the normaliser, and fp32 rounding 2^-22 |lse|.
"""
import dataclasses
import time

import numpy as np
import pytest

from mla_tree_verify_absorbed_gb300 import api
from oracle import kvq as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SLOT, NONFINITE, PREFIX, INDPTR, PARENT, PAGES, TIMEOUT = 0x4, 0x200, 0x1, 0x2, 0x8, 0x10, 0x40


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def bits_of(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
def latents(kind, n, dtype, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, 512))
    if kind == "gain":
        x *= np.exp(2.0 * r.standard_normal(512))
    elif kind == "ties":  # every value a tie point of its block's scale, with the block's maximum at 7 scales
        s = O.SCALES[r.integers(8, 127, (n, 32))].repeat(16, 1)
        x = r.integers(-13, 14, (n, 512)) / 2 * s
        x[:, ::16] = 7 * s[:, ::16]
    elif kind == "scale_ties":  # block maxima half way between two scales, times 7
        b = r.integers(0, 126, (n, 32))
        mid = (O.SCALES[b] + O.SCALES[b + 1]) / 2
        x = r.uniform(-1, 1, (n, 512)) * (7 * mid).repeat(16, 1)
        x[:, 5::16] = -7 * mid
    elif kind == "tiny":
        x *= 2.0 ** r.integers(-14, -4, (n, 1))
    elif kind == "huge":
        x *= 2.0 ** r.integers(8, 100, (n, 1))
    elif kind == "zeros":
        x[:, :256] = 0
        x[0] = -0.0
    t = torch.from_numpy(x).to(torch.float32).to(dtype)
    k = torch.from_numpy(r.standard_normal((n, 64))).to(torch.float32).to(dtype)
    return t, k


def packed(t, k, exponent):
    kb = k.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    return np.stack([O.pack_row(a, b, exponent) for a, b in zip(t.double().numpy(), kb)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind,exponent", [("normal", 0), ("gain", 0), ("gain", 3), ("gain", -32), ("gain", 32),
                                           ("ties", 0), ("scale_ties", 0), ("tiny", 0), ("tiny", -7), ("huge", 0),
                                           ("huge", 32), ("huge", -32), ("zeros", 1)])
def test_write_is_the_oracles_bytes(kind, exponent, dtype):
    n, slots = 19, 40
    t, k = latents(kind, n, dtype, 11)
    want = np.full((slots, 416), 0xab, np.uint8)
    at = np.random.default_rng(5).permutation(slots)[:n].astype(np.int32)
    at[3] = at[n - 1] = -1
    keep = at >= 0
    want[at[keep]] = packed(t, k, exponent)[keep]
    cache = api.QuantCache(torch.full((slots, 416), 0xab, dtype=torch.uint8, device="cuda"), exponent)
    sl = torch.from_numpy(at).cuda()
    ws = api.kvq_write(cache, t.cuda(), k.cuda(), sl)
    assert api.kvq_check(ws) == 0
    got = cache.rows.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    # and back: exactly what the bytes stand for; skipped rows keep their values
    for name, dt in (("bf16", torch.bfloat16), ("fp32", torch.float32)):
        c0, r0 = torch.full((n, 512), 5.0, dtype=dt).cuda(), torch.full((n, 64), 6.0, dtype=dt).cuda()
        c, r, ws = api.kvq_read(cache, sl, kv_c=c0, k_pe=r0)
        assert api.kvq_check(ws) == 0
        lat, rope = O.unpack_rows(want[at[keep]], exponent)
        assert np.array_equal(c.double().cpu().numpy()[keep], lat)
        assert np.array_equal(r.double().cpu().numpy()[keep], rope)
        assert (c.float().cpu().numpy()[~keep] == 5).all() and (r.float().cpu().numpy()[~keep] == 6).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 2, 7, 64, 2433, 2434, 40011])
def test_rows_of_any_count_with_strides(n, dtype):
    # one wide array holds kv_c and k_pe; cache rows 448 bytes apart; more rows than warps
    t, k = latents("normal", min(n, 50), dtype, 12)
    rep = -(-n // 50)
    wide = torch.full((n, 704), 9.0, dtype=dtype)
    wide[:, :512] = t.repeat(rep, 1)[:n]
    wide[:, 640:] = k.repeat(rep, 1)[:n]
    wide = wide.cuda()
    pool = torch.full((n + 3, 448), 7, dtype=torch.uint8, device="cuda")
    cache = api.QuantCache(pool[:, :416])
    sl = torch.randperm(n + 3, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32).cuda()
    ws = api.kvq_write(cache, wide[:, :512], wide[:, 640:], sl)
    assert api.kvq_check(ws) == 0
    want = torch.from_numpy(packed(t, k, 0)).repeat(rep, 1)[:n]
    assert torch.equal(pool[sl.long(), :416].cpu(), want)
    assert bool((pool[:, 416:] == 7).all())
    rest = torch.ones(n + 3, dtype=torch.bool)
    rest[sl.long().cpu()] = False
    assert bool((pool[rest.cuda()] == 7).all())
    back = torch.full((n, 704), 3.0, dtype=dtype, device="cuda")
    api.kvq_read(cache, sl, kv_c=back[:, :512], k_pe=back[:, 640:])
    lat, rope = O.unpack_rows(want[:50].numpy())
    assert torch.equal(back[:, :512].double().cpu(), torch.from_numpy(lat).repeat(rep, 1)[:n])
    assert torch.equal(back[:, 640:].double().cpu(), torch.from_numpy(rope).repeat(rep, 1)[:n])
    assert bool((back[:, 512:640] == 3).all())


@pytest.mark.parametrize("exponent", [0, -32, 32, 5])
def test_read_of_any_bytes(exponent):
    rng = np.random.default_rng(2)
    rows = rng.integers(0, 256, (300, 416), dtype=np.uint8)
    rows[:, 289::2] &= 0xbf  # rope keys without NaN, which would not compare
    rows[0, 256:288] = 0x7f
    rows[1, 256:288] = 0xff
    cache = api.QuantCache(torch.from_numpy(rows).cuda(), exponent)
    at = rng.integers(0, 300, 500).astype(np.int32)  # slots named several times
    lat, rope = O.unpack_rows(rows[at], exponent)
    for name in ("bf16", "fp32"):
        c, r, ws = api.kvq_read(cache, torch.from_numpy(at).cuda(), name)
        assert api.kvq_check(ws) == 0
        assert np.array_equal(c.double().cpu().numpy(), lat)
        assert np.array_equal(r.double().cpu().numpy(), rope)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_write_of_infinities_and_nan(dtype):
    t, k = latents("normal", 4, dtype, 13)
    t[1, 20], t[1, 40], t[2, 511], t[2, 500] = float("inf"), float("nan"), float("-inf"), float("nan")
    k[3, 7], k[3, 8] = float("nan"), float("inf")
    cache = api.kvq_alloc(4)
    ws = api.kvq_write(cache, t.cuda(), k.cuda(), torch.arange(4, dtype=torch.int32).cuda())
    assert api.kvq_check(ws) == NONFINITE
    got, want = cache.rows.cpu().numpy(), packed(t, k, 0)
    assert np.array_equal(got[:, :288], want[:, :288])
    assert np.array_equal(got[:3], want[:3])
    c, r, _ = api.kvq_read(cache, torch.arange(4, dtype=torch.int32).cuda(), "fp32")
    assert float(c[1, 20]) == 7 * 448 and float(c[1, 40]) == 0 and float(c[2, 511]) == -7 * 448
    assert bool(torch.isnan(r[3, 7])) and float(r[3, 8]) == float("inf")
    # only rope keys are not finite: no error
    ws = api.kvq_write(cache, t[3:].cuda(), k[3:].cuda(), torch.zeros(1, dtype=torch.int32).cuda())
    assert api.kvq_check(ws) == 0


def test_slots_outside_the_pool():
    t, k = latents("normal", 5, torch.bfloat16, 14)
    pool = torch.full((12, 416), 1, dtype=torch.uint8, device="cuda")
    cache = api.QuantCache(pool[2:10])
    at = torch.tensor([3, 8, -2, 0, 2 ** 31 - 1], dtype=torch.int32).cuda()
    ws = api.kvq_write(cache, t.cuda(), k.cuda(), at)
    assert api.kvq_check(ws) == SLOT
    want = np.full((12, 416), 1, np.uint8)
    want[[5, 2]] = packed(t, k, 0)[[0, 3]]
    assert np.array_equal(pool.cpu().numpy(), want)
    c = torch.full((5, 512), 2.0, device="cuda")
    r = torch.full((5, 64), 2.0, device="cuda")
    _, _, ws = api.kvq_read(cache, at, kv_c=c, k_pe=r)
    assert api.kvq_check(ws) == SLOT
    assert bool((c[[1, 2, 4]] == 2).all()) and bool((r[[1, 2, 4]] == 2).all())
    assert np.array_equal(c[[0, 3]].double().cpu().numpy(), O.unpack_rows(want[[5, 2]])[0])
    # the next call on the workspace starts without the error
    api.kvq_read(cache, torch.zeros(5, dtype=torch.int32).cuda(), kv_c=c, k_pe=r, workspace=ws)
    assert api.kvq_check(ws) == 0


def test_rows_beyond_32_bit_offsets():
    # slot 11,000,000 lies 4.6 GB into the pool
    n = 11_000_001
    rows = torch.empty((n, 416), dtype=torch.uint8, device="cuda")
    cache = api.QuantCache(rows)
    t, k = latents("normal", 3, torch.bfloat16, 15)
    at = torch.tensor([n - 1, 5_200_000, 0], dtype=torch.int32).cuda()
    api.kvq_write(cache, t.cuda(), k.cuda(), at)
    want = packed(t, k, 0)
    assert np.array_equal(rows[at.long()].cpu().numpy(), want)
    c, _, ws = api.kvq_read(cache, at, "fp32")
    assert api.kvq_check(ws) == 0
    assert np.array_equal(c.double().cpu().numpy(), O.unpack_rows(want)[0])
    # the attention reads the same rows
    p = problem(B=1, Q=1, H=4, lens=[2], seed=3)
    ki = dataclasses.replace(p.ki, cache=cache, kv_indices=at,
                             kv_indptr=torch.tensor([0, 3], dtype=torch.int32).cuda())
    check_attn(dataclasses.replace(p, ki=ki, rows=want, slots=[np.arange(3)]))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
@dataclasses.dataclass
class Prob:
    ki: object
    rows: np.ndarray        # host copy of the cache
    slots: list             # per sequence: pool slot of each position
    lens: list
    parent: np.ndarray


def random_rows(n, seed, sharp=1.0):
    r = np.random.default_rng(seed)
    rows = r.integers(0, 256, (n, 416), dtype=np.uint8)
    rows[:, 256:288] = r.integers(0x20, 0x34, (n, 32))  # scales 1/8 .. 0.7
    rope = torch.from_numpy(sharp * r.standard_normal((n, 64))).to(torch.bfloat16)
    rows[:, 288:] = rope.view(torch.int16).numpy().view(np.uint8)
    return rows


def random_parents(B, Q, seed, kind="tree"):
    r = np.random.default_rng(seed)
    par = np.zeros((B, Q), np.int32)
    for b in range(B):
        for i in range(Q):
            par[b, i] = i - 1 if kind == "chain" else r.integers(-1, i) if kind == "forest" else r.integers(0, max(i, 1))
        par[b, 0] = -1
    return par


def problem(B=1, Q=4, H=8, lens=None, page=1, seed=0, tree="tree", window=0, sinks=0, exponent=0, q_scale=1.0,
            scale=0.0721688, stride=416, freed=False):
    r = np.random.default_rng(seed)
    need = [0 if v < 0 else v + Q for v in lens]
    slots = []
    kw = {}
    if page == 1:
        pool = sum(need) + 9
        idx = r.permutation(pool)[:sum(need)].astype(np.int32)
        ptr = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
        slots = [idx[ptr[b]:ptr[b + 1]].copy() for b in range(B)]
        table = idx
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
    rows = random_rows(pool, seed + 1)
    buf = torch.zeros((pool, stride), dtype=torch.uint8)
    buf[:, :416] = torch.from_numpy(rows)
    buf = buf.cuda()
    parent = random_parents(B, Q, seed + 2, tree)
    q = torch.from_numpy(q_scale * r.standard_normal((B, Q, H, 576))).to(torch.bfloat16)
    if page == 1:
        kw = dict(kv_indptr=torch.from_numpy(ptr).cuda(), kv_indices=torch.from_numpy(table).cuda())
    else:
        kw = dict(block_table=torch.from_numpy(table).cuda())
    ki = api.KvqInputs(B=B, Q=Q, H=H, scale=scale, q_lat=q[..., :512].contiguous().cuda(),
                       q_pe=q[..., 512:].contiguous().cuda(), cache=api.QuantCache(buf[:, :416], exponent),
                       prefix_lens=torch.tensor(lens, dtype=torch.int32).cuda(), page_size=page,
                       tree_parent=None if tree == "null" else torch.from_numpy(parent).cuda(), window=window,
                       sinks=sinks, **kw)
    if tree == "null":
        parent = random_parents(B, Q, 0, "chain")
    return Prob(ki, rows, slots, list(lens), parent)


def run(ki, **kw):
    out, lse = api.kvq_attn(ki, **kw)
    torch.cuda.synchronize()
    return out, lse


def compare(p, out, lse):
    ki = p.ki
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, P in enumerate(p.lens):
        if P < 0:
            continue
        lat, rope = O.unpack_rows(p.rows[p.slots[b]], ki.cache.exponent)
        o, l, mag, smag = O.attention(lat, rope, ki.q_lat[b].double().cpu().numpy(), ki.q_pe[b].double().cpu().numpy(),
                                      ki.scale, p.parent[b], P, ki.H, ki.window, ki.sinks)
        n = P + ki.Q
        ds = 584 * 2.0 ** -24 * smag
        dw = np.expm1(2 * ds + 2.0 ** -21) + 2.0 ** -11 + n * 2.0 ** -24
        top = np.abs(lat).max() * n * 2.0 ** -31  # weights below f16's normal range
        tol = 2.0 ** -8 * np.abs(o) + 1.01 * dw[..., None] * mag + top
        bad = np.abs(out[b] - o) > tol
        assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(out[b] - o).max(), tol.min())
        ltol = ds + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(l)
        bad = np.abs(lse[b] - l) > ltol
        assert not bad.any(), (b, np.argwhere(bad)[:4], np.abs(lse[b] - l).max(), ltol.min())


def check_attn(p, **kw):
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    ws.fill_(0xee)  # a workspace needs no clearing
    out, lse = run(p.ki, workspace=ws, **kw)
    assert api.kvq_check(ws) == 0
    compare(p, out, lse)
    return out, lse


# shapes with one thing out of the ordinary each: lengths of 0 and 1, tile and
# page borders, head counts around the row groups, odd everything
SHAPES = [
    dict(B=1, Q=1, H=1, lens=[0]),
    dict(B=1, Q=1, H=16, lens=[1]),
    dict(B=1, Q=1, H=128, lens=[62], tree="null"),
    dict(B=1, Q=1, H=128, lens=[63], tree="null"),
    dict(B=1, Q=1, H=129, lens=[64], tree="null"),
    dict(B=1, Q=2, H=64, lens=[127]),
    dict(B=1, Q=3, H=43, lens=[128]),
    dict(B=1, Q=64, H=5, lens=[0], tree="forest"),
    dict(B=2, Q=64, H=16, lens=[301, 0], tree="tree"),
    dict(B=3, Q=8, H=16, lens=[700, 0, 1500], tree="forest"),
    dict(B=3, Q=5, H=7, lens=[33, 3000, 1], page=16),
    dict(B=2, Q=17, H=3, lens=[999, 65], page=100, tree="null"),
    dict(B=4, Q=1, H=16, lens=[5, -1, 257, -1], page=64, tree="null"),
    dict(B=5, Q=3, H=9, lens=[-1, 60, -1, 61, 62], tree="chain"),
    dict(B=1, Q=4, H=64, lens=[2900], stride=448),
    dict(B=70, Q=1, H=2, lens=[(37 * i) % 400 for i in range(70)], tree="null"),
    dict(B=1, Q=64, H=64, lens=[130], tree="chain"),
    dict(B=1, Q=7, H=8, lens=[2000], page=1 << 20),
]


@pytest.mark.parametrize("kw", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
def test_attention_matches_oracle(kw):
    check_attn(problem(seed=21, **kw))


@pytest.mark.parametrize("exponent", [-32, -5, 7, 32])
def test_attention_exponent(exponent):
    # the latent part of the scores scales by 2^exponent: a scale that keeps them moderate
    p = problem(B=2, Q=3, H=8, lens=[200, 77], seed=22, exponent=exponent, scale=0.07 * 2.0 ** -max(exponent, 0))
    check_attn(p)


@pytest.mark.parametrize("scale,q_scale", [(1e-6, 1.0), (1.0, 1.0), (8.0, 3.0), (0.07, 100.0)])
def test_attention_flat_and_sharp(scale, q_scale):
    # flat: a mean over all rows; sharp: the running maximum moves over thousands
    check_attn(problem(B=2, Q=4, H=8, lens=[1500, 300], seed=23, scale=scale, q_scale=q_scale))


def test_rising_maximum():
    # keys sorted by their score against one head's query: its maximum rises with every tile, another's falls
    p = problem(B=1, Q=1, H=2, lens=[1600], seed=24, tree="null", q_scale=2.0)
    lat, rope = O.unpack_rows(p.rows)
    q = p.ki.q_lat[0, 0, 0].double().cpu().numpy()
    p.ki.q_lat[0, 0, 1] = -p.ki.q_lat[0, 0, 0]
    p.ki.q_pe[0, 0, 1] = -p.ki.q_pe[0, 0, 0]
    s = lat[p.slots[0]] @ q + rope[p.slots[0]] @ p.ki.q_pe[0, 0, 0].double().cpu().numpy()
    order = np.argsort(s)
    p.slots[0] = p.slots[0][order]
    p.ki.kv_indices.copy_(torch.from_numpy(p.slots[0].astype(np.int32)))
    check_attn(p)


@pytest.mark.parametrize("rows", [129, 150, 198, 225, 1, 33])
def test_row_groups_with_few_rows_between_full_ones(rows):
    # many sequences of one or two row groups, the last of them a fraction of 128 rows, so that a cluster's pieces
    # alternate between groups that use all rows and groups that leave most out
    n = 24
    check_attn(problem(B=n, Q=1, H=rows, lens=[(97 * i) % 700 for i in range(n)], page=16, seed=25, tree="null"))


WINDOWS = [
    dict(B=1, Q=1, H=4, lens=[500], window=1, sinks=0),
    dict(B=1, Q=1, H=4, lens=[500], window=1, sinks=1),
    dict(B=1, Q=1, H=16, lens=[500], window=64, sinks=4),
    dict(B=1, Q=1, H=16, lens=[511], window=65, sinks=64),
    dict(B=2, Q=8, H=8, lens=[900, 30], window=100, sinks=70, tree="tree"),
    dict(B=2, Q=64, H=4, lens=[777, 5], window=9, sinks=7, tree="chain"),
    dict(B=2, Q=64, H=4, lens=[777, 5], window=9, sinks=40, tree="null"),
    dict(B=1, Q=64, H=3, lens=[0], window=5, sinks=20, tree="forest"),
    dict(B=3, Q=5, H=8, lens=[1000, 1000, 63], window=1 << 30, sinks=3, tree="forest"),
    dict(B=3, Q=5, H=8, lens=[1000, 100, 63], window=333, sinks=1 << 30, tree="forest"),
    dict(B=4, Q=2, H=8, lens=[2000, -1, 64, 640], window=130, sinks=66, page=16, tree="null"),
    dict(B=2, Q=33, H=6, lens=[1999, 450], window=200, sinks=129, page=48, tree="tree"),
]


@pytest.mark.parametrize("freed", [False, True], ids=["tables", "freed"])
@pytest.mark.parametrize("kw", WINDOWS, ids=[f"{i}" for i in range(len(WINDOWS))])
def test_window_and_sinks_match_oracle(kw, freed):
    check_attn(problem(seed=31, freed=freed, **kw))


@pytest.mark.parametrize("seed", range(8))
def test_maximum_moves_after_a_few_first_tokens(seed):
    # the first tile of the row group shows 4 tokens, so the next ones move the maxima of most rows, at tiles
    # that differ from warp to warp, in pieces of a few tiles: the oracle's values, and the same bytes every time
    B = 1 + seed % 2
    p = problem(B=B, Q=1, H=64, lens=[60000 + 1000 * seed, 9000][:B], seed=40 + seed, window=4096 - 60 * seed,
                sinks=4, page=64, tree="null", freed=True)
    n = len(p.rows)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 576, generator=g)
    x[:, :512] *= torch.exp(0.4 * torch.randn(512, generator=g))
    x = x.to(torch.bfloat16).cuda()
    api.kvq_write(p.ki.cache, x[:, :512], x[:, 512:], torch.arange(n, dtype=torch.int32).cuda())
    p = dataclasses.replace(p, rows=p.ki.cache.rows.cpu().numpy())
    out, lse = check_attn(p)
    for _ in range(10):
        o, l = run(p.ki)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("tiles", range(2, 13))
def test_some_rows_maxima_move_at_every_tile_and_others_never(tiles):
    # heads 32-63 meet their keys in rising order, far apart; heads 0-31 see flat scores
    p = problem(B=1, Q=1, H=64, lens=[64 * tiles - 1], seed=60, tree="null")
    p.ki.q_lat[0, 0, 32:] = p.ki.q_lat[0, 0, 32].clone() * 16
    p.ki.q_pe[0, 0, 32:] = p.ki.q_pe[0, 0, 32].clone() * 16
    p.ki.q_lat[0, 0, :32] *= 2.0 ** -6
    p.ki.q_pe[0, 0, :32] *= 2.0 ** -6
    lat, rope = O.unpack_rows(p.rows)
    s = lat[p.slots[0]] @ p.ki.q_lat[0, 0, 32].double().cpu().numpy() \
        + rope[p.slots[0]] @ p.ki.q_pe[0, 0, 32].double().cpu().numpy()
    p.slots[0] = p.slots[0][np.argsort(s)]
    p.ki.kv_indices.copy_(torch.from_numpy(p.slots[0].astype(np.int32)))
    for _ in range(3):
        check_attn(p)


def test_window_that_covers_everything_changes_nothing():
    p = problem(B=2, Q=6, H=8, lens=[333, 70], seed=32)
    out, lse = run(p.ki)
    o2, l2 = run(dataclasses.replace(p.ki, window=400, sinks=2))
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_rows_that_a_node_does_not_see_do_not_reach_it():
    # a sibling branch, tokens before the window and the pool's other rows hold the worst bytes there are
    p = problem(B=2, Q=6, H=16, lens=[400, 90], seed=33, window=50, sinks=3)
    par = np.array([[-1, 0, 0, 1, 2, -1]] * 2, np.int32)
    p.ki.tree_parent.copy_(torch.from_numpy(par))
    p = dataclasses.replace(p, parent=par)
    out, lse = check_attn(p)
    dirty = p.ki.cache.rows.clone()
    used = torch.zeros(dirty.shape[0], dtype=torch.bool, device="cuda")
    for b, P in enumerate(p.lens):
        pos = [j for i in (3,) for j in O.visible(par[b], i, P, 50, 3)]
        used[torch.from_numpy(p.slots[b][pos].astype(np.int64)).cuda()] = True
    dirty[~used] = 0xff  # scale 0x7f, code 15, rope NaN
    o2, l2 = run(dataclasses.replace(p.ki, cache=api.QuantCache(dirty)))
    assert torch.equal(out[:, 3], o2[:, 3]) and torch.equal(lse[:, 3], l2[:, 3])


def test_unused_sequences_are_left_as_they_were():
    p = problem(B=4, Q=3, H=8, lens=[-1, 200, -1, 65], seed=34)
    out = torch.full((4, 3, 8, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 3, 8), 4.0, device="cuda")
    check_attn(p, out=out, lse=lse)
    assert bool((out[[0, 2]] == 3).all()) and bool((lse[[0, 2]] == 4).all())
    # all of them unused
    p.ki.prefix_lens.fill_(-1)
    p.ki.kv_indptr.zero_()
    out.fill_(3)
    run(p.ki, out=out, lse=lse)
    assert bool((out == 3).all())


@pytest.mark.parametrize("gap", [1, 2, 31, 32, 33, 127, 128, 129, 130, 500])
def test_unused_sequences_between_used_ones(gap):
    # three short sequences of one cluster, the gaps of every length around the scheduler's steps, and some behind
    lens = [70] + [-1] * gap + [5] + [-1] * (2 * gap) + [130] + [-1] * gap
    p = problem(B=len(lens), Q=2, H=3, lens=lens, seed=54)
    out = torch.full((len(lens), 2, 3, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    check_attn(p, out=out)
    assert bool((out[torch.tensor(lens, device="cuda") < 0] == 3).all())


def test_many_unused_sequences_between_used_ones():
    # one after the other, 14 million would outlast the two seconds that a wait may take
    B = 14_000_000
    lens = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    lens[0], lens[-1] = 70, 9
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")  # page 0 holds every position
    p = problem(B=2, Q=1, H=1, lens=[70, 9], seed=55, tree="null")
    big = {n: torch.zeros((B, 1, 1, w), dtype=torch.bfloat16, device="cuda") for n, w in (("q_lat", 512), ("q_pe", 64))}
    for n, t in big.items():
        t[[0, -1]] = getattr(p.ki, n)
    ki = dataclasses.replace(p.ki, B=B, prefix_lens=lens, page_size=1 << 20, block_table=table, **big)
    ws = api.alloc_workspace(api.kvq_workspace_size(ki))
    out, lse = run(ki, workspace=ws)
    assert api.kvq_check(ws) == 0
    compare(dataclasses.replace(p, slots=[np.arange(71), np.arange(10)]), out[[0, -1]], lse[[0, -1]])
    assert not bool(out[1:-1].any()) and not bool(lse[1:-1].any())


def test_lse_may_be_null_and_streams_and_repeats_agree():
    p = problem(B=2, Q=8, H=16, lens=[1500, 700], seed=35)
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    out, lse = run(p.ki, workspace=ws)
    o2 = torch.zeros_like(out)
    import ctypes
    a = p.ki.c_args(o2, None)
    st = api.load().mla_kvq_attn(ctypes.byref(a), ws.data_ptr(), ws.numel(), api._stream(None))
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(out, o2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o3, l3 = api.kvq_attn(p.ki, out=torch.zeros_like(out), lse=torch.zeros_like(lse), workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    # two calls at once, each with its own workspace
    ss = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for k in range(6):
        st = ss[k % 2]
        st.wait_stream(torch.cuda.current_stream())
        res.append(api.kvq_attn(p.ki, out=torch.zeros_like(out), lse=torch.zeros_like(lse),
                                workspace=api.alloc_workspace(ws.numel()), stream=st))
    torch.cuda.synchronize()
    for o, l in res:
        assert torch.equal(out, o) and torch.equal(lse, l)


@pytest.mark.parametrize("kw", [
    dict(B=1500, Q=1, H=2, lens=[(7 * i) % 300 - 1 for i in range(1500)], tree="null"),  # more than a block's threads
    dict(B=641, Q=2, H=1, lens=[-1] * 640 + [900], page=16),
    dict(B=2, Q=3, H=700, lens=[700, 90]),                                               # 17 row groups, the last of 52 rows
    dict(B=700, Q=1, H=1, lens=[0] * 700, tree="null", window=1),
], ids=["1500", "last_of_641", "700_heads", "nothing_but_nodes"])
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
    ws = api.alloc_workspace(api.kvq_workspace_size(ki))
    out, lse = run(ki, workspace=ws)
    assert api.kvq_check(ws) == 0
    compare(p, out[:, :, heads], lse[:, :, heads])
    # every row was written: weights sum to one, so no row of these latents is zeros, and no lse is 0
    assert bool((lse != 0).all()) and bool((out.view(torch.int32) != 0).any(-1).all())


@pytest.mark.parametrize("page", [2, 3, 7, 33, 127, 1000, 4097])
def test_page_sizes(page):
    check_attn(problem(B=3, Q=3, H=8, lens=[1400, 2 * page - 3 if page > 1 else 0, 65], page=page, seed=46))


@pytest.mark.parametrize("page", [2 ** 31 - 1, 2 ** 30, 2 ** 30 + 1])
def test_a_page_larger_than_the_pool(page):
    # page 0 holds every position: slots are positions
    p = problem(B=1, Q=2, H=8, lens=[900], seed=47)
    ki = dataclasses.replace(p.ki, page_size=page, block_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    check_attn(dataclasses.replace(p, ki=ki, slots=[np.arange(902)]))


def test_arrays_aligned_to_16_bytes_only():
    # whole row groups, cut ones, and queries and outputs whose rows do not fall on sectors
    p = problem(B=5, Q=4, H=40, lens=[70, 3000, 0, 513, 64], seed=43)
    out, lse = check_attn(p)

    def moved(t):
        m = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape)
        assert m.data_ptr() % 32 == 16
        return m.copy_(t)
    o2 = moved(torch.zeros_like(out))
    l2 = torch.zeros(lse.numel() + 1, device="cuda")[1:].view(lse.shape)
    run(dataclasses.replace(p.ki, q_lat=moved(p.ki.q_lat), q_pe=moved(p.ki.q_pe)), out=o2, lse=l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("B", [40, 61, 76, 130])
def test_many_cut_row_groups(B):
    # more boundaries inside row groups than a warp counts: every one of them is merged, in every call
    p = problem(B=B, Q=1, H=3, lens=[1000 + (337 * i) % 1000 for i in range(B)], tree="null", seed=41)
    out, lse = check_attn(p)
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    for _ in range(20):
        o2, l2 = run(p.ki, workspace=ws.fill_(0xee))
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_arrays_made_by_a_call_on_another_stream():
    # the current stream is kept busy: a fill or a reuse of the memory on it would come at another time
    p = problem(B=4, Q=3, H=8, lens=[-1, 200, 900, 65], seed=38)
    out, lse = run(p.ki)
    at = torch.tensor([5, -1, 3], dtype=torch.int32).cuda()
    c0, k0, _ = api.kvq_read(p.ki.cache, at)
    big = torch.randn(6000, 6000, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        big @ big
        o2, l2 = api.kvq_attn(p.ki, stream=s)
        c, k, ws = api.kvq_read(p.ki.cache, at, stream=s)
        junk = [torch.full((1 << 20,), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(40)]
        s.synchronize()
        got = [t.cpu() for t in (o2, l2, c, k)]
        assert api.kvq_check(ws, s) == 0
        del junk
        for a, b in zip(got, (out, lse, c0, k0)):
            assert torch.equal(a, b.cpu())
    with pytest.raises(ValueError, match="contiguous"):
        api.kvq_attn(p.ki, workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 30))


def test_short_pieces_one_after_another():
    # one tile to a row group: the two producer groups take turns by piece
    p = problem(B=600, Q=1, H=20, lens=[(7 * i) % 60 for i in range(600)], tree="null", seed=39)
    out, lse = check_attn(p)
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    other = torch.randn(1 << 16, device="cuda")
    for i in range(60):  # other kernels in between: the next call's code is not in the caches
        other.sort(), other.cumsum(0), (other[:1024, None] * other[None, :1024]) @ other[:1024]
        o2, l2 = run(p.ki, workspace=ws)
        assert torch.equal(out, o2) and torch.equal(lse, l2), i


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1), (2 ** 31 - 2, 7)])
def test_largest_windows_and_sinks(window, sinks):
    check_attn(problem(B=3, Q=9, H=7, lens=[0, 500, 61], seed=40, window=window, sinks=sinks))


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_calls_that_follow_each_other_see_each_other(captured):
    # rows written, attended to, read back and written over, one call right behind the other: each starts
    # before the last has ended, none may look before it has
    p = problem(B=6, Q=4, H=16, lens=[700, 90, 1300, 5, 64, 250], seed=44)
    n = sum(v + 4 for v in p.lens)
    at = p.ki.kv_indices[:n].contiguous()
    both = [latents("normal", n, torch.bfloat16, 45 + i) for i in range(2)]
    both = [(t.cuda(), k.cuda()) for t, k in both]
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    ws2 = api.alloc_workspace(api.KVQ_WORKSPACE_BYTES)

    def buffers():
        return (torch.zeros((6, 4, 16, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((6, 4, 16), device="cuda"),
                torch.zeros((n, 512), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda"))

    def step(i, o, sync):
        api.kvq_write(p.ki.cache, *both[i], at, workspace=ws2, check=False)
        if sync:
            torch.cuda.synchronize()
        api.kvq_attn(p.ki, out=o[0], lse=o[1], workspace=ws, check=False)
        if sync:
            torch.cuda.synchronize()
        api.kvq_read(p.ki.cache, at, kv_c=o[2], k_pe=o[3], workspace=ws2, check=False)
        if sync:
            torch.cuda.synchronize()
    want = [buffers() for _ in range(2)]
    for i in range(2):
        step(i, want[i], True)
    got = [buffers() for _ in range(30)]
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


@pytest.mark.parametrize("page", [1, 16])
def test_bad_tables_are_reported(page):
    def go(**kw):
        ki = dataclasses.replace(p.ki, **kw)
        ws = api.alloc_workspace(api.kvq_workspace_size(ki))
        out = torch.full((3, 4, 8, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((3, 4, 8), 4.0, device="cuda")
        run(ki, out=out, lse=lse, workspace=ws)
        return api.kvq_check(ws), out, lse
    p = problem(B=3, Q=4, H=8, lens=[150, 90, 10], page=page, seed=36)
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
        for v in (-1, p.ki.cache.rows.shape[0], 2 ** 31 - 1):
            e, out, lse = go(kv_indices=edit(p.ki.kv_indices, 7, v))  # sequence 0
            assert e == SLOT and torch.equal(out[1:], out0[1:]) and torch.equal(lse[1:], lse0[1:])
    else:
        e, out, lse = go(block_table=p.ki.block_table[:, :9].contiguous())
        assert e == PAGES and bool((out == 3).all())
        for v in (-1, p.ki.cache.rows.shape[0] // page, 2 ** 31 - 1):
            e, out, lse = go(block_table=edit(p.ki.block_table, 3, v))
            assert e == SLOT and torch.equal(out[1:], out0[1:]) and torch.equal(lse[1:], lse0[1:])
    for i, v in ((0, 0), (2, 2), (3, -2), (1, 77)):
        e, out, lse = go(tree_parent=edit(p.ki.tree_parent, i, v))
        assert e == PARENT and torch.equal(out[1:], out0[1:]) and torch.equal(lse[1:], lse0[1:])


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("value", [-2, -3, -17, -2 ** 31])
def test_every_negative_table_entry_is_reported(page, value):
    # at the first and the last position of the prefix and at a node's, of a whole row group and of a cut one
    p = problem(B=3, Q=4, H=8, lens=[150, 2900, 10], page=page, seed=48)
    out0, lse0 = check_attn(p)
    first = [0, 154, 154 + 2904] if page == 1 else [b * p.ki.block_table.shape[1] for b in range(3)]
    for b, pos in ((0, 0), (0, 149), (1, 2899), (1, 2903), (2, 9), (2, 13)):
        name = "kv_indices" if page == 1 else "block_table"
        t = getattr(p.ki, name).clone()
        t.view(-1)[first[b] + pos // page] = value
        ki = dataclasses.replace(p.ki, **{name: t})
        ws = api.alloc_workspace(api.kvq_workspace_size(ki))
        out, lse = run(ki, workspace=ws)
        assert api.kvq_check(ws) == SLOT, (b, pos)
        for o in {0, 1, 2} - {b}:
            assert torch.equal(out[o], out0[o]) and torch.equal(lse[o], lse0[o]), (b, pos, o)


def test_scores_of_minus_infinity():
    # rope keys of -infinity: tokens without weight, and rows that have no others, whole or cut into pieces
    p = problem(B=4, Q=1, H=4, lens=[3000, 200, 5, 2500], seed=49, tree="null")
    p.ki.q_pe[..., 0] = 1.0
    dead = np.concatenate([p.slots[0], p.slots[1][:150], p.slots[2], p.slots[3][:2490]]).astype(np.int64)
    p.ki.cache.rows[torch.from_numpy(dead).cuda(), 288] = 0x80
    p.ki.cache.rows[torch.from_numpy(dead).cuda(), 289] = 0xff
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    out, lse = run(p.ki, workspace=ws)
    assert api.kvq_check(ws) == 0
    for b in (0, 2):
        assert bool((out[b] == 0).all()), b
        assert bool((lse[b] == -float("inf")).all()), b
    # the others are those of the tokens with weight
    compare(dataclasses.replace(p, lens=[-1, 50, -1, 10],
                                slots=[None, p.slots[1][150:], None, p.slots[3][2490:]]), out, lse)


@pytest.mark.parametrize("exponent", [0, 4])
def test_attention_over_every_scale(exponent):
    # block i holds the scale bytes 4i .. 4i + 3 (zero, subnormals, .., 0x7f), with and without bit 7; the queries
    # make up for it, so that every block has its share of the scores
    p = problem(B=2, Q=3, H=8, lens=[333, 900], seed=50, exponent=exponent, scale=0.003)
    r = np.random.default_rng(51)
    p.rows[:, 256:288] = 4 * np.arange(32) + r.integers(0, 4, (len(p.rows), 32)) + 128 * r.integers(0, 2, (len(p.rows), 32))
    p.ki.cache.rows.copy_(torch.from_numpy(p.rows))
    up = 2.0 ** (9 - np.arange(32) // 2 - exponent)
    p.ki.q_lat.mul_(torch.from_numpy(up.repeat(16)).to(torch.bfloat16).cuda())
    check_attn(p)


@pytest.mark.parametrize("page", [1, 64])
def test_long_prefix(page):
    # 200,000 tokens, a head that sees them all alike, an ordinary one and a sharp one
    p = problem(B=1, Q=2, H=3, lens=[200_000], page=page, seed=52)
    for h, f in ((0, 2.0 ** -8), (2, 4.0)):
        p.ki.q_lat[:, :, h] *= f
        p.ki.q_pe[:, :, h] *= f
    out, lse = check_attn(p)
    # compare() allows the normaliser as many roundings as there are tokens.  It has fewer: a term passes the 31 + 1
    # additions of its tile, at most one for each of the 3,126 tiles and one for each of the fewer than 256 partial
    # results (the same again for their rescaling).  So a lost tile, 64 / 200,000 of the flat head's sum, would show.
    lat, rope = O.unpack_rows(p.rows[p.slots[0]])
    for i in range(2):
        pos = O.visible(p.parent[0], i, 200_000)
        q = p.ki.q_lat[0, i, 0].double().cpu().numpy(), p.ki.q_pe[0, i, 0].double().cpu().numpy()
        s = p.ki.scale * (lat[pos] @ q[0] + rope[pos] @ q[1])
        ds = 584 * 2.0 ** -24 * p.ki.scale * (np.abs(lat[pos]) @ np.abs(q[0]) + np.abs(rope[pos]) @ np.abs(q[1])).max()
        want = np.log(np.exp(s).sum())
        tol = ds + 2.0 ** -21 + (32 + 3126 + 2 * 256) * 2.0 ** -24 + 2.0 ** -22 * want
        assert tol < 64 / 200_000 * np.exp(s.min() - s.max())
        assert abs(float(lse[0, i, 0]) - want) <= tol


@pytest.mark.parametrize("kw", [
    dict(B=2, Q=16, H=64, lens=[900, 2100]),             # several row groups, cut ones among them
    dict(B=1, Q=1, H=16, lens=[0], tree="null"),         # one tile in one cluster
    dict(B=1, Q=1, H=128, lens=[200], tree="null"),
    dict(B=300, Q=1, H=20, lens=[(7 * i) % 60 for i in range(300)], tree="null"),  # pieces of one tile, rows left out
], ids=["groups", "one_tile", "four_tiles", "short_pieces"])
def test_timeout_is_reported_and_the_context_recovers(kw):
    p = problem(seed=53, **kw)
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    out, lse = run(p.ki)
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    for _ in range(2):
        t0 = time.monotonic()
        api.kvq_selftest_timeout(p.ki, o2, l2, ws, hold_ns=20_000_000)
        assert api.kvq_check(ws) == TIMEOUT
        assert time.monotonic() - t0 < 10
        o3, l3 = run(p.ki, workspace=ws)
        assert api.kvq_check(ws) == 0
        assert torch.equal(out, o3) and torch.equal(lse, l3)
    compare(p, out, lse)


def test_captured_call_follows_its_inputs():
    p = problem(B=3, Q=4, H=16, lens=[900, 300, 64], page=16, seed=37, window=128, sinks=5)
    ws = api.alloc_workspace(api.kvq_workspace_size(p.ki))
    out, lse = torch.zeros((3, 4, 16, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 4, 16), device="cuda")
    run(p.ki, out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.kvq_attn(p.ki, out=out, lse=lse, workspace=ws, check=False)
    for lens in ([900, 300, 64], [40, 299, 65], [-1, 0, 500], [700, -1, 1]):
        p.ki.prefix_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        # a table wide enough for every length: any page will do
        p.ki.block_table.copy_(torch.arange(p.ki.block_table.numel(), device="cuda").view_as(p.ki.block_table)
                               % (p.ki.cache.rows.shape[0] // 16))
        tab = p.ki.block_table.cpu().numpy()
        slots = [tab[b, np.arange(max(0, v + 4)) // 16].astype(np.int64) * 16 + np.arange(max(0, v + 4)) % 16
                 for b, v in enumerate(lens)]
        g.replay()
        torch.cuda.synchronize()
        assert api.kvq_check(ws) == 0
        compare(dataclasses.replace(p, slots=slots, lens=lens), out, lse)


# ---------------------------------------------------------------------------
# the operators together, as a speculative-decoding step uses them
# ---------------------------------------------------------------------------
def test_decode_loop_writes_attends_and_accepts():
    """Prefill rows are written, then each step drafts a tree, writes its
    nodes' rows to free slots, verifies it over the cache, accepts a path and
    keeps its rows by appending their slots to the sequence."""
    from mla_tree_verify_absorbed_gb300 import draft_inputs as DI
    torch.manual_seed(1)
    B, H, budget, L = 2, 8, 15, 6
    Q, pool = budget + 1, 600
    cache = api.kvq_alloc(pool, exponent=1)
    free = list(range(pool))[::-1]
    seq = [[free.pop() for _ in range(n)] for n in (130, 61)]
    truth = torch.zeros(pool, 576, dtype=torch.bfloat16)
    first = torch.tensor([s for q in seq for s in q], dtype=torch.int32)
    truth[first.long()] = torch.randn(len(first), 576).to(torch.bfloat16)
    api.kvq_write(cache, truth[first.long(), :512].cuda(), truth[first.long(), 512:].contiguous().cuda(), first.cuda())
    for step in range(4):
        d = DI.make_draft(name="loop", B=B, L=L, K=4, budget=budget, seed=50 + step)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        parent, token, _, _, ws = api.ddtree_build(t(d.root_token), t(d.cand_token), t(d.cand_logp), budget)
        nodes = torch.tensor([[free.pop() for _ in range(Q)] for _ in range(B)], dtype=torch.int32)
        new = torch.randn(B * Q, 576).to(torch.bfloat16)
        truth[nodes.view(-1).long()] = new
        new = new.cuda()
        api.kvq_write(cache, new[:, :512], new[:, 512:], nodes.view(-1).cuda())
        idx = [q + n.tolist() for q, n in zip(seq, nodes)]
        ptr = np.concatenate([[0], np.cumsum([len(i) for i in idx])]).astype(np.int32)
        lens = [len(q) for q in seq]
        q = torch.randn(B, Q, H, 576).to(torch.bfloat16)
        ki = api.KvqInputs(B=B, Q=Q, H=H, scale=0.07, q_lat=q[..., :512].contiguous().cuda(),
                           q_pe=q[..., 512:].contiguous().cuda(), cache=cache,
                           prefix_lens=torch.tensor(lens, dtype=torch.int32).cuda(), page_size=1, tree_parent=parent,
                           kv_indptr=t(ptr), kv_indices=torch.tensor(sum(idx, []), dtype=torch.int32).cuda())
        p = Prob(ki, cache.rows.cpu().numpy(), [np.array(i) for i in idx], lens, parent.cpu().numpy())
        # the cache holds what was written, to its 4 bits: an error of at most half a step and a scale's rounding
        lat, rope = O.unpack_rows(p.rows[np.concatenate(p.slots)], 1)
        want = truth[torch.tensor(sum(idx, [])).long()].double().numpy()
        top = np.abs(want[:, :512]).reshape(-1, 32, 16).max(-1).repeat(16, 1)
        assert (np.abs(lat - want[:, :512]) <= top / 14 * 1.07 + 1e-9).all()
        assert np.array_equal(rope, want[:, 512:])
        check_attn(p)
        tgt = DI.make_targets(d, parent.cpu().numpy(), seed=60 + step)
        n_len, _, _, kept, ws = api.ddtree_accept(parent, token, t(tgt), node_slot=nodes.cuda())
        assert api.check(ws) == 0
        for b in range(B):
            keep = kept[b, :int(n_len[b])].tolist()
            seq[b] += keep
            free = [s for s in nodes[b].tolist() if s not in keep] + free
