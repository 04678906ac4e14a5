"""The paged 8-bit latent cache's operators as cases to measure: each in its plain form
(elementary torch operations) and, with ``own`` set, through this package's entry points.

Operators
  tables  a step's page tables: pages taken from and returned to a ring of free ones by the
          requests' lengths, the new tokens' slots, and the page-size-1 form of the tables
  append  latent and rope rows are quantised into pool slots under the blocks' scales; the
          written rows and their blocks' other rows are read back
  read    rows of a filled cache are read back by slot (a context gathered for another use)
  attn    DDTree verify attention / decode over the 8-bit cache, sliding windows included

A cache row is 640 bytes: 512 latents as e4m3 codes and 64 rope values in bf16, both in units
of 2^(exponent + k), where k in 0..15 is the scale of the row's block of ``block`` pool slots.
``scales`` holds k + 1 for each block, 0 for one without rows.  A write raises k to what its
rows need (the least k with max|x| <= 448 * 2^(exponent + k)) and never lowers it; rows that
were in the block are rounded to the new unit.
"""
import math
import random

import torch

own = False

DL, DR, DK = 512, 64, 576
ROW = 640
KMAX = 15


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of eight requests, a page taken now and then: latency
        dict(name="tables_8_decode", op="tables", B=8, Q=1, lo=100, hi=4000, page=64, padded=1, ragged=0, width=128,
             lens_seed=11),
        # a large ragged batch in 16-token pages, prefill chunks of odd sizes for some, requests ended in others
        dict(name="tables_256_ragged", op="tables", B=256, Q=1, lo=64, hi=32768, page=16, padded=24, ragged=900,
             width=2200, lens_seed=12),
        # one draft tree's 64 nodes into the scattered rows of blocks that hold rows already: the per-step append
        dict(name="append_tree_64", op="append", n=64, dtype="bf16", skip=0, block=64, blocks=4096, scattered=True,
             old=0.5, exponent=-7),
        # a prefill chunk from an fp32 projection into fresh pages, padding rows skipped
        dict(name="append_prefill_fp32", op="append", n=40011, dtype="fp32", skip=37, block=64, blocks=1024,
             scattered=False, old=0.05, exponent=-7),
        # a few hundred rows of one short context, handed on in fp32
        dict(name="read_777_fp32", op="read", n=777, dtype="fp32", skip=3, block=16, blocks=256, exponent=2),
        # a 200k-token context read back as bf16 from scattered slots
        dict(name="read_200k", op="read", n=200000, dtype="bf16", skip=0, block=64, blocks=4096, exponent=-7),
        # single-token decode of one short sequence, 16 heads: latency
        dict(name="decode_1x257_h16", op="attn", B=1, Q=1, H=16, lo=257, hi=257, padded=0, page=1, block=64,
             chain=True, window=0, sinks=0, lens_seed=1),
        # a decode batch of 128-head sequences over 64-token pages, two slots of the batch unused
        dict(name="decode_32x8k_h128", op="attn", B=32, Q=1, H=128, lo=4096, hi=8192, padded=2, page=64, block=64,
             chain=True, window=0, sinks=0, lens_seed=2),
        # a large decode batch of very different lengths on a 16-head shard
        dict(name="decode_128ragged_h16", op="attn", B=128, Q=1, H=16, lo=64, hi=16384, padded=0, page=16, block=16,
             chain=True, window=0, sinks=0, lens_seed=3),
        # eight ragged sequences with 32-node draft trees, rows scattered over the pool
        dict(name="tree_8ragged_h64", op="attn", B=8, Q=32, H=64, lo=1024, hi=32768, padded=0, page=1, block=64,
             chain=False, window=0, sinks=0, lens_seed=1003),
        # the 64-node tree over a 200k prefix: the largest call
        dict(name="tree_1x200k_h64", op="attn", B=1, Q=64, H=64, lo=200000, hi=200000, padded=0, page=64, block=64,
             chain=False, window=0, sinks=0, lens_seed=5),
        # decode of long sequences that keep 4 first tokens and the last 4096; pages between are freed
        dict(name="window_16x100k_h64", op="attn", B=16, Q=1, H=64, lo=50000, hi=100000, padded=0, page=64, block=64,
             chain=True, window=4096, sinks=4, lens_seed=6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "read", "attn", "attn", "attn"])
    if op == "tables":
        B = _log_int(rng, 1, 256)
        hi = _log_int(rng, 32, 32768)
        page = rng.choice([1, 16, 64, rng.randint(2, 100)])
        ragged = rng.choice([0, 0, rng.randint(1, 2000)])
        Q = rng.choice([1, 1, rng.randint(2, 64)])
        while B * hi > 2000000:
            hi //= 2
        return dict(op=op, B=B, Q=Q, lo=rng.randint(0, hi), hi=hi, page=page, padded=rng.randint(0, B // 3),
                    ragged=ragged, width=-(-(hi + max(Q, ragged)) // page) + rng.randint(2, 40),
                    lens_seed=rng.randint(0, 10 ** 6))
    if op in ("append", "read"):
        n = _log_int(rng, 1, 40000 if op == "append" else 200000)
        block = rng.choice([1, 8, 16, 64, rng.randint(2, 128)])
        c = dict(op=op, n=n, dtype=rng.choice(["bf16", "fp32"]), skip=rng.randint(0, max(0, min(n - 1, 40))),
                 block=block, blocks=-(-n // block) + rng.randint(1, max(1, 60000 // block)),
                 exponent=rng.randint(-9, 3))
        if op == "append":
            c["scattered"] = rng.random() < 0.5
            c["old"] = rng.choice([0.0, 0.05, 0.5])
        return c
    H = rng.choice([8, 16, 32, 64, 128, rng.randint(1, 96)])
    Q = rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, 64)])
    B = _log_int(rng, 1, 96)
    hi = _log_int(rng, 32, 131072)
    # the padded batch of the plain form and the work stay below the largest listed case's
    while B * hi > 600000 or B * hi * Q * H > 600000000:
        hi = max(32, hi // 2)
        if hi == 32:
            B = max(1, B // 2)
    lo = rng.randint(max(0, hi // 8), hi)
    c = dict(op=op, B=B, Q=Q, H=H, lo=lo, hi=hi, padded=rng.choice([0, 0, min(B - 1, 1)]),
             page=rng.choice([1, 8, 16, 64, rng.randint(2, 100)]), block=rng.choice([1, 16, 64, rng.randint(2, 128)]),
             chain=rng.random() < 0.4, window=0, sinks=0, lens_seed=rng.randint(0, 10 ** 6))
    if rng.random() < 0.3:
        c["window"] = _log_int(rng, 1, 8192)
        c["sinks"] = rng.choice([0, 1, 4, rng.randint(2, 200)])
    return c


def _lens(case):
    """Prefix lengths of the batch (host list): -1 marks an unused slot of the batch."""
    r = random.Random(case["lens_seed"])
    B, lo, hi = case["B"], case["lo"], case["hi"]
    wide = lo > 0 and hi > 10 * lo
    v = [_log_int(r, lo, hi) if wide else r.randint(lo, hi) for _ in range(B - case["padded"])]
    v += [-1] * case["padded"]
    if case["op"] == "tables":
        r.shuffle(v)
    return v


def _new(case):
    """New tokens of each sequence of a tables case."""
    if not case["ragged"]:
        return [case["Q"]] * case["B"]
    r = random.Random(case["lens_seed"] + 1)
    return [r.choice([0, 1, 1, 1, r.randint(1, case["ragged"])]) for _ in range(case["B"])]


def _pages(case):
    """Pages of each sequence before and after the step."""
    r = random.Random(case["lens_seed"] + 2)
    ps, held, need = case["page"], [], []
    for p, n in zip(_lens(case), _new(case)):
        need.append(-(-(p + n) // ps) if p >= 0 else 0)
        # what the step before left: the prefix's pages, sometimes those of rejected nodes too; an ended request's
        held.append(-(-p // ps) + r.choice([0, 0, 1, 2]) if p >= 0 else r.choice([0, r.randint(1, case["width"])]))
        held[-1] = min(held[-1], case["width"])
    return held, need


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _latents(n, g, dev, exponent=0):
    """Normalised latents of about unit size times 2^(exponent + 7): rows times a per-channel gain and
    a size of their own, as an RMS norm's output has."""
    gain = torch.exp(0.4 * torch.randn(DL, generator=g, device=dev))
    x = torch.randn(n, DL, generator=g, device=dev)
    x *= gain
    x *= torch.exp(0.3 * torch.randn(n, 1, generator=g, device=dev)) * 2.0 ** (exponent + 7)
    return x, torch.randn(n, DR, generator=g, device=dev)


def _filled(blocks, block, exponent, g, dev):
    """A filled cache: rows [blocks * block][640] uint8 and scales [blocks] int32."""
    rows = torch.empty(blocks * block, ROW, dtype=torch.uint8, device=dev)
    scales = torch.empty(blocks, dtype=torch.int32, device=dev)
    step = max(1, (1 << 17) // block)
    for a in range(0, blocks, step):
        m = min(step, blocks - a)
        x, r = _latents(m * block, g, dev, exponent)
        k = _needed(x.abs().amax(1), exponent).view(m, block).amax(1)
        unit = torch.exp2(-(exponent + k).float()).repeat_interleave(block)[:, None]
        at = slice(a * block, (a + m) * block)
        rows[at, :DL] = (x * unit).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        rows[at, DL:] = (r * unit).to(torch.bfloat16).view(torch.uint8)
        scales[a:a + m] = k.int() + 1
    return rows, scales


def _parents(Q, r, cap=8):
    """A random draft tree: node 0 the root, depth capped."""
    par, dep = [-1], [1]
    for i in range(1, Q):
        p = r.randrange(0, i)
        while dep[p] >= cap:
            p = r.randrange(0, i)
        par.append(p)
        dep.append(dep[p] + 1)
    return par


def _prepare_tables(case, st, g, dev):
    B, ps, width = case["B"], case["page"], case["width"]
    held, need = _pages(case)
    take = sum(max(0, n - h) for h, n in zip(held, need))
    count = sum(held) + take + 37
    ids = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    ring = torch.full((count,), -1, dtype=torch.int32, device=dev)
    head = 5 * count + count // 3  # a ring that has turned a few times
    free = count - at
    ring[(head + torch.arange(free, device=dev)) % count] = ids[at:]
    new = _new(case)
    live = [p >= 0 for p in _lens(case)]
    total = sum(p + n for p, n, u in zip(_lens(case), new, live) if u)
    st.update(block_table=table, pages_held=torch.tensor(held, dtype=torch.int32, device=dev), free_ring=ring,
              free_state=torch.tensor([head, head + free, 0], dtype=torch.int64, device=dev),
              prefix_lens=torch.tensor(_lens(case), dtype=torch.int32, device=dev), num_pages=count,
              new_lens=torch.tensor(new, dtype=torch.int32, device=dev) if case["ragged"] else None)
    rows = sum(n for n, u in zip(new, live) if u) + 29 if case["ragged"] else B * case["Q"]
    st["slots"] = torch.zeros(rows, dtype=torch.int32, device=dev)
    st["kv_indptr"] = torch.zeros(B + 1, dtype=torch.int32, device=dev)
    st["kv_indices"] = torch.zeros(total + 3, dtype=torch.int32, device=dev)
    # the cache whose blocks are the pages: those taken become empty
    st["scales"] = torch.randint(0, KMAX + 2, (count,), generator=g, device=dev).to(torch.int32)
    st["rows"] = torch.empty(count * ps, ROW, dtype=torch.uint8, device=dev)  # not touched by this step
    st["ws"] = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = random.Random(seed)
    st = dict(case)
    if case["op"] == "tables":
        return _prepare_tables(case, st, g, dev)
    if case["op"] in ("append", "read"):
        n, block, blocks, e = case["n"], case["block"], case["blocks"], case["exponent"]
        pool = blocks * block
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rows, scales = _filled(blocks, block, e, g, dev)
        if case["op"] == "append" and not case["scattered"]:
            # whole blocks in random order, filled row after row
            order = torch.randperm(blocks, generator=g, device=dev)
            slots = (order[:, None] * block + torch.arange(block, device=dev)).view(-1)[:n].to(torch.int32)
        else:
            slots = torch.randperm(pool, generator=g, device=dev)[:n].to(torch.int32)
        if case["skip"]:
            slots[torch.randperm(n, generator=g, device=dev)[:case["skip"]]] = -1
        st["rows"], st["scales"], st["slots"] = rows, scales, slots
        look = n
        if case["op"] == "append":
            # blocks without rows yet are empty, and their bytes mean nothing
            scales[torch.rand(blocks, generator=g, device=dev) >= case["old"]] = 0
            x, k = _latents(n, g, dev, e)
            st["kv_c"], st["k_pe"] = x.to(dt), k.to(dt)
            # read back: the new rows, and rows that their blocks held before
            mine = slots[slots >= 0]
            near = ((mine // block).long() * block + torch.randint(0, block, (len(mine),), generator=g, device=dev))
            fresh = torch.zeros(pool, dtype=torch.bool, device=dev)
            fresh[mine.long()] = True
            ok = (scales[(near // block)] > 0) & ~fresh[near]
            near = torch.where(ok, near, torch.full_like(near, -1)).to(torch.int32)
            st["look"] = torch.cat([slots, near])
            look = st["look"].numel()
        st["out_c"] = torch.zeros(look, DL, dtype=dt, device=dev)
        st["out_r"] = torch.zeros(look, DR, dtype=dt, device=dev)
        st["ws"] = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
        return st
    B, Q, H, ps, block = case["B"], case["Q"], case["H"], case["page"], case["block"]
    lens = _lens(case)
    need = [0 if p < 0 else p + Q for p in lens]
    W, sinks = case["window"], case["sinks"]
    st["n_max"] = max(need)
    st["prefix_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["tree_parent"] = None if case["chain"] else torch.tensor([_parents(Q, r) for _ in range(B)], dtype=torch.int32,
                                                                device=dev)
    if ps == 1:
        total = sum(need)
        pool = total + total // 4 + 64
        idx = torch.randperm(pool, generator=g, device=dev)[:total].to(torch.int32)
        ptr = [0]
        for v in need:
            ptr.append(ptr[-1] + v)
        st["kv_indices"] = idx
        st["kv_indptr"] = torch.tensor(ptr, dtype=torch.int32, device=dev)
    else:
        pages = [-(-v // ps) for v in need]
        width = max(max(pages), 1)
        count = sum(pages) + 3
        ids = torch.randperm(count, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, c in enumerate(pages):
            table[b, :c] = ids[at:at + c]
            at += c
            if W and lens[b] >= 0:  # pages that no node sees any more are gone from the table
                a, z = -(-sinks // ps), max(0, lens[b] - W + 1) // ps
                if z > a:
                    table[b, a:z] = -1
        st["block_table"] = table
        pool = count * ps
    st["exponent"] = -7
    st["rows"], st["scales"] = _filled(-(-pool // block), block, -7, g, dev)
    st["q_lat"] = torch.randn(B, Q, H, DL, generator=g, device=dev).to(torch.bfloat16)
    st["q_pe"] = torch.randn(B, Q, H, DR, generator=g, device=dev).to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(192.0)
    st["out"] = torch.zeros(B, Q, H, DL, dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.zeros(B, Q, H, dtype=torch.float32, device=dev)
    # scratch that the program keeps: partial results of one device's SMs
    st["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _needed(amax, exponent):
    """The least k in 0..15 with amax <= 448 * 2^(exponent + k); 15 where there is none."""
    k = torch.arange(KMAX, device=amax.device)
    return (amax.float()[:, None] > 448.0 * torch.exp2((exponent + k).float())).sum(1)


def _to_e4m3(v):
    """fp32 values rounded to e4m3 (ties to even, at most 448), exactly."""
    e = torch.frexp(v).exponent - 1
    step = torch.exp2((torch.clamp(e, min=-6) - 3).float())
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _codes(by):
    """e4m3 codes as fp32."""
    by = by.to(torch.int32)
    e, m = (by >> 3) & 15, (by & 7).float()
    v = torch.where(e > 0, (8.0 + m) * torch.exp2((e - 10).float()), m * 2.0 ** -9)
    return torch.where(by > 127, -v, v)


def _values(rows):
    """Latents [..., 512] and rope keys [..., 64] of cache rows in their blocks' units, fp32 (exact)."""
    return _codes(rows[..., :DL]), rows[..., DL:].contiguous().view(torch.bfloat16).float()


def _plain_tables(st):
    dev = st["prefix_lens"].device
    B, Q, ps, width = st["B"], st["Q"], st["page"], st["width"]
    P = st["prefix_lens"].long()
    live = P >= 0
    n = torch.full_like(P, Q) if st["new_lens"] is None else st["new_lens"].long()
    n = torch.where(live, n, torch.zeros_like(n))
    length = torch.where(live, P + n, torch.zeros_like(P))
    need, held = (length + ps - 1) // ps, st["pages_held"].long()
    take, drop = torch.clamp(need - held, min=0), torch.clamp(held - need, min=0)
    head, tail = st["free_state"][0], st["free_state"][1]
    ring = st["free_ring"]
    cap = ring.numel()
    j = torch.arange(width, device=dev)
    got = (head + (torch.cumsum(take, 0) - take)[:, None] + (j - held[:, None])) % cap
    table = torch.where(j < torch.minimum(held, need)[:, None], st["block_table"], torch.full_like(st["block_table"], -1))
    taken = (j >= held[:, None]) & (j < need[:, None])
    table = torch.where(taken, ring[got], table)
    # pages that are left over go behind the ring's last, in order
    back = (tail + (torch.cumsum(drop, 0) - drop)[:, None] + (j - need[:, None])) % cap
    left = (j >= need[:, None]) & (j < held[:, None])
    ring = ring.clone()
    ring[back[left]] = st["block_table"][left]
    scales = st["scales"].clone()
    scales[table[taken].long()] = 0
    # page-size-1 form
    ptr = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(length, 0)])
    total = int(ptr[-1])
    flat = torch.arange(total, device=dev)
    b = torch.searchsorted(ptr[1:], flat, right=True)
    pos = flat - ptr[b]
    idx = st["kv_indices"].clone()
    idx[:total] = (table[b, pos // ps] * ps + pos % ps).int()
    # the new tokens' slots
    slots = torch.full_like(st["slots"], -1)
    if st["new_lens"] is None:
        p = torch.clamp(P, min=0)[:, None] + torch.arange(Q, device=dev)
        s = torch.gather(table.long(), 1, torch.clamp(p // ps, max=width - 1)) * ps + p % ps
        slots = torch.where(live[:, None], s, torch.full_like(s, -1)).int().view(-1)
    else:
        m = torch.cumsum(n, 0)
        row = torch.arange(int(m[-1]), device=dev)
        b = torch.searchsorted(m, row, right=True)
        p = P[b] + row - (m[b] - n[b])
        slots[:len(row)] = (table[b, p // ps] * ps + p % ps).int()
    state = torch.stack([head + take.sum(), tail + drop.sum(), st["free_state"][2]])
    return table, need.int(), ring, state, slots, ptr.int(), idx, scales


def _plain_append(st):
    e, block, dt = st["exponent"], st["block"], st["out_c"].dtype
    live = st["slots"] >= 0
    at = st["slots"].clamp(min=0).long()
    x = st["kv_c"].float()
    # scales: the larger of what was there and what the rows need
    k = torch.where(live, _needed(x.abs().amax(1), e), torch.zeros_like(at))
    old = torch.clamp(st["scales"].long() - 1, min=0)
    new = old.scatter_reduce(0, at // block, k, "amax")
    touched = torch.zeros_like(old).scatter_reduce(0, at // block, live.long(), "amax") > 0
    scales = torch.where((st["scales"] > 0) | touched, new + 1, torch.zeros_like(new)).int()
    ku = torch.exp2((e + new[at // block]).float())[:, None]
    lat_n, rope_n = _to_e4m3(x / ku) * ku, (st["k_pe"].float() / ku).to(torch.bfloat16).float() * ku
    # rows that were there, in the new unit
    look = st["look"][len(at):]
    near = look.clamp(min=0).long()
    lat, rope = _values(st["rows"][near])
    d = torch.exp2((old - new)[near // block].float())[:, None]
    u = torch.exp2((e + new[near // block]).float())[:, None]
    lat_o, rope_o = _to_e4m3(lat * d) * u, (rope * d).to(torch.bfloat16).float() * u
    keep = (st["look"] >= 0)[:, None]
    out_c = torch.where(keep, torch.cat([lat_n, lat_o]).to(dt), st["out_c"])
    return out_c, torch.where(keep, torch.cat([rope_n, rope_o]).to(dt), st["out_r"]), scales


def _plain_read(st):
    dt = st["out_c"].dtype
    live = (st["slots"] >= 0)[:, None]
    at = st["slots"].clamp(min=0).long()
    lat, rope = _values(st["rows"][at])
    u = torch.exp2((st["exponent"] + st["scales"][at // st["block"]] - 1).float())[:, None]
    return torch.where(live, (lat * u).to(dt), st["out_c"]), torch.where(live, (rope * u).to(dt), st["out_r"])


def _plain_attn(st):
    B, Q, H, W, sinks = st["B"], st["Q"], st["H"], st["window"], st["sinks"]
    dev = st["q_lat"].device
    P = st["prefix_lens"].long()
    # ancestor-or-self relation and depths
    if st["tree_parent"] is None:
        anc = torch.ones(Q, Q, device=dev).tril().expand(B, Q, Q)
    else:
        node = torch.arange(Q, device=dev)
        anc = (st["tree_parent"].long()[:, :, None] == node).float() + torch.eye(Q, device=dev)
        for _ in range(6):
            anc = torch.clamp(anc @ anc, max=1.0)
    depth = anc.sum(-1).long() - 1
    # positions that some node of the sequence may see
    if W:
        first = min(sinks, st["n_max"])
        lo = torch.clamp(P - W + 1, min=first)
        pos = torch.cat([torch.arange(first, device=dev).expand(B, first),
                         lo[:, None] + torch.arange(min(W - 1, st["n_max"]) + Q, device=dev)], 1)
    else:
        pos = torch.arange(st["n_max"], device=dev).expand(B, -1)
    inside = (pos < (P + Q)[:, None]) & (P >= 0)[:, None]
    safe = torch.where(inside, pos, torch.zeros_like(pos))
    if st["page"] == 1:
        at = st["kv_indptr"][:-1].long()[:, None] + safe
        slot = st["kv_indices"][at.clamp(max=st["kv_indices"].numel() - 1)].long()
    else:
        slot = torch.gather(st["block_table"].long(), 1, safe // st["page"]) * st["page"] + safe % st["page"]
    slot = torch.where(inside, slot, torch.zeros_like(slot))
    lat, rope = _values(st["rows"][slot])
    unit = torch.exp2((st["exponent"] + st["scales"][slot // st["block"]] - 1).float())[..., None]
    lat *= unit
    rope *= unit
    # visibility
    t = (pos - P[:, None])
    tree = (t >= 0) & (t < Q)
    tc = t.clamp(0, Q - 1)
    row_anc = torch.gather(anc, 2, tc[:, None, :].expand(B, Q, -1)) > 0
    see = inside[:, None, :] & torch.where(tree[:, None, :], row_anc, (t < 0)[:, None, :])
    if W:
        own_pos = P[:, None] + depth
        key_pos = torch.where(tree, P[:, None] + torch.gather(depth, 1, tc), pos)
        see = see & ((key_pos < sinks)[:, None, :] | (own_pos[:, :, None] - key_pos[:, None, :] < W))
    s = torch.bmm(st["q_lat"].float().view(B, Q * H, DL), lat.transpose(1, 2))
    s += torch.bmm(st["q_pe"].float().view(B, Q * H, DR), rope.transpose(1, 2))
    s *= st["scale"]
    s = s.view(B, Q, H, -1)
    s.masked_fill_(~see[:, :, None, :], -math.inf)
    mx = s.amax(-1, keepdim=True)
    mx = torch.where(mx == -math.inf, torch.zeros_like(mx), mx)
    s = s.sub_(mx).exp_()
    z = s.sum(-1, keepdim=True)
    o = torch.bmm(s.view(B, Q * H, -1), lat).view(B, Q, H, DL) / z
    live = (P >= 0)[:, None, None]
    out = torch.where(live[..., None], o.to(torch.bfloat16), st["out"])
    return out, torch.where(live, (mx + z.log())[..., 0], st["lse"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    op = st["op"]
    if not own:
        return {"tables": _plain_tables, "append": _plain_append, "read": _plain_read, "attn": _plain_attn}[op](st)
    from mla_tree_verify_absorbed_gb300 import api
    if op == "tables":
        ti = api.TableInputs(page_size=st["page"], Q=st["Q"], prefix_lens=st["prefix_lens"], new_lens=st["new_lens"],
                             block_table=st["block_table"], pages_held=st["pages_held"], free_ring=st["free_ring"],
                             free_state=st["free_state"], num_pages=st["num_pages"])
        cache = api.BlockCache(st["rows"], st["scales"], st["page"])
        api.kv_tables(ti, slots=st["slots"], kv_indptr=st["kv_indptr"], kv_indices=st["kv_indices"], cache=cache,
                      workspace=st["ws"], check=False)
        return (st["block_table"], st["pages_held"], st["free_ring"], st["free_state"], st["slots"], st["kv_indptr"],
                st["kv_indices"], st["scales"])
    cache = api.BlockCache(st["rows"], st["scales"], st["block"], st["exponent"])
    if op == "append":
        api.kv8_write(cache, st["kv_c"], st["k_pe"], st["slots"], workspace=st["ws"], check=False)
        api.kv8_read(cache, st["look"], kv_c=st["out_c"], k_pe=st["out_r"], workspace=st["ws"], check=False)
        return st["out_c"], st["out_r"], st["scales"]
    if op == "read":
        api.kv8_read(cache, st["slots"], kv_c=st["out_c"], k_pe=st["out_r"], workspace=st["ws"], check=False)
        return st["out_c"], st["out_r"]
    ki = api.Kv8Inputs(B=st["B"], Q=st["Q"], H=st["H"], scale=st["scale"], q_lat=st["q_lat"], q_pe=st["q_pe"],
                       cache=cache, prefix_lens=st["prefix_lens"], page_size=st["page"],
                       tree_parent=st["tree_parent"], kv_indptr=st.get("kv_indptr"), kv_indices=st.get("kv_indices"),
                       block_table=st.get("block_table"), window=st["window"], sinks=st["sinks"])
    return api.kv8_attn(ki, out=st["out"], lse=st["lse"], workspace=st["ws"], check=False)


def work(case):
    if case["op"] == "tables":
        held, need = _pages(case)
        lens, new = _lens(case), _new(case)
        tokens = sum(p + n for p, n in zip(lens, new) if p >= 0)
        fresh = sum(n for p, n in zip(lens, new) if p >= 0) if case["ragged"] else case["B"] * case["Q"]
        moved = sum(abs(h - n) for h, n in zip(held, need))
        # lengths, held counts and offsets; the held entries; pages moved through the ring; indices and slots out
        b = 4 * case["B"] * (5 if case["ragged"] else 4) + 4 * sum(held) + 12 * moved + 4 * (tokens + fresh)
        return {"bytes": b, "flops": 0}
    if case["op"] in ("append", "read"):
        m, el = case["n"] - case["skip"], 2 if case["dtype"] == "bf16" else 4
        b = m * (ROW + DK * el) + 4 * case["n"]
        if case["op"] == "append":  # source rows in, cache rows out, and the same slots read back
            b += m * (DK * el + ROW) + 8 * case["n"] + 4 * case["blocks"]
        return {"bytes": b, "flops": 0}
    B, Q, H, W, sinks = case["B"], case["Q"], case["H"], case["window"], case["sinks"]
    rows, pairs = 0, 0
    for p in _lens(case):
        if p < 0:
            continue
        # every node sees at least this much of the prefix, and itself
        seen = p if not W else min(p, sinks) + max(0, p - max(min(p, sinks), p - W + 1))
        rows += seen + Q
        pairs += Q * H * (max(0, seen - (Q if W else 0)) + 1)
    live = sum(p >= 0 for p in _lens(case))
    b = rows * (ROW + (4 if case["page"] == 1 else 0)) + live * Q * H * (2 * DK + 2 * DL + 4)
    return {"bytes": b, "flops": 2 * pairs * (DK + DL)}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_table(dev):
    """The 127 finite non-negative e4m3 values in order, float64: index = code."""
    i = torch.arange(127, device=dev, dtype=torch.float64)
    e, m = torch.floor(i / 8), i % 8
    return torch.where(e > 0, (8 + m) * torch.exp2(e - 10), m * 2.0 ** -9)


def _nearest64(v):
    """The e4m3 value nearest each float64 (the even code wins a tie)."""
    table = _e4m3_table(v.device)
    a = v.abs().clamp(max=448.0)
    i = torch.searchsorted(table, a).clamp(max=126)
    j = (i - 1).clamp(min=0)
    up, down = table[i] - a, a - table[j]
    m = torch.where((up < down) | ((up == down) & (i % 2 == 0)), table[i], table[j])
    return torch.where(v < 0, -m, m)


def _decode64(rows):
    """Latents and rope keys of cache rows in their blocks' units."""
    table = _e4m3_table(rows.device)
    code = rows[:, :DL].long()
    lat = table[code % 128] * torch.where(code < 128, 1.0, -1.0)
    bits = (rows[:, DL::2].long() | rows[:, DL + 1::2].long() << 8) << 16
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    return lat, bits.view(torch.float32).double()


def _exact_append(case, st):
    e, block = case["exponent"], case["block"]
    out_c, out_r = st["out_c"].double(), st["out_r"].double()
    n = case["n"]
    live = (st["slots"] >= 0).nonzero()[:, 0]
    at = st["slots"][live].long()
    x = st["kv_c"][live].double()
    was = st["scales"].cpu().tolist()
    now = list(was)
    for b, a in zip((at // block).tolist(), x.abs().amax(1).tolist()):
        k = 0
        while k < KMAX and a > 448.0 * 2.0 ** (e + k):
            k += 1
        now[b] = max(now[b], k + 1)
    dev = x.device
    was, now = torch.tensor(was, device=dev), torch.tensor(now, device=dev)
    u = torch.exp2(e + now[at // block].double() - 1)[:, None]
    out_c[live], out_r[live] = _nearest64(x / u) * u, (st["k_pe"][live].double() / u).float().to(torch.bfloat16).double() * u
    rest = (st["look"][n:] >= 0).nonzero()[:, 0]
    at = st["look"][n:][rest].long()
    if len(at):
        lat, rope = _decode64(st["rows"][at])
        d = torch.exp2((was - now)[at // block].double())[:, None]
        u = torch.exp2(e + now[at // block].double() - 1)[:, None]
        out_c[n + rest] = _nearest64(lat * d) * u
        out_r[n + rest] = (rope * d).float().to(torch.bfloat16).double() * u
    return out_c, out_r, now.to(torch.int32)


def _exact_tables(case, st):
    ps, ring = case["page"], st["free_ring"].tolist()
    cap = len(ring)
    head, tail, zero = st["free_state"].tolist()
    table, held = st["block_table"].tolist(), st["pages_held"].tolist()
    scales, slots, ptr, idx = st["scales"].tolist(), [], [0], []
    lens, new = _lens(case), _new(case)
    for b, p in enumerate(lens):
        need = (p + new[b] + ps - 1) // ps if p >= 0 else 0
        for j in range(held[b], need):
            table[b][j] = ring[head % cap]
            scales[table[b][j]] = 0
            head += 1
        for j in range(need, held[b]):
            ring[tail % cap] = table[b][j]
            table[b][j] = -1
            tail += 1
        held[b] = need
        where = [table[b][i // ps] * ps + i % ps for i in range(p + new[b])] if p >= 0 else []
        idx += where
        ptr.append(len(idx))
        slots += where[p:] if p >= 0 else [] if case["ragged"] else [-1] * case["Q"]
    slots += [-1] * (st["slots"].numel() - len(slots))
    idx += [0] * (st["kv_indices"].numel() - len(idx))
    dev = st["slots"].device
    ints = [torch.tensor(v, dtype=torch.int32, device=dev) for v in (table, held, ring, slots, ptr, idx, scales)]
    return (*ints[:3], torch.tensor([head, tail, zero], dtype=torch.int64, device=dev), *ints[3:])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "read":
        out_c, out_r = st["out_c"].double(), st["out_r"].double()
        live = (st["slots"] >= 0).nonzero()[:, 0]
        at = st["slots"][live].long()
        lat, rope = _decode64(st["rows"][at])
        u = torch.exp2(case["exponent"] + st["scales"][at // case["block"]].double() - 1)[:, None]
        out_c[live], out_r[live] = lat * u, rope * u
        return out_c, out_r
    B, Q, H, W, sinks, ps = (case[k] for k in ("B", "Q", "H", "window", "sinks", "page"))
    out, lse = st["out"].double(), st["lse"].double()
    for b, p in enumerate(_lens(case)):
        if p < 0:
            continue
        par = list(range(-1, Q - 1)) if st["tree_parent"] is None else st["tree_parent"][b].tolist()
        chains = []
        for i in range(Q):
            up = [i]
            while par[up[-1]] >= 0:
                up.append(par[up[-1]])
            chains.append(up)
        depth = [len(u) - 1 for u in chains]
        pos = torch.arange(p + Q, device=out.device)
        if W:
            pos = pos[(pos < sinks) | (pos > p - W)]
        if ps == 1:
            slot = st["kv_indices"][int(st["kv_indptr"][b]) + pos].long()
        else:
            slot = st["block_table"][b][pos // ps].long() * ps + pos % ps
        lat, rope = _decode64(st["rows"][slot])
        keys = torch.cat([lat, rope], 1)
        keys *= torch.exp2(st["exponent"] + st["scales"][slot // case["block"]].double() - 1)[:, None]
        at = pos.clone()  # a node stands at its depth below the prefix
        at[pos >= p] = p + torch.tensor(depth, device=pos.device)[pos[pos >= p] - p]
        for i in range(Q):
            see = (pos < p) | torch.isin(pos, p + torch.tensor(chains[i], device=pos.device))
            if W:
                see = see & ((at < sinks) | (p + depth[i] - at < W))
            kk = keys if bool(see.all()) else keys[see]
            s = st["scale"] * (torch.cat([st["q_lat"][b, i], st["q_pe"][b, i]], 1).double() @ kk.T)
            lse[b, i] = torch.logsumexp(s, -1)
            out[b, i] = torch.exp(s - lse[b, i][:, None]) @ kk[:, :DL]
    return out, lse
