"""A step's page tables on the GPU, entry for entry against the oracle, and the serving
loop that they make: tables, writes, verify attention and acceptance without a host
round trip in between."""
import dataclasses

import numpy as np
import pytest

from mla_tree_verify_absorbed_gb300 import api
from oracle import kv8 as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SLOT, PREFIX, PAGES, CAPACITY = 0x4, 0x1, 0x10, 0x20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.load()


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


class State:
    """Tables on the device and in the oracle, side by side."""

    def __init__(self, B, max_pages, num_pages, page, block=0, ring=None, head=0, seed=0):
        r = np.random.default_rng(seed)
        ring = ring or num_pages
        self.page, self.block = page, block
        self.ti = api.kv_tables_alloc(B, max_pages, num_pages, page)
        ids = np.full(ring, -7)
        ids[(head + np.arange(num_pages)) % ring] = r.permutation(num_pages)
        self.ti.free_ring = i32(ids)
        self.ti.free_state.copy_(torch.tensor([head, head + num_pages, 0]))
        self.cache = None
        if block:
            self.cache = api.BlockCache(torch.empty((num_pages * page, 640), dtype=torch.uint8, device="cuda"),
                                        i32(r.integers(0, 17, -(-num_pages * page // block))), block)
        self.host()

    def host(self):
        t = self.ti
        self.h = dict(table=t.block_table.tolist(), held=t.pages_held.tolist(), ring=t.free_ring.tolist(),
                      state=t.free_state.tolist(), words=None if self.cache is None else self.cache.scales.tolist())

    def step(self, prefix, new=None, Q=1, status=0, spare=5, slots_len=None, idx_len=None, ws=None, stream=None):
        h, t = self.h, self.ti
        t.prefix_lens = i32(prefix)
        t.Q, t.new_lens = Q, None if new is None else i32(new)
        if status in (0, SLOT):
            want = O.tables(self.page, Q, prefix, new, h["table"], h["held"], h["ring"], h["state"], t.num_pages,
                            words=h["words"], block=self.block or 1)
        else:
            want = dict(h, slots=[-1] * 100, idx=[-1] * 100, ptr=[])  # room enough
        n = len(want["slots"]) + (0 if new is None else spare) if slots_len is None else slots_len
        if new is None:
            n = len(prefix) * Q
        slots, ptr = torch.full((n,), -9, dtype=torch.int32).cuda(), torch.full((len(prefix) + 1,), -9, dtype=torch.int32).cuda()
        idx = torch.full((len(want["idx"]) + spare if idx_len is None else idx_len,), -9, dtype=torch.int32).cuda()
        ws = api.kv_tables(t, slots, ptr, idx, cache=self.cache, workspace=ws, stream=stream)
        assert api.kv8_check(ws, stream) == status
        if status == 0:
            assert slots.tolist() == want["slots"] + [-1] * (n - len(want["slots"]))
            assert ptr.tolist() == want["ptr"]
            assert idx.tolist() == want["idx"] + [-9] * (len(idx) - len(want["idx"]))
        elif status != SLOT:
            for x in (slots, ptr, idx):
                assert bool((x == -9).all())
        self.host()
        for k in ("table", "held", "ring", "state", "words"):
            assert self.h[k] == want[k], k
        return slots, ptr, idx


@pytest.mark.parametrize("page,block", [(1, 0), (1, 1), (1, 3), (16, 16), (16, 4), (16, 64), (16, 5), (7, 0), (64, 64),
                                        (100, 50)])
@pytest.mark.parametrize("seed", range(3))
def test_random_steps_match_the_oracle(page, block, seed):
    # requests that begin, grow by one token, by a tree or by a chunk, are cut back and end; a ring that has turned
    r = np.random.default_rng(seed)
    B = int(r.integers(1, 40))
    s = State(B, 60, 60 * B, page, block, ring=60 * B + int(r.integers(0, 9)), head=int(r.integers(0, 10 ** 6)), seed=seed)
    prefix = [-1] * B
    for step in range(8):
        for b in range(B):
            u = r.random()
            prefix[b] = -1 if u < 0.15 else int(r.integers(0, 40 * page)) if prefix[b] < 0 or u < 0.3 else \
                min(40 * page, prefix[b] + int(r.integers(0, 2 * page + 2)))
        if step % 2:
            new = [int(r.choice([0, 1, 1, r.integers(0, 20 * page)])) for _ in range(B)]
            s.step(prefix, new)
        else:
            s.step(prefix, Q=int(r.integers(0, 65)) if page > 4 else int(r.integers(0, 4)))


def test_only_blocks_inside_a_page_are_emptied():
    # every page is handed out at once: a block over two pages keeps its scale, and so does one over the last page's end
    s = State(1, 7, 7, 100, block=64)
    s.cache.scales.fill_(5)
    s.host()
    s.step([699], Q=1)
    inside = [k * 64 // 100 == (k * 64 + 63) // 100 and k * 64 + 64 <= 700 for k in range(11)]
    assert inside[10] is False and s.h["words"] == [0 if i else 5 for i in inside]
    s = State(1, 40, 40, 1, block=8)
    s.cache.scales.fill_(3)
    s.host()
    s.step([39], Q=1)
    assert s.h["words"] == [3] * 5


def test_lengths_of_zero_and_one_and_borders():
    s = State(8, 10, 40, 4, block=4)
    s.step([0, 1, 3, 4, 5, 0, -1, 8], [0, 0, 1, 0, 3, 1, 5, 32])   # the last fills its row of the table
    s.step([0, 0, 0, 0, 0, 0, 0, 0], [0] * 8)                      # nothing is held any more
    assert s.h["held"] == [0] * 8
    s.step([-1] * 8, Q=3)
    s.step([40, -1, -1, -1, -1, -1, -1, 36], Q=0)


@pytest.mark.parametrize("B", [1, 2, 511, 512, 513, 1025, 4096])
def test_batches_around_the_blocks_threads(B):
    r = np.random.default_rng(B)
    s = State(B, 12, 12 * B, 8, block=8, seed=1)
    s.step([int(x) for x in r.integers(-1, 60, B)], Q=2)
    s.step([int(x) for x in r.integers(-1, 60, B)], [int(x) for x in r.integers(0, 30, B)])


def test_long_lists():
    # more positions than all threads list at once, in whole pages and in single slots
    for page, lens in ((16, [70_000, 3, -1, 250_000, 64]), (1, [100_001, 0, 17, -1, 90_000])):
        s = State(5, 260_000 // page, 360_000 // page, page, block=page)
        s.step(lens, Q=3)


def test_pages_so_large_that_the_sums_take_64_bits():
    s = State(3, 4, 7, 2 ** 28)
    s.step([2000, -1, 1500], [7, 0, 0])
    s.step([2 ** 28 - 1, 2 ** 28, 3], [2, 0, 1], status=CAPACITY, idx_len=100)


@pytest.mark.parametrize("page", [2 ** 31 - 1, 2 ** 30 + 1, 2 ** 31 - 1000])
def test_pages_of_nearly_2_to_the_31_slots(page):
    # one page is the pool: length + page_size passes 2^31 in every step, and what is held has to be right for the next
    s = State(2, 1, 1, page)
    s.step([0, -1], Q=11)
    s.step([2000, -1], Q=2)
    s.step([2000, 0], [0, 1], status=CAPACITY)   # the page is taken
    s.step([2002, -1], Q=0)


def test_pages_of_nearly_2_to_the_31_slots_change_hands():
    s = State(2, 1, 1, 2 ** 31 - 1)
    s.step([1, -1], Q=1)
    s.step([-1, -1], Q=1)
    s.step([-1, 70], Q=1)
    assert s.h["held"] == [0, 1]


@pytest.mark.parametrize("page,max_pages", [(2 ** 31 - 1, 1), (2 ** 30 + 1, 1), (100, 21_474_836), (4096, 2 ** 19 - 1)])
def test_lengths_near_2_to_the_31(page, max_pages):
    # the table's last page is partly used, then full, then all of it comes back; positions are not listed
    full = page * max_pages
    ti = api.kv_tables_alloc(1, max_pages, max_pages, page)
    slots = torch.zeros(1, dtype=torch.int32).cuda()
    for prefix, pages in ((full - page + 1, max_pages), (full - 9, max_pages), (full - 1, max_pages), (0, 1),
                          (full - 2, max_pages)):
        ti.prefix_lens = i32([prefix])
        assert api.kv8_check(api.kv_tables(ti, slots)) == 0
        assert ti.pages_held.tolist() == [pages]
        assert int(ti.free_state[1] - ti.free_state[0]) == max_pages - pages
        at = int(ti.block_table[0, prefix // page]) * page + prefix % page
        assert slots.tolist() == [at]


def test_tables_that_cannot_be_built_leave_everything():
    s = State(3, 8, 12, 4, block=4, head=7)
    s.step([10, 5, -1], Q=2)
    s.step([10, -2, -1], Q=2, status=PREFIX)
    s.step([10, 5, -1], [1, -1, 0], status=PREFIX)
    s.step([10, 31, -1], [1, 2, 0], status=PAGES)           # 33 positions, 8 pages of 4
    s.step([31, 31, 3], Q=1, status=CAPACITY)               # 17 pages of 12
    s.step([10, 5, -1], [2, 3, 0], status=CAPACITY, slots_len=4)
    s.step([10, 5, -1], [2, 3, 0], status=CAPACITY, idx_len=19)
    s.step([10, 5, -1], [2, 3, 0], idx_len=20, slots_len=5)
    held = s.ti.pages_held.clone()
    for bad in (-1, 9):
        s.ti.pages_held[1] = bad
        s.host()
        s.step([10, 5, -1], Q=1, status=PAGES)
    s.ti.pages_held.copy_(held)
    good = s.ti.free_state.clone()
    for head, tail in ((-1, 3), (9, 8), (0, 13)):
        s.ti.free_state.copy_(torch.tensor([head, tail, 0]))
        s.host()
        s.step([10, 5, -1], Q=1, status=PAGES)
    s.ti.free_state.copy_(good)
    s.host()
    s.step([10, 5, 3], Q=1)
    # a ring with too little room for the pages that come back
    small = State(2, 8, 12, 4)
    small.step([16, 8], Q=0)
    small.ti.free_ring = small.ti.free_ring[:8].contiguous()
    small.host()
    small.step([-1, -1], Q=0, status=CAPACITY)


def test_page_ids_outside_the_pool_are_reported():
    s = State(2, 8, 12, 4)
    s.step([10, 5], Q=1)
    s.ti.block_table[0, 1] = 12
    s.host()
    slots, ptr, idx = s.step([10, 5], Q=1, status=SLOT)
    assert idx[4:8].tolist() == [-1] * 4 and idx[:4].tolist() != [-1] * 4 and slots.min() >= 0
    s.ti.block_table[0, 1] = -3
    s.ti.free_ring[int(s.ti.free_state[0]) % 12] = 2 ** 31 - 1  # the next to be handed out
    s.host()
    slots, ptr, idx = s.step([10, 7], Q=2, status=SLOT)
    assert slots.tolist()[3] == -1


def test_outputs_may_be_left_out():
    s = State(3, 8, 24, 4, block=8)
    want = O.tables(4, 2, [9, -1, 3], None, s.h["table"], s.h["held"], s.h["ring"], s.h["state"], 24)
    s.ti.prefix_lens, s.ti.Q = i32([9, -1, 3]), 2
    ws = api.kv_tables(s.ti)
    assert api.kv8_check(ws) == 0
    words = s.h["words"]
    s.host()
    assert s.h["table"] == want["table"] and s.h["state"] == want["state"] and s.h["words"] == words


def test_captured_step_and_streams():
    # a captured call is replayed with new lengths; another stream's copy of the state takes the same steps
    a, b = State(6, 20, 120, 8, block=8, seed=3), State(6, 20, 120, 8, block=8, seed=3)
    ws = api.alloc_workspace(api.KV_TABLES_WORKSPACE_BYTES)
    slots, ptr = torch.zeros((6, 4), dtype=torch.int32).cuda(), torch.zeros(7, dtype=torch.int32).cuda()
    idx = torch.zeros(6 * 160, dtype=torch.int32).cuda()
    a.ti.Q = 4
    lens = torch.full((6,), -1, dtype=torch.int32).cuda()
    a.ti.prefix_lens = lens
    api.kv_tables(a.ti, slots, ptr, idx, cache=a.cache, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.kv_tables(a.ti, slots, ptr, idx, cache=a.cache, workspace=ws, check=False)
    s = torch.cuda.Stream()
    for prefix in ([0, 5, 7, 100, -1, 8], [4, 9, 11, 90, 3, -1], [-1] * 6, [150, 3, 0, 1, 2, 3]):
        lens.copy_(torch.tensor(prefix, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert api.kv8_check(ws) == 0
        sl, pt, ix = b.step(prefix, Q=4, stream=s)
        n = int(pt[-1])
        assert torch.equal(slots.view(-1), sl) and torch.equal(ptr, pt) and torch.equal(idx[:n], ix[:n])
        for x, y in zip(a.ti.tensors().values(), b.ti.tensors().values()):
            assert x is None or torch.equal(x, y)
        assert torch.equal(a.cache.scales, b.cache.scales)


@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("page", [1, 16])
def test_serving_loop_without_a_host_round_trip(page, H):
    """Chunks of prompts, then steps that draft a tree, get pages and slots for its nodes, write them, verify the tree
    over the cache, accept a path and move its rows behind the prefix; requests end and others take their pages.  The
    lengths never leave the device; the host only follows what it expects."""
    from mla_tree_verify_absorbed_gb300 import draft_inputs as DI
    rng = np.random.default_rng(1)
    B, budget, L = 3, 15, 6
    Q = budget + 1
    pages = 600 // page
    ti = api.kv_tables_alloc(B, 400 // page, pages, page)
    cache = api.kv8_alloc(pages * page, block=page if page > 1 else 8, exponent=-7)
    cap = 512
    slots, idx = torch.zeros(cap, dtype=torch.int32).cuda(), torch.zeros(3 * 400, dtype=torch.int32).cuda()
    ptr = torch.zeros(B + 1, dtype=torch.int32).cuda()
    prefix = torch.zeros(B, dtype=torch.int32).cuda()
    ti.prefix_lens = prefix
    ws, ws8 = api.alloc_workspace(1 << 14), api.alloc_workspace(1 << 14)
    truth = [np.zeros((0, 576)) for _ in range(B)]  # what the requests' positions were written with

    def rows(n):
        x = rng.standard_normal((n, 576)) * np.exp(0.5 * rng.standard_normal((n, 1)))
        return torch.from_numpy(x).to(torch.bfloat16)

    def prefill(lens):
        ti.new_lens = i32(lens)
        new = torch.zeros(cap, 576, dtype=torch.bfloat16)
        parts = [rows(n) for n in lens]
        new[:sum(lens)] = torch.cat(parts)
        new = new.cuda()
        api.kv_tables(ti, slots, ptr, idx, cache=cache, workspace=ws)
        api.kv8_write(cache, new[:, :512], new[:, 512:], slots, workspace=ws8)
        prefix.add_(ti.new_lens)
        assert api.kv8_check(ws) == 0 and api.kv8_check(ws8) == 0
        for b, x in enumerate(parts):
            truth[b] = np.concatenate([truth[b], x.double().numpy()])
        ti.new_lens = None

    prefill([130, 61, 0])
    for step in range(5):
        d = DI.make_draft(name="loop", B=B, L=L, K=4, budget=budget, seed=50 + step)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        parent, token, _, _, _ = api.ddtree_build(t(d.root_token), t(d.cand_token), t(d.cand_logp), budget)
        new = rows(B * Q)
        dev = new.cuda()
        q = torch.from_numpy(rng.standard_normal((B, Q, H, 576))).to(torch.bfloat16).cuda()
        # from here on to the accepted lengths nothing is read on the host
        ti.Q = Q
        node = slots[:B * Q].view(B, Q)
        api.kv_tables(ti, node, ptr, idx, cache=cache, workspace=ws)
        api.kv8_write(cache, dev[:, :512], dev[:, 512:], node.view(-1), workspace=ws8)
        ki = api.Kv8Inputs(B=B, Q=Q, H=H, scale=0.05, q_lat=q[..., :512].contiguous(), q_pe=q[..., 512:].contiguous(),
                           cache=cache, prefix_lens=prefix, page_size=page, tree_parent=parent, kv_indptr=ptr,
                           kv_indices=idx, block_table=ti.block_table)
        out, lse = api.kv8_attn(ki)
        flat, l1 = api.kv8_attn(dataclasses.replace(ki, page_size=1))  # the same through the flat tables
        n_len, nodes, _, _, _ = api.ddtree_accept(parent, token, t(DI.make_targets(d, parent.cpu().numpy(), seed=60 + step)))
        # accepted nodes' rows move to the positions behind the prefix: read back, then written
        pick = nodes.clamp(min=0).long()
        live = torch.arange(Q, device="cuda") < n_len[:, None]
        src = torch.where(live, torch.gather(node, 1, pick), -1)
        kept_c, kept_r, _ = api.kv8_read(cache, src.view(-1).contiguous())
        to = torch.where(live, node, -1)
        api.kv8_write(cache, kept_c, kept_r, to.view(-1).contiguous(), workspace=ws8)
        prefix.add_(n_len)
        assert api.kv8_check(ws) == 0 and api.kv8_check(ws8) == 0
        # what came out is the attention over what was written
        host_idx, host_ptr, par = idx.cpu().numpy(), ptr.cpu().numpy(), parent.cpu().numpy()
        words = cache.scales.cpu().numpy()
        for b in range(B):
            P = len(truth[b])
            x = np.concatenate([truth[b], new[b * Q:(b + 1) * Q].double().numpy()])
            assert host_ptr[b + 1] - host_ptr[b] == P + Q
            at = host_idx[host_ptr[b]:host_ptr[b + 1]]
            unit = 2.0 ** (cache.exponent + words[at // cache.block] - 1)[:, None]
            o, l, mag, _ = O.attention(x[:, :512], x[:, 512:], q[b, ..., :512].double().cpu().numpy(),
                                       q[b, ..., 512:].double().cpu().numpy(), 0.05, par[b], P, H)
            # each latent is within half a step of what was written: 2^-4 of it, or 2^-10 units (twice, where a
            # block has grown since or a row has moved)
            err = 2 * np.maximum(2.0 ** -4 * np.abs(x[:, :512]), 2.0 ** -10 * unit)
            ds = 0.05 * np.einsum("qhc,nc->qhn", np.abs(q[b, ..., :512].double().cpu().numpy()), err).max(-1)
            assert (np.abs(l - lse[b].double().cpu().numpy()) <= ds + 1e-3).all()
            f = np.expm1(2 * ds)[..., None] + 2.0 ** -7
            tol = f * mag + (1 + f) * err.max()
            assert (np.abs(o - out[b].double().cpu().numpy()) <= tol).all()
        assert torch.equal(lse, l1) and torch.equal(out, flat)
        for b in range(B):
            take = nodes[b, :int(n_len[b])].tolist()
            truth[b] = np.concatenate([truth[b], new[b * Q:(b + 1) * Q].double().numpy()[take]])
        if step == 1:  # a request ends, and its row of the batch takes another prompt
            prefix[0] = -1
            ti.Q = 0
            api.kv_tables(ti, workspace=ws, cache=cache)
            assert api.kv8_check(ws) == 0 and int(ti.pages_held[0]) == 0
            prefix[0] = 0
            truth[0] = np.zeros((0, 576))
            prefill([99, 0, 40])
    # every page is somewhere, once
    held = [ti.block_table[b, :int(ti.pages_held[b])].tolist() for b in range(B)]
    head, tail = ti.free_state[:2].tolist()
    free = [int(ti.free_ring[i % pages]) for i in range(head, tail)]
    assert sorted(sum(held, free)) == list(range(pages))
