"""The paged 8-bit latent cache and the page tables without a GPU: the oracle's
pins, and what the library and its binding refuse before anything is launched."""
import ctypes
import dataclasses
import os
import re

import numpy as np
import pytest

from mla_tree_verify_absorbed_gb300 import api, build as B
from oracle import kv8 as O


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.load()


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
def test_code_table():
    assert O.e4m3_value(0x38) == 1.0 and O.e4m3_value(0xb8) == -1.0 and O.e4m3_value(0x01) == 2.0 ** -9
    assert O.e4m3_value(0x7e) == 448 and np.isnan(O.e4m3_value(0x7f)) and np.isnan(O.e4m3_value(0xff))
    assert (np.diff(O.POSITIVE) > 0).all()


def test_nearest_code_hand_worked():
    # 1 and 1.125 are neighbours: their midpoint goes to the even code, that of 1.125 and 1.25 too
    assert O.nearest_code(1.0625) == 0x38 and O.nearest_code(1.1875) == 0x3a
    assert O.nearest_code(1.0626) == 0x39 and O.nearest_code(-1.0626) == 0xb9
    assert O.nearest_code(1e9) == 0x7e and O.nearest_code(-np.inf) == 0xfe and O.nearest_code(np.nan) == 0
    assert O.nearest_code(2.0 ** -10) == 0 and O.nearest_code(1.5 * 2.0 ** -9) == 2 and O.nearest_code(-0.0) == 0x80
    r = np.random.default_rng(0)
    x = np.concatenate([r.standard_normal(400) * 2.0 ** r.integers(-14, 12, 400), O.VALUES[:127],
                        (O.POSITIVE[1:] + O.POSITIVE[:-1]) / 2, [np.nan, np.inf, -0.0]])
    assert O.nearest_codes(x).tolist() == [O.nearest_code(v) for v in x]


def test_needed_scale_hand_worked():
    assert O.needed([448.0], 0) == 0 and O.needed([448.5], 0) == 1 and O.needed([-896.0], 0) == 1
    assert O.needed([7.0], -6) == 0 and O.needed([7.5], -6) == 1 and O.needed([0.0], -32) == 0
    assert O.needed([1e30], 0) == 15 and O.needed([np.inf, 500.0, np.nan], 0) == 1


def test_write_hand_worked():
    rows, words = np.zeros((6, 640), np.uint8), np.zeros(3, np.int64)
    one = np.ones((1, 512)) * 448
    rows, words = O.write(rows, words, 2, 0, one, np.full((1, 64), 3.0), [2])
    assert words.tolist() == [0, 1, 0] and (rows[2, :512] == 0x7e).all()
    # a neighbour that needs twice the unit: the first row's codes are halved, its values stay
    rows, words = O.write(rows, words, 2, 0, one * 2, np.full((1, 64), 1.0), [3])
    assert words.tolist() == [0, 2, 0] and (rows[2, :512] == O.nearest_code(224.0)).all()
    lat, rope = O.unpack_rows(rows[2:4], [1, 1])
    assert (lat[0] == 448).all() and (lat[1] == 896).all() and (rope[0] == 3).all() and (rope[1] == 1).all()
    # a smaller row changes nothing but itself
    again, w2 = O.write(rows, words, 2, 0, one / 448, np.zeros((1, 64)), [3])
    assert w2.tolist() == words.tolist() and np.array_equal(again[2], rows[2])


def test_bf16_rounding():
    x = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -3.1415926, 0.0, 65280.0])
    assert O.bf16_bits(x).tolist() == [0x3f80, 0x3f80, 0x3f82, 0xc049, 0, 0x477f]
    assert O.bf16_value(O.bf16_bits(x))[2] == 1 + 2.0 ** -6


def test_tables_hand_worked():
    # two requests of 4-slot pages: the first grows into a second page, the second has ended
    t = O.tables(4, 2, [3, -1], None, [[5, -1], [7, 8]], [1, 2], [1, 2, 3, 9], [6, 8, 0], 10)
    assert t["table"] == [[5, 3], [-1, -1]] and t["held"] == [2, 0]
    assert t["ring"] == [7, 8, 3, 9] and t["state"] == [7, 10, 0]  # entry 6 % 4 is taken, 8 and 9 are filled
    assert t["slots"] == [23, 12, -1, -1] and t["ptr"] == [0, 5, 5] and t["idx"] == [20, 21, 22, 23, 12]


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_struct_layout_matches_header(lib):
    A, C, T = api.MlaKv8AttnArgs, api.MlaKv8Cache, api.MlaKvTablesArgs
    assert C.scales.offset == 24 and C.block.offset == 32 and C.exponent.offset == 36 and ctypes.sizeof(C) == 40
    assert A.cache.offset == 16 and A.q_lat.offset == 56 and A.page_size.offset == 72 and A.out.offset == 144
    assert ctypes.sizeof(A) == 160
    assert T.prefix_lens.offset == 24 and T.ring.offset == 72 and T.slots_len.offset == 88 and T.scales.offset == 120
    assert ctypes.sizeof(T) == 136


def cache_struct(**kw):
    c = api.MlaKv8Cache(0x100000, 640, 1000, 0x180000, 64, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rows_struct(**kw):
    r = api.MlaKvqRows(10, api.MLA_BF16, 0x200000, 0x300000, 512, 64, 0x400000)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def attn_struct(**kw):
    a = api.MlaKv8AttnArgs(2, 4, 8, cache_struct(), 0x200000, 0x300000, 1, 0x400000, 0x410000, None, 0, 0x420000,
                           0x430000, 0, 0, 0.07, 0x500000, 0x600000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHE = [("rows", None), ("rows", 0x100010), ("row_stride", 608), ("row_stride", 656), ("row_stride", 1 << 32),
             ("slots", 0), ("slots", 1 << 31), ("exponent", 33), ("exponent", -33), ("scales", None),
             ("scales", 0x180002), ("block", 0), ("block", -1)]


@pytest.mark.parametrize("f", ["mla_kv8_write", "mla_kv8_read"])
def test_io_refusals(lib, f):
    f = getattr(lib, f)

    def call(c, r, ws=0x700000, n=api.KV8_WORKSPACE_BYTES):
        return f(c and ctypes.byref(c), r and ctypes.byref(r), ctypes.c_void_p(ws), ctypes.c_size_t(n), None)

    for k, v in BAD_CACHE:
        assert call(cache_struct(**{k: v}), rows_struct()) == api.MLA_ERR_INVALID_ARG, (k, v)
    for k, v in [("n", -1), ("n", 1 << 31), ("dtype", 2), ("kv_c", None), ("k_pe", None), ("slots", None),
                 ("kv_c", 0x200008), ("k_pe", 0x300008), ("slots", 0x400002), ("kv_c_stride", 504),
                 ("kv_c_stride", 516), ("k_pe_stride", 56), ("k_pe_stride", 68), ("kv_c_stride", 1 << 32)]:
        assert call(cache_struct(), rows_struct(**{k: v})) == api.MLA_ERR_INVALID_ARG, (k, v)
    assert call(None, rows_struct()) == api.MLA_ERR_INVALID_ARG
    assert call(cache_struct(), None) == api.MLA_ERR_INVALID_ARG
    assert call(cache_struct(), rows_struct(), ws=0) == api.MLA_ERR_WORKSPACE
    assert call(cache_struct(), rows_struct(), ws=0x700010) == api.MLA_ERR_WORKSPACE
    assert call(cache_struct(), rows_struct(), n=api.KV8_WORKSPACE_BYTES - 1) == api.MLA_ERR_WORKSPACE
    # nothing to do: nothing is looked at but the cache
    assert call(cache_struct(), rows_struct(n=0, kv_c=None, slots=None), ws=0, n=0) == api.MLA_OK


def attn_call(lib, a, ws=0x700000, n=1 << 40):
    return lib.mla_kv8_attn(ctypes.byref(a), ctypes.c_void_p(ws), ctypes.c_size_t(n), None)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, api.MLA_ERR_INVALID_ARG), ("Q", -1, api.MLA_ERR_INVALID_ARG), ("H", 0, api.MLA_ERR_INVALID_ARG),
    ("Q", 65, api.MLA_ERR_UNSUPPORTED), ("H", 1 << 24, api.MLA_ERR_UNSUPPORTED),
])
def test_attn_shape_refusals(lib, field, value, status):
    a = attn_struct(**{field: value})
    assert attn_call(lib, a) == status
    assert lib.mla_kv8_attn_workspace_size(ctypes.byref(a)) == 0


@pytest.mark.parametrize("field,value", [
    ("q_lat", None), ("q_pe", None), ("q_lat", 0x200008), ("out", None), ("out", 0x500008), ("prefix_lens", None),
    ("prefix_lens", 0x420002), ("tree_parent", 0x430002), ("lse", 0x600002), ("page_size", 0), ("kv_indptr", None),
    ("kv_indices", None), ("kv_indices", 0x410001), ("page_size", 64), ("window", -1), ("sinks", -1), ("sinks", 4),
    ("scale", 0.0), ("scale", -1.0), ("scale", float("nan")), ("scale", float("inf")),
])
def test_attn_argument_refusals(lib, field, value):
    assert attn_call(lib, attn_struct(**{field: value})) == api.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("scale,exponent", [(1e-38, -32), (1e-30, -32), (3e38, 0), (1e30, 32), (1e-40, 0)])
def test_attn_refuses_a_scale_that_leaves_fp32(lib, scale, exponent):
    assert attn_call(lib, attn_struct(scale=scale, cache=cache_struct(exponent=exponent))) == api.MLA_ERR_INVALID_ARG
    back = 20 if scale < 1 else -20
    assert attn_call(lib, attn_struct(scale=scale, cache=cache_struct(exponent=back)), ws=0) == api.MLA_ERR_WORKSPACE


def test_attn_cache_and_table_refusals(lib):
    for k, v in BAD_CACHE:
        assert attn_call(lib, attn_struct(cache=cache_struct(**{k: v}))) == api.MLA_ERR_INVALID_ARG, (k, v)
    paged = dict(page_size=64, block_table=0x440000, kv_indptr=None, kv_indices=None)
    assert attn_call(lib, attn_struct(**paged, max_pages=0)) == api.MLA_ERR_INVALID_ARG
    assert attn_call(lib, attn_struct(**paged, max_pages=1 << 26)) == api.MLA_ERR_INVALID_ARG
    assert attn_call(lib, attn_struct(**{**paged, "block_table": 0x440001}, max_pages=8)) == api.MLA_ERR_INVALID_ARG
    assert lib.mla_kv8_attn(None, None, 0, None) == api.MLA_ERR_INVALID_ARG


def test_attn_workspace_and_noop(lib):
    assert attn_call(lib, attn_struct(), ws=0) == api.MLA_ERR_WORKSPACE
    assert attn_call(lib, attn_struct(), ws=0x700010) == api.MLA_ERR_WORKSPACE
    assert attn_call(lib, attn_struct(), n=100) == api.MLA_ERR_WORKSPACE
    for kw in (dict(B=0), dict(Q=0)):
        assert attn_call(lib, attn_struct(**kw), ws=0, n=0) == api.MLA_OK
    assert lib.mla_kv8_check(None, None, None) == api.MLA_ERR_WORKSPACE


def test_selftest_timeout_refusals(lib):
    def call(a, hold, ws=0x700000, n=1 << 40):
        return lib.mla_kv8_selftest_timeout(ctypes.byref(a), ctypes.c_void_p(ws), ctypes.c_size_t(n),
                                            ctypes.c_uint64(hold), None)
    for hold in (0, 1_000_000_001, 2 ** 63):
        assert call(attn_struct(), hold) == api.MLA_ERR_INVALID_ARG
    for kw in (dict(B=0), dict(Q=0), dict(H=0), dict(q_lat=None), dict(page_size=0)):
        assert call(attn_struct(**kw), 1000) == api.MLA_ERR_INVALID_ARG, kw
    assert call(attn_struct(Q=65), 1000) == api.MLA_ERR_UNSUPPORTED
    assert call(attn_struct(), 1000, ws=0) == api.MLA_ERR_WORKSPACE


def tables_struct(**kw):
    a = api.MlaKvTablesArgs(4, 2, 16, 100, 1000, 0x100000, None, 0x200000, 0x300000, 0x400000, 0x500000, 1000,
                            0x600000, 8, 0x700000, 0x800000, 5000, 0x900000, 16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, 1), ("Q", -1, 1), ("page_size", 0, 1), ("max_pages", 0, 1), ("num_pages", 0, 1), ("ring", 0, 1),
    ("B", 4097, 2), ("max_pages", 1 << 28, 1), ("num_pages", 1 << 28, 1), ("prefix_lens", None, 1),
    ("block_table", None, 1), ("pages_held", None, 1), ("free_ring", None, 1), ("free_state", None, 1),
    ("free_state", 0x500004, 1), ("prefix_lens", 0x100002, 1), ("new_lens", 0x100001, 1), ("slots", 0x600002, 1),
    ("kv_indptr", 0x700002, 1), ("kv_indices", 0x800001, 1), ("scales", 0x900002, 1), ("slots_len", 7, 1),
    ("slots_len", 9, 1), ("indices_len", -1, 1), ("indices_len", 1 << 31, 1), ("block", 0, 1),
])
def test_tables_refusals(lib, field, value, status):
    def call(a, ws=0xa00000, n=api.KV_TABLES_WORKSPACE_BYTES):
        return lib.mla_kv_tables(ctypes.byref(a), ctypes.c_void_p(ws), ctypes.c_size_t(n), None)
    assert call(tables_struct(**{field: value})) == status
    assert call(tables_struct(), ws=0) == api.MLA_ERR_WORKSPACE
    assert call(tables_struct(), n=100) == api.MLA_ERR_WORKSPACE
    assert call(tables_struct(B=0, prefix_lens=None), ws=0, n=0) == api.MLA_OK
    assert lib.mla_kv_tables(None, None, 0, None) == api.MLA_ERR_INVALID_ARG


def test_binding_refuses_wrong_tensors(lib):
    torch = pytest.importorskip("torch")
    cache = api.kv8_alloc(20, block=8, device="cpu")
    assert cache.scales.shape == (3,)
    c, k = torch.zeros(6, 512, dtype=torch.bfloat16), torch.zeros(6, 64, dtype=torch.bfloat16)
    s = torch.zeros(6, dtype=torch.int32)
    for bad in (dict(kv_c=c.half()), dict(kv_c=c.float()), dict(kv_c=c[:, :256]), dict(k_pe=k[:5]),
                dict(slots=s.long()), dict(slots=s[:5]), dict(kv_c=c.t().contiguous().t()),
                dict(kv_c=c[:1].expand(6, 512))):
        with pytest.raises(ValueError):
            api.kv8_write(**{**dict(cache=cache, kv_c=c, k_pe=k, slots=s), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        api.kv8_write(cache, c, k, s)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv8_read(cache, s)
    for bad in (dict(rows=torch.zeros(20, 416, dtype=torch.uint8)), dict(rows=torch.zeros(20, 640, dtype=torch.int8)),
                dict(rows=torch.zeros(1, 640, dtype=torch.uint8).expand(20, 640)), dict(scales=cache.scales.long()),
                dict(scales=cache.scales[:2]), dict(scales=None), dict(block=0), dict(block=7), dict(exponent=40)):
        with pytest.raises(ValueError):
            api.kv8_write(dataclasses.replace(cache, **bad), c, k, s)
    ki = api.Kv8Inputs(B=2, Q=1, H=4, scale=0.1, q_lat=torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16),
                       q_pe=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), cache=cache,
                       prefix_lens=torch.zeros(2, dtype=torch.int32), page_size=1,
                       kv_indptr=torch.zeros(3, dtype=torch.int32), kv_indices=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.kv8_attn(ki)
    for bad in (dict(q_lat=ki.q_lat.float()), dict(q_pe=ki.q_pe[:1]), dict(prefix_lens=ki.prefix_lens.long()),
                dict(kv_indptr=ki.kv_indptr[:2]), dict(kv_indices=None), dict(page_size=16),
                dict(tree_parent=torch.zeros(2, 2, dtype=torch.int32)), dict(window=2 ** 32 + 5)):
        with pytest.raises(ValueError):
            api.kv8_attn(dataclasses.replace(ki, **bad))
    with pytest.raises(ValueError, match="dtype"):
        api.kv8_read(cache, s, "fp16")


def test_tables_binding_refuses_wrong_tensors(lib):
    torch = pytest.importorskip("torch")
    ti = api.kv_tables_alloc(3, 8, 20, 4, device="cpu")
    assert ti.free_state.tolist() == [0, 20, 0] and (ti.prefix_lens == -1).all()
    i32 = dict(dtype=torch.int32)
    slots, idx, ptr = torch.zeros(3, 1, **i32), torch.zeros(50, **i32), torch.zeros(4, **i32)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv_tables(ti, slots, ptr, idx)
    for bad in (dict(block_table=ti.block_table.long()), dict(block_table=ti.block_table[:, ::2]),
                dict(prefix_lens=ti.prefix_lens[:2]), dict(pages_held=ti.pages_held.long()),
                dict(free_state=ti.free_state[:2]), dict(free_ring=ti.free_ring.view(4, 5)),
                dict(new_lens=torch.zeros(2, **i32)), dict(num_pages=2 ** 40), dict(Q=2)):
        with pytest.raises(ValueError):
            api.kv_tables(dataclasses.replace(ti, **bad), slots, ptr, idx)
    for bad in (dict(slots=slots.long()), dict(slots=torch.zeros(4, **i32)), dict(kv_indptr=ptr[:3]),
                dict(kv_indices=idx.view(5, 10)), dict(cache=api.kv8_alloc(79, block=4, device="cpu"))):
        with pytest.raises(ValueError):
            api.kv_tables(ti, **{**dict(slots=slots, kv_indptr=ptr, kv_indices=idx), **bad})


# ---------------------------------------------------------------------------
# arithmetic and orderings that a run on one chip cannot show
# ---------------------------------------------------------------------------
def test_three_bytes_hold_a_weight():
    # the terms that the kernels cut off an f16 weight: upper byte, upper byte of the rest, rounded rest
    w = np.arange(0x0001, 0x7800, dtype=np.uint16)  # every positive f16 number up to 2^15

    def f(u):
        return u.astype(np.uint16).view(np.float16).astype(np.float64)
    t1 = w & 0xff00
    r1 = f(w) - f(t1)
    r1h = r1.astype(np.float16)
    assert np.array_equal(r1h.astype(np.float64), r1)  # exact
    t2 = r1h.view(np.uint16) & 0xff00
    r2 = r1 - f(t2)
    r2h = r2.astype(np.float16)
    assert np.array_equal(r2h.astype(np.float64), r2)
    t3 = (r2h.view(np.uint16) + 0x80) & 0xff00
    err = np.abs(f(w) - f(t1) - f(t2) - f(t3))
    assert (err <= np.maximum(2.0 ** -9 * f(w), 2.0 ** -17)).all()


def test_three_scaled_bytes_hold_a_weight():
    # the kernel for few rows: what a byte leaves is taken times 2^3, exactly
    w = np.arange(0x0001, 0x7801, dtype=np.uint16)  # every positive f16 number up to 2^15

    def f(u):
        return u.astype(np.uint16).view(np.float16).astype(np.float64)

    def rest(u):
        r = 8 * (f(u) - f(u & 0xff00))
        h = r.astype(np.float16)
        assert np.array_equal(h.astype(np.float64), r)
        return h.view(np.uint16)
    r1 = rest(w)
    r2 = rest(r1)
    t3 = (r2 + 0x80) & 0xff00
    assert (f(t3) <= 2.0 ** 15).all()
    err = np.abs(f(w) - f(w & 0xff00) - f(r1 & 0xff00) / 8 - f(t3) / 64)
    assert (err <= np.maximum(2.0 ** -9 * f(w), 2.0 ** -23)).all()
    assert (err <= f(w)).all()


def test_two_codes_hold_a_query():
    # every bf16 significand at every exponent, in a row whose largest element is scaled to 448 or 255: hi keeps
    # sign, exponent and 3 bits, lo the other 4
    for top in (1.75, 1.9921875):
        t = 8 if top == 1.75 else 7
        m = 1 + np.arange(128) / 128
        for e in range(-30, 1):
            x = m * 2.0 ** e
            if e == 0:
                x = x[x <= top]
            u = x.astype(np.float32).view(np.uint32)
            hi = (u & 0xfff00000).view(np.float32).astype(np.float64)
            got = O.VALUES[O.nearest_codes(hi * 2.0 ** t)] + O.VALUES[O.nearest_codes((x - hi) * 2.0 ** t)]
            err = np.abs(got - x * 2.0 ** t)
            assert err.max() <= 2.0 ** -9 and (err[x * 2.0 ** t >= 0.25] == 0).all()


def test_relaxed_cluster_arrivals_follow_no_loads():
    # as for the 4-bit cache's kernel: a relaxed arrive on another CTA's barrier may only pass on what another
    # barrier has said; the signals about the row sums release
    src = open(os.path.join(B.CSRC, "kv8_rows.cu")).read()
    assert set(re.findall(r"mbar_arrive_cluster_relaxed\(&c->(\w+)", src)) == {"ps_free"}
    assert set(re.findall(r"mbar_arrive_cluster\(&c->(\w+)", src)) == {"fin_free", "fin_full"}
