"""The 4-bit latent cache without a GPU: the oracle's pins, and what the
library and its binding refuse before anything is launched."""
import ctypes
import os
import re

import numpy as np
import pytest

from mla_tree_verify_absorbed_gb300 import api, build as B
from oracle import kvq as O


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.load()


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
def test_scale_table():
    # three spot values, monotone, and the ends of the e4m3 range
    assert O.e4m3_value(0x38) == 1.0 and O.e4m3_value(0x01) == 2.0 ** -9 and O.e4m3_value(0x45) == 3.25
    assert (np.diff(O.SCALES) > 0).all() and O.SCALES[0] == 0 and O.SCALES[-1] == 448


def test_quantise_hand_worked():
    # max 7 -> scale 1: whole numbers are themselves, halves go to the even neighbour
    x = np.array([7, -7, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 6.5, 0.49, 0.51, 3, -4, 0, 1, -6.5])
    codes, byte = O.quantise_block(x, 0)
    assert byte == 0x38
    assert [c - 8 for c in codes] == [7, -7, 0, 2, 2, 0, -2, -2, 6, 0, 1, 3, -4, 0, 1, -6]
    # a power of two moves the scale's exponent only, and `exponent` takes it back
    assert O.quantise_block(x * 4, 0) == (codes, 0x48)
    assert O.quantise_block(x * 4, 2) == (codes, 0x38)
    # nothing above 448 * 7, nothing but zeros below half the smallest scale
    assert O.quantise_block(np.full(16, 1e9), 0) == ([15] * 16, 0x7e)
    assert O.quantise_block(np.full(16, 7 * 2.0 ** -10), 0) == ([8] * 16, 0)  # the tie goes to scale 0


def test_pack_unpack_positions():
    # one non-zero latent at a time lands in the word and nibble of the layout
    for e, byte, high in ((0, 0, 0), (1, 2, 0), (2, 0, 1), (7, 3, 1), (8, 4, 0), (511, 255, 1)):
        x = np.zeros(512)
        x[e] = 7.0
        row = O.pack_row(x, np.zeros(64, np.uint16))
        assert (row[byte] >> (4 * high)) & 15 == 15
        assert np.array_equal(O.unpack_row(row)[0], x)
    rng = np.random.default_rng(0)
    rows = rng.integers(0, 256, (5, 416), dtype=np.uint8)
    rows[:, 289::2] &= 0x3f  # finite rope keys
    many = O.unpack_rows(rows, -3)
    for r, a, b in zip(rows, *many):
        one = O.unpack_row(r, -3)
        assert np.array_equal(one[0], a) and np.array_equal(one[1], b)
    assert np.isfinite(many[0]).all()


def test_visible_hand_worked():
    chain = [-1, 0, 1, 2]
    tree = [-1, 0, 0, 1, -1]
    assert O.visible(chain, 2, 5) == [0, 1, 2, 3, 4, 5, 6, 7]
    assert O.visible(tree, 3, 2) == [0, 1, 2, 3, 5]
    assert O.visible(tree, 4, 2) == [0, 1, 6]
    # node 3 stands at place 2 + 2: a window of 3 keeps places 2, 3, 4
    assert O.visible(tree, 3, 2, window=3) == [2, 3, 5]
    assert O.visible(tree, 3, 2, window=1) == [5]
    assert O.visible(tree, 3, 2, window=1, sinks=1) == [0, 5]
    assert O.visible(tree, 3, 2, window=1, sinks=3) == [0, 1, 2, 5]  # node 0 stands at place 2
    assert O.visible(chain, 0, 9, window=4, sinks=2) == [0, 1, 6, 7, 8, 9]


def test_attention_of_equal_rows_is_the_row():
    rng = np.random.default_rng(1)
    v = rng.standard_normal(512)
    out, lse, mag, _ = O.attention(np.tile(v, (7, 1)), np.zeros((7, 64)), rng.standard_normal((2, 3, 512)),
                                   rng.standard_normal((2, 3, 64)), 0.1, [-1, 0], 5, 3)
    assert np.allclose(out, v, atol=1e-12) and np.allclose(mag, np.abs(v), atol=1e-12)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_struct_layout_matches_header(lib):
    A, R, C = api.MlaKvqAttnArgs, api.MlaKvqRows, api.MlaKvqCache
    assert ctypes.sizeof(C) == 32 and C.exponent.offset == 24
    assert R.kv_c.offset == 16 and R.slots.offset == 48 and ctypes.sizeof(R) == 56
    assert A.cache.offset == 16 and A.q_lat.offset == 48 and A.page_size.offset == 64
    assert A.block_table.offset == 88 and A.prefix_lens.offset == 104 and A.window.offset == 120
    assert A.scale.offset == 128 and A.out.offset == 136 and ctypes.sizeof(A) == 152


def cache_struct(**kw):
    c = api.MlaKvqCache(0x100000, 416, 1000, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rows_struct(**kw):
    r = api.MlaKvqRows(10, api.MLA_BF16, 0x200000, 0x300000, 512, 64, 0x400000)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def attn_struct(**kw):
    a = api.MlaKvqAttnArgs(2, 4, 8, cache_struct(), 0x200000, 0x300000, 1, 0x400000, 0x410000, None, 0, 0x420000,
                           0x430000, 0, 0, 0.07, 0x500000, 0x600000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHE = [("rows", None), ("rows", 0x100010), ("row_stride", 400), ("row_stride", 432), ("row_stride", 1 << 32),
             ("slots", 0), ("slots", 1 << 31), ("exponent", 33), ("exponent", -33)]


@pytest.mark.parametrize("f", ["mla_kvq_write", "mla_kvq_read"])
def test_io_refusals(lib, f):
    f = getattr(lib, f)

    def call(c, r, ws=0x700000, n=api.KVQ_WORKSPACE_BYTES):
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
    assert call(cache_struct(), rows_struct(), n=api.KVQ_WORKSPACE_BYTES - 1) == api.MLA_ERR_WORKSPACE
    # nothing to do: nothing is looked at but the cache
    assert call(cache_struct(), rows_struct(n=0, kv_c=None, slots=None), ws=0, n=0) == api.MLA_OK


def attn_call(lib, a, ws=0x700000, n=1 << 40):
    return lib.mla_kvq_attn(ctypes.byref(a), ctypes.c_void_p(ws), ctypes.c_size_t(n), None)


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, api.MLA_ERR_INVALID_ARG), ("Q", -1, api.MLA_ERR_INVALID_ARG), ("H", 0, api.MLA_ERR_INVALID_ARG),
    ("Q", 65, api.MLA_ERR_UNSUPPORTED), ("H", 1 << 24, api.MLA_ERR_UNSUPPORTED),
])
def test_attn_shape_refusals(lib, field, value, status):
    a = attn_struct(**{field: value})
    assert attn_call(lib, a) == status
    assert lib.mla_kvq_attn_workspace_size(ctypes.byref(a)) == 0


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
    # with the cache's exponent and log2(e) it would round to a subnormal, 0 or infinity
    assert attn_call(lib, attn_struct(scale=scale, cache=cache_struct(exponent=exponent))) == api.MLA_ERR_INVALID_ARG
    assert attn_call(lib, attn_struct(scale=scale, cache=cache_struct(exponent=exponent)), ws=0) \
        == api.MLA_ERR_INVALID_ARG
    # the exponent that brings it back into range is taken
    back = 20 if scale < 1 else -20
    assert attn_call(lib, attn_struct(scale=scale, cache=cache_struct(exponent=back)), ws=0) == api.MLA_ERR_WORKSPACE


def test_page_of_a_position_by_multiplication():
    # the kernel's pos * ceil(2^(31 + L) / page) >> (31 + L), 2^(L - 1) < page <= 2^L, for every border that could fail
    rng = np.random.default_rng(5)
    pages = {1, 2, 3, 7, 2 ** 30, 2 ** 30 + 1, 2 ** 31 - 1}
    pages |= {int(2 ** e) for e in rng.uniform(0, 31, 400)} | {2 ** k + d for k in range(2, 31) for d in (-1, 0, 1)}
    for page in pages:
        L = (page - 1).bit_length()
        mul = -(-2 ** (31 + L) // page)
        assert mul < 2 ** 32
        last = (2 ** 31 - 1) // page
        for k in {0, 1, 2, last // 2, last, *map(int, rng.integers(0, last + 1, 20))}:
            for pos in (k * page - 1, k * page, k * page + page - 1):
                if 0 <= pos < 2 ** 31:
                    assert pos * mul >> (31 + L) == pos // page


def test_attn_cache_and_table_refusals(lib):
    for k, v in BAD_CACHE:
        assert attn_call(lib, attn_struct(cache=cache_struct(**{k: v}))) == api.MLA_ERR_INVALID_ARG, (k, v)
    paged = dict(page_size=64, block_table=0x440000, kv_indptr=None, kv_indices=None)
    assert attn_call(lib, attn_struct(**paged, max_pages=0)) == api.MLA_ERR_INVALID_ARG
    assert attn_call(lib, attn_struct(**paged, max_pages=1 << 26)) == api.MLA_ERR_INVALID_ARG
    assert attn_call(lib, attn_struct(**{**paged, "block_table": 0x440001}, max_pages=8)) == api.MLA_ERR_INVALID_ARG
    assert lib.mla_kvq_attn(None, None, 0, None) == api.MLA_ERR_INVALID_ARG


def test_attn_workspace_and_noop(lib):
    assert attn_call(lib, attn_struct(), ws=0) == api.MLA_ERR_WORKSPACE
    assert attn_call(lib, attn_struct(), ws=0x700010) == api.MLA_ERR_WORKSPACE
    assert attn_call(lib, attn_struct(), n=100) == api.MLA_ERR_WORKSPACE
    for kw in (dict(B=0), dict(Q=0)):
        assert attn_call(lib, attn_struct(**kw), ws=0, n=0) == api.MLA_OK
    assert lib.mla_kvq_check(None, None, None) == api.MLA_ERR_WORKSPACE


def test_empty_kv_indices_are_refused(lib):
    # a batch without a used sequence needs none, but an empty tensor has no address
    torch = pytest.importorskip("torch")
    ki = api.KvqInputs(B=1, Q=1, H=1, scale=0.1, q_lat=torch.zeros(1, 1, 1, 512, dtype=torch.bfloat16),
                       q_pe=torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), cache=api.kvq_alloc(4, device="cpu"),
                       prefix_lens=torch.full((1,), -1, dtype=torch.int32), page_size=1,
                       kv_indptr=torch.zeros(2, dtype=torch.int32), kv_indices=torch.zeros(0, dtype=torch.int32))
    ki.check_layout()
    out, lse = torch.zeros(1, 1, 1, 512, dtype=torch.bfloat16), torch.zeros(1, 1, 1)
    assert attn_call(lib, ki.c_args(out, lse)) == api.MLA_ERR_INVALID_ARG


def test_selftest_timeout_refusals(lib):
    def call(a, hold, ws=0x700000, n=1 << 40):
        return lib.mla_kvq_selftest_timeout(ctypes.byref(a), ctypes.c_void_p(ws), ctypes.c_size_t(n),
                                            ctypes.c_uint64(hold), None)
    for hold in (0, 1_000_000_001, 2 ** 63):
        assert call(attn_struct(), hold) == api.MLA_ERR_INVALID_ARG
    for kw in (dict(B=0), dict(Q=0), dict(H=0), dict(q_lat=None), dict(page_size=0)):
        assert call(attn_struct(**kw), 1000) == api.MLA_ERR_INVALID_ARG, kw
    assert call(attn_struct(Q=65), 1000) == api.MLA_ERR_UNSUPPORTED
    assert call(attn_struct(), 1000, ws=0) == api.MLA_ERR_WORKSPACE
    assert call(attn_struct(), 1000, n=100) == api.MLA_ERR_WORKSPACE


def test_binding_refuses_wrong_tensors(lib):
    torch = pytest.importorskip("torch")
    import dataclasses
    cache = api.kvq_alloc(20, device="cpu")
    c, k = torch.zeros(6, 512, dtype=torch.bfloat16), torch.zeros(6, 64, dtype=torch.bfloat16)
    s = torch.zeros(6, dtype=torch.int32)
    for bad in (dict(kv_c=c.half()), dict(kv_c=c.float()), dict(kv_c=c[:, :256]), dict(k_pe=k[:5]),
                dict(slots=s.long()), dict(slots=s[:5]), dict(kv_c=c.t().contiguous().t()),
                dict(kv_c=c[:1].expand(6, 512))):
        with pytest.raises(ValueError):
            api.kvq_write(**{**dict(cache=cache, kv_c=c, k_pe=k, slots=s), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        api.kvq_write(cache, c, k, s)
    with pytest.raises(ValueError, match="CUDA"):
        api.kvq_read(cache, s)
    for bad in (torch.zeros(20, 400, dtype=torch.uint8), torch.zeros(20, 416, dtype=torch.int8),
                torch.zeros(416, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="cache rows"):
            api.kvq_write(api.QuantCache(bad), c, k, s)
    with pytest.raises(ValueError, match="exponent"):
        api.kvq_write(api.QuantCache(cache.rows, 40), c, k, s)
    ki = api.KvqInputs(B=2, Q=1, H=4, scale=0.1, q_lat=torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16),
                       q_pe=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), cache=cache,
                       prefix_lens=torch.zeros(2, dtype=torch.int32), page_size=1,
                       kv_indptr=torch.zeros(3, dtype=torch.int32), kv_indices=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.kvq_attn(ki)
    for bad in (dict(q_lat=ki.q_lat.float()), dict(q_pe=ki.q_pe[:1]), dict(prefix_lens=ki.prefix_lens.long()),
                dict(kv_indptr=ki.kv_indptr[:2]), dict(kv_indices=None), dict(page_size=16),
                dict(tree_parent=torch.zeros(2, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            api.kvq_attn(dataclasses.replace(ki, **bad))
    for bad in (dict(window=2 ** 32 + 5), dict(window=4, sinks=2 ** 31), dict(page_size=2 ** 32 + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            api.kvq_attn(dataclasses.replace(ki, **bad))
    with pytest.raises(ValueError, match="dtype"):
        api.kvq_read(cache, s, "fp16")


# ---------------------------------------------------------------------------
# orderings that a run on one chip cannot show
# ---------------------------------------------------------------------------
def test_relaxed_cluster_arrivals_follow_no_loads():
    # A relaxed arrive on another CTA's barrier orders none of the thread's own loads and stores before it, so it may
    # only pass on what another barrier has said: that a bulk copy has read its source (ps_free).  Every other signal
    # to the peer, fin_free (the row sums have been read) and fin_full (they are written), releases.
    src = open(os.path.join(B.CSRC, "kvq_attn.cu")).read()
    relaxed = re.findall(r"mbar_arrive_cluster_relaxed\(&c->(\w+)", src)
    release = re.findall(r"mbar_arrive_cluster\(&c->(\w+)", src)
    assert set(relaxed) == {"ps_free"}
    assert set(release) == {"fin_free", "fin_full"}
