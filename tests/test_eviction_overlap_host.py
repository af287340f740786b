"""Host-side checks (no GPU needed): the eviction calls refuse an output that overlaps
another of their buffers, before anything is launched, and nothing else that lies close by."""
import ctypes
import os

import pytest
import torch

import head_latent_attention_07_b200 as M

BASE = 1 << 20          # 16-byte aligned fake device addresses, 256 MB apart (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from head_latent_attention_07_b200 import build
        build.build()
    return M.load_library()


DIMS = M.MlaDims(n_heads=128, d_c=512, d_rope=64, qk_nope=128, v_head=128, d_model=7168, page_size=64)
B, NQ, PAGES, POOL, KEEP = 4, 2, 8, 40, 100
TOKENS = PAGES * 64
BYTES = dict(q_lat=B * NQ * 128 * 576 * 2, pool=POOL * 64 * 576 * 2, page_table=B * PAGES * 4, seq_lens=B * 4,
             mass_lens=B * 4, lse=B * NQ * 128 * 4, mass=B * TOKENS * 4, budgets=B * 4, keep_idx=B * KEEP * 4,
             new_lens=B * 4)


def addresses():
    return {name: BASE + (i << 28) for i, name in enumerate(BYTES)}


def attn_mass(lib, p, stride=TOKENS):
    return lib.mla_attn_mass(ctypes.byref(DIMS), p["q_lat"], p["pool"], p["page_table"], p["seq_lens"], p["lse"], B, NQ,
                             PAGES, POOL, 1.0, p["mass_lens"], p["mass"], stride, None, None)


def evict_select(lib, p, stride=TOKENS):
    return lib.mla_evict_select(p["mass"], stride, p["seq_lens"], p["budgets"], B, 0, 0, p["keep_idx"], KEEP,
                                p["new_lens"], None, None)


def cache_compact(lib, p, stride=TOKENS):
    return lib.mla_cache_compact(ctypes.byref(DIMS), p["pool"], p["page_table"], p["seq_lens"], p["keep_idx"], KEEP,
                                 p["new_lens"], B, PAGES, POOL, 1, p["mass"], stride, None, None)


# buffers whose used part the host knows: an output may not share a byte with another one
KNOWN = {attn_mass: (["mass"], ["q_lat", "pool", "page_table", "seq_lens", "mass_lens", "lse"]),
         evict_select: (["new_lens"], ["seq_lens", "budgets"]),
         cache_compact: (["pool", "mass"], ["page_table", "seq_lens", "new_lens"])}
PAIRS = [(call, out, other) for call, (outs, ins) in KNOWN.items()
         for out in outs for other in ins + outs if other != out]


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where nothing can be launched")
@pytest.mark.parametrize("call,out,other", PAIRS, ids=lambda v: getattr(v, "__name__", v))
def test_overlapping_output_is_refused(lib, call, out, other):
    p = addresses()
    last = lambda name: (BYTES[name] - 4) // 16 * 16        # an aligned address in the last bytes
    for at in (p[other], p[other] + last(other), p[other] - last(out)):
        assert call(lib, {**p, out: at}) == M.MLA_ERR_INVALID_ARG, at - p[other]
    # right before and right behind it lie other buffers: these calls get as far as the device
    for at in (p[other] + (BYTES[other] + 15) // 16 * 16, p[other] - (BYTES[out] + 15) // 16 * 16):
        assert call(lib, {**p, out: at}) == M.MLA_ERR_CUDA


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where nothing can be launched")
@pytest.mark.parametrize("call,name,other", [
    (evict_select, "keep_idx", "mass"), (evict_select, "keep_idx", "seq_lens"), (evict_select, "keep_idx", "budgets"),
    (evict_select, "keep_idx", "new_lens"), (evict_select, "new_lens", "mass"), (evict_select, "new_lens", "keep_idx"),
    (cache_compact, "pool", "keep_idx"), (cache_compact, "mass", "keep_idx"),
], ids=lambda v: getattr(v, "__name__", v))
def test_rows_of_a_length_unknown_to_the_host(lib, call, name, other):
    # the same start is refused
    p = addresses()
    assert call(lib, {**p, name: p[other]}) == M.MLA_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where nothing can be launched")
def test_rows_of_mass_and_indices_may_take_turns(lib):
    # one buffer of a row of mass and a row of indices for each sequence
    p = addresses()
    row = TOKENS + KEEP
    p["keep_idx"] = p["mass"] + TOKENS * 4
    assert lib.mla_evict_select(p["mass"], row, p["seq_lens"], p["budgets"], B, 0, 0, p["keep_idx"], row, p["new_lens"],
                                None, None) == M.MLA_ERR_CUDA
    assert lib.mla_cache_compact(ctypes.byref(DIMS), p["pool"], p["page_table"], p["seq_lens"], p["keep_idx"], row,
                                 p["new_lens"], B, PAGES, POOL, 1, p["mass"], row, None, None) == M.MLA_ERR_CUDA


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where nothing can be launched")
@pytest.mark.parametrize("call", [attn_mass, cache_compact])
def test_rows_of_the_mass_with_room_between_them(lib, call):
    # the other buffer lies in row 2, before it, behind it, and behind the last row
    p = addresses()
    p["mass"] = BASE + (1 << 34)
    stride = 4 * TOKENS
    row = p["mass"] + 2 * stride * 4
    for name in ("page_table", "seq_lens"):
        size = (BYTES[name] + 15) // 16 * 16
        for at in (row, row + TOKENS * 4 - 16, row - size + 16):
            assert call(lib, {**p, name: at}, stride=stride) == M.MLA_ERR_INVALID_ARG
        for at in (row - size, row + TOKENS * 4, row + stride * 4 + TOKENS * 4, p["mass"] - size):
            assert call(lib, {**p, name: at}, stride=stride) == M.MLA_ERR_CUDA
    assert call(lib, p, stride=2**63 - 1) == M.MLA_ERR_CUDA       # the largest stride does not wrap round


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where nothing can be launched")
def test_optional_buffers_overlap_nothing(lib):
    p = addresses()
    assert attn_mass(lib, {**p, "mass_lens": None}) == M.MLA_ERR_CUDA
    assert cache_compact(lib, {**p, "mass": None}, stride=0) == M.MLA_ERR_CUDA
    assert cache_compact(lib, {**p, "seq_lens": p["new_lens"]}) == M.MLA_ERR_CUDA     # two inputs may be one
