"""Host-side checks of the eviction calls (no GPU needed): the C entry points and
the binding refuse bad arguments before anything is launched."""
import ctypes
import os

import pytest
import torch

import head_latent_attention_07_b200 as M

FAKE = 1 << 20          # 16-byte aligned fake device address (never dereferenced)
FAKE_MIS = FAKE + 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from head_latent_attention_07_b200 import build
        build.build()
    return M.load_library()


def v3_dims(**kw):
    d = dict(n_heads=128, d_c=512, d_rope=64, qk_nope=128, v_head=128, d_model=7168, page_size=64,
             softmax_scale=0.0, rope_theta=0.0)
    d.update(kw)
    return M.MlaDims(**d)


def test_attn_mass_argument_checks(lib):
    def call(dims=v3_dims(), **kw):
        return lib.mla_attn_mass(
            ctypes.byref(dims) if dims is not None else None, kw.get("q", FAKE), kw.get("pool", FAKE),
            kw.get("pt", FAKE), kw.get("lens", FAKE), kw.get("lse", FAKE), kw.get("B", 2), kw.get("nq", 1),
            kw.get("mp", 4), kw.get("np_", 8), kw.get("decay", 1.0), kw.get("ml", None), kw.get("mass", FAKE),
            kw.get("stride", 256), kw.get("st", None), None)
    assert call(dims=None) == M.MLA_ERR_INVALID_ARG
    assert call(dims=v3_dims(d_rope=0)) == M.MLA_ERR_UNSUPPORTED
    assert call(dims=v3_dims(n_heads=129)) == M.MLA_ERR_UNSUPPORTED
    assert call(dims=v3_dims(d_c=500)) == M.MLA_ERR_UNSUPPORTED
    assert call(dims=v3_dims(page_size=257)) == M.MLA_ERR_UNSUPPORTED
    assert call(dims=v3_dims(softmax_scale=float("nan"))) == M.MLA_ERR_INVALID_ARG
    for name in ("q", "pool", "pt", "lens", "lse", "mass"):
        assert call(**{name: None}) == M.MLA_ERR_INVALID_ARG, name
        assert call(**{name: FAKE_MIS}) == M.MLA_ERR_MISALIGNED, name
    assert call(ml=FAKE_MIS) == M.MLA_ERR_MISALIGNED
    assert call(st=FAKE + 4) == M.MLA_ERR_MISALIGNED
    for bad in (-0.1, 1.5, float("nan"), float("inf")):
        assert call(decay=bad) == M.MLA_ERR_INVALID_ARG, bad
    assert call(B=0) == M.MLA_ERR_INVALID_ARG
    assert call(nq=0) == M.MLA_ERR_INVALID_ARG
    assert call(mp=0) == M.MLA_ERR_INVALID_ARG
    assert call(np_=0) == M.MLA_ERR_INVALID_ARG
    assert call(stride=255) == M.MLA_ERR_INVALID_ARG           # below max_pages * page_size
    assert call(B=1025) == M.MLA_ERR_UNSUPPORTED
    assert call(nq=1025) == M.MLA_ERR_UNSUPPORTED
    assert call(B=1000, nq=1000) == M.MLA_ERR_UNSUPPORTED
    assert call(mp=1 << 26) == M.MLA_ERR_UNSUPPORTED
    assert call(mp=(1 << 24) + 1, stride=1 << 40) == M.MLA_ERR_UNSUPPORTED     # longer than 2^30 tokens


def test_evict_select_argument_checks(lib):
    call = lambda **kw: lib.mla_evict_select(
        kw.get("mass", FAKE), kw.get("stride", 256), kw.get("lens", FAKE), kw.get("bud", FAKE), kw.get("B", 2),
        kw.get("sink", 0), kw.get("recent", 0), kw.get("keep", FAKE), kw.get("ks", 16), kw.get("new", FAKE),
        kw.get("st", None), None)
    for name in ("mass", "lens", "bud", "keep", "new"):
        assert call(**{name: None}) == M.MLA_ERR_INVALID_ARG, name
        assert call(**{name: FAKE_MIS}) == M.MLA_ERR_MISALIGNED, name
    assert call(st=FAKE + 4) == M.MLA_ERR_MISALIGNED
    for bad in (dict(B=0), dict(stride=0), dict(ks=0), dict(sink=-1), dict(recent=-1)):
        assert call(**bad) == M.MLA_ERR_INVALID_ARG, bad
    assert call(B=1025) == M.MLA_ERR_UNSUPPORTED
    assert call(stride=(1 << 30) + 1) == M.MLA_ERR_UNSUPPORTED


def test_cache_compact_argument_checks(lib):
    def call(dims=v3_dims(), **kw):
        return lib.mla_cache_compact(
            ctypes.byref(dims) if dims is not None else None, kw.get("pool", FAKE), kw.get("pt", FAKE),
            kw.get("lens", FAKE), kw.get("keep", FAKE), kw.get("ks", 16), kw.get("new", FAKE), kw.get("B", 2),
            kw.get("mp", 4), kw.get("np_", 8), kw.get("rot", 1), kw.get("mass", None), kw.get("stride", 0),
            kw.get("st", None), None)
    assert call(dims=None) == M.MLA_ERR_INVALID_ARG
    assert call(dims=v3_dims(d_rope=0)) == M.MLA_ERR_UNSUPPORTED
    assert call(dims=v3_dims(d_rope=264)) == M.MLA_ERR_UNSUPPORTED
    assert call(dims=v3_dims(rope_theta=-1.0)) == M.MLA_ERR_INVALID_ARG
    for name in ("pool", "pt", "lens", "keep", "new"):
        assert call(**{name: None}) == M.MLA_ERR_INVALID_ARG, name
        assert call(**{name: FAKE_MIS}) == M.MLA_ERR_MISALIGNED, name
    assert call(st=FAKE + 4) == M.MLA_ERR_MISALIGNED
    assert call(mass=FAKE_MIS, stride=256) == M.MLA_ERR_MISALIGNED
    assert call(mass=FAKE, stride=255) == M.MLA_ERR_INVALID_ARG
    assert call(rot=2) == M.MLA_ERR_INVALID_ARG
    for bad in (dict(B=0), dict(ks=0), dict(mp=0), dict(np_=0)):
        assert call(**bad) == M.MLA_ERR_INVALID_ARG, bad
    assert call(B=1025) == M.MLA_ERR_UNSUPPORTED
    assert call(mp=1 << 26) == M.MLA_ERR_UNSUPPORTED
    assert call(np_=1 << 26) == M.MLA_ERR_UNSUPPORTED                          # row numbers past 32 bits


# ------------------------------------------------------------------ the binding, on CPU tensors

def tensors(B=2, nq=1, pages=4):
    d = v3_dims(n_heads=4, d_c=16, d_rope=8, page_size=8)
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    return d, dict(q_lat=torch.zeros(B, nq, 4, 24, dtype=bf), pool=torch.zeros(9, 8, 24, dtype=bf),
                   page_table=torch.zeros(B, pages, dtype=i32), seq_lens=torch.zeros(B, dtype=i32),
                   lse=torch.zeros(B, nq, 4, dtype=f32), mass=torch.zeros(B, 8 * pages, dtype=f32),
                   budgets=torch.zeros(B, dtype=i32), keep_idx=torch.zeros(B, 5, dtype=i32),
                   new_lens=torch.zeros(B, dtype=i32))


def mass_call(d, t, **kw):
    M.mla_attn_mass(d, t["q_lat"], t["pool"], t["page_table"], t["seq_lens"], t["lse"], t["mass"], **kw)


def select_call(t, **kw):
    M.mla_evict_select(t["mass"], t["seq_lens"], t["budgets"], t["keep_idx"], t["new_lens"], **kw)


def compact_call(d, t, **kw):
    M.mla_cache_compact(d, t["pool"], t["page_table"], t["seq_lens"], t["keep_idx"], t["new_lens"], **kw)


@pytest.mark.parametrize("name,bad", [
    ("q_lat", torch.zeros(2, 1, 3, 24, dtype=torch.bfloat16)),
    ("pool", torch.zeros(9, 8, 16, dtype=torch.bfloat16)),
    ("page_table", torch.zeros(3, 4, dtype=torch.int32)),
    ("seq_lens", torch.zeros(3, dtype=torch.int32)),
    ("lse", torch.zeros(2, 1, 5)),
])
def test_attn_mass_binding_refuses_shapes(name, bad):
    d, t = tensors()
    t[name] = bad
    with pytest.raises(ValueError):
        mass_call(d, t)


@pytest.mark.parametrize("name,bad,error", [
    ("mass", torch.zeros(2, 32, dtype=torch.float64), TypeError),
    ("mass", torch.zeros(2, 32), ValueError),                    # on the CPU
    ("budgets", torch.zeros(3, dtype=torch.int32), ValueError),
    ("new_lens", torch.zeros(1, dtype=torch.int32), ValueError),
])
def test_evict_select_binding_refuses(name, bad, error):
    _, t = tensors()
    t[name] = bad
    with pytest.raises(error):
        select_call(t)


@pytest.mark.parametrize("kw", [dict(n_sink=-1), dict(n_recent=-3), dict(n_recent=2**31), dict(n_sink=2**40)])
def test_evict_select_binding_refuses_counts(kw):
    with pytest.raises(ValueError):
        select_call(tensors()[1], **kw)


@pytest.mark.parametrize("name,bad,error", [
    ("pool", torch.zeros(9, 7, 24, dtype=torch.bfloat16), ValueError),
    ("seq_lens", torch.zeros(1, dtype=torch.int32), ValueError),
    ("new_lens", torch.zeros(4, dtype=torch.int32), ValueError),
    ("keep_idx", torch.zeros(2, 5, dtype=torch.int64), TypeError),
])
def test_cache_compact_binding_refuses(name, bad, error):
    d, t = tensors()
    t[name] = bad
    with pytest.raises(error):
        compact_call(d, t)
