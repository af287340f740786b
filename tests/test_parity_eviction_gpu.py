"""GPU parity of the eviction calls with the float64 oracle.

Tolerances.  Attention mass: a weight is exp2(scale2 * dot - lse2).  The product
sums R terms in fp32 in steps of 16; each step may lose one unit of 2^-23 of the
partial sum, which is at most A = sum |q k|, and so may the sums inside a step, so
the dot is off by at most (R / 16 + 16) 2^-23 A.  The exponent's own rounding adds
2^-23 max|lse2| (lse2 rounded, the FMA rounded), the exponential 2^-22, and the sum of the
N = nq H positive weights N 2^-24, all relative to the weight.  The old mass adds one
rounding.  Selection: whole numbers, equal.  Compaction: rows that do not turn and
masses, bit for bit; a turned value is off by half a bf16 step, 2^-8 of it, and by
the fp32 arithmetic, 2^-20 of the pair's length.
"""
import numpy as np
import pytest
import torch

import head_latent_attention_07_b200 as M
import workload as W
from mla_gpu_util import GpuStep, assert_close, bits_of, dev_bf16, dev_i32, dims_of, f64_of
from oracle import eviction as E
from oracle import mla as O

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


class Cache:
    """A paged cache of random rows and the queries of one step, on both sides."""

    def __init__(self, lens, nq=1, heads=8, d_c=512, d_rope=64, page=64, nope=128, seed=0, spare=2, max_pages=None,
                 spread=1.0):
        g = np.random.default_rng([seed, 7])
        self.lens = np.asarray(lens, dtype=np.int32)
        self.B, self.nq, self.H, self.d_c, self.R = len(lens), nq, heads, d_c, d_c + d_rope
        self.table, self.pages = W.make_page_table(self.lens, page, seed, True, spare, max_pages)
        self.pool_bits = W.bf16_bits(g.standard_normal((self.pages, page, self.R), dtype=np.float32))
        q = spread * g.standard_normal((self.B, nq, heads, self.R), dtype=np.float32)
        self.q_bits = W.bf16_bits(q)
        self.dims = M.MlaDims(n_heads=heads, d_c=d_c, d_rope=d_rope, qk_nope=nope, v_head=64, d_model=64, page_size=page)
        self.scale = O.softmax_scale(nope, d_rope)
        self.width = self.table.shape[1] * page
        self.pool = dev_bf16(self.pool_bits)
        self.q = dev_bf16(self.q_bits)
        self.page_table = dev_i32(self.table)
        self.seq_lens = dev_i32(self.lens)
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.mass0 = np.exp(g.standard_normal((self.B, self.width))).astype(np.float32)
        self.mass = torch.from_numpy(self.mass0).cuda()
        self.q64 = W.bf16_to_f32(self.q_bits).astype(np.float64)
        self.pool64 = W.bf16_to_f32(self.pool_bits).astype(np.float64)

    def make_lse(self):
        out = np.full((self.B, self.nq, self.H), -np.inf)
        for b in range(self.B):
            rows = O.gather_cache(self.pool64, self.table[b], int(self.lens[b]))
            for i in range(self.nq):
                s = self.scale * rows[: self.lens[b] - self.nq + i + 1] @ self.q64[b, i].T
                m = s.max(axis=0)
                out[b, i] = m + np.log(np.exp(s - m).sum(axis=0))
        self.lse_host = out.astype(np.float32)
        self.lse = torch.from_numpy(self.lse_host).cuda()
        return self

    def tolerance(self):
        a = max(float((np.abs(self.q64[b].reshape(-1, self.R))
                       @ np.abs(O.gather_cache(self.pool64, self.table[b], int(self.lens[b]))).T).max())
                for b in range(self.B))
        l = float(np.abs(self.lse_host[np.isfinite(self.lse_host)]).max(initial=0.0))
        return (self.scale * a * (self.R / 16 + 16) * 2**-23 + 2 * l * LOG2E * 2**-23 + 2**-22
                + self.nq * self.H * 2**-24 + 2**-23)

    def run(self, decay=1.0, mass_lens=None, **kw):
        M.mla_attn_mass(self.dims, self.q, self.pool, self.page_table, self.seq_lens, self.lse, self.mass,
                        mass_lens=None if mass_lens is None else dev_i32(mass_lens), decay=decay,
                        dev_status=self.status, **kw)
        torch.cuda.synchronize()
        return self.mass.cpu().numpy()

    def want(self, decay=1.0, mass_lens=None):
        return E.attention_mass(self.q64, self.pool64, self.table, self.lens, self.lse_host, self.scale, self.mass0,
                                decay, mass_lens)


def check_mass(c, decay=1.0, mass_lens=None):
    got = c.run(decay, mass_lens)
    assert M.mla_status_read(c.status) == 0
    want = c.want(decay, mass_lens)
    tol = c.tolerance()
    for b, n in enumerate(c.lens):
        d = np.abs(got[b, :n] - want[b, :n]) / want[b, :n]
        assert d.max(initial=0.0) <= tol, f"sequence {b}: off by {d.max():.2e} (<= {tol:.2e}) at {d.argmax()}"
        assert np.array_equal(got[b, n:], c.mass0[b, n:]), "mass past the end changed"
    return got


# the tensor-core shape: tile and page edges, one token, ragged batches
@pytest.mark.parametrize("nq,heads,lens", [
    (1, 8, [1]), (1, 8, [63, 64, 65]), (1, 128, [127, 128, 129, 255, 256, 257]),
    (1, 1, [300, 1, 77]), (1, 16, [511, 512, 513, 1025]), (1, 40, [2000, 3]),
    (2, 128, [2, 3, 64, 65, 66, 1000]), (2, 64, [129, 700]), (3, 128, [3, 500, 257]), (5, 12, [5, 6, 320]),
    (32, 128, [32, 33, 300, 600]), (33, 8, [40, 1100]), (64, 4, [64, 129]),
])
def test_mass_tensor_core_shape(nq, heads, lens):
    check_mass(Cache(lens, nq, heads, seed=nq + heads).make_lse())


# the other shapes: narrow and odd rows, other pages
@pytest.mark.parametrize("d_c,d_rope,page,nope,nq,heads,lens", [
    (64, 16, 64, 32, 1, 4, [128]), (64, 16, 64, 32, 1, 4, [1, 15, 16, 17, 127, 129]),
    (128, 32, 64, 64, 2, 16, [2, 200, 65]), (192, 24, 16, 64, 1, 40, [16, 17, 333]), (8, 8, 1, 16, 1, 1, [1, 5, 40]),
    (256, 64, 64, 128, 3, 65, [3, 100]), (512, 64, 32, 128, 1, 128, [31, 33, 300]), (24, 16, 7, 32, 4, 5, [4, 50, 51]),
    (512, 256, 128, 128, 1, 9, [1, 129]), (504, 64, 64, 128, 17, 8, [17, 90]),
    (64, 16, 8, 32, 1, 32, [1, 7, 8, 9, 130, 300]), (128, 32, 256, 64, 2, 128, [2, 255, 256, 257, 900]),
    (256, 64, 128, 128, 8, 128, [127, 129, 700]), (192, 24, 64, 64, 5, 128, [640, 77]), (8, 8, 16, 16, 1, 128, [500]),
    (64, 16, 48, 32, 2, 16, [2, 100, 200]),
])
def test_mass_other_shapes(d_c, d_rope, page, nope, nq, heads, lens):
    check_mass(Cache(lens, nq, heads, d_c, d_rope, page, nope, seed=d_c + nq).make_lse())


@pytest.mark.parametrize("decay", [0.0, 0.5, 0.99])
@pytest.mark.parametrize("shape", [(512, 64), (64, 16)])
def test_mass_decay(decay, shape):
    c = Cache([300, 70, 2], 2, 16, *shape, seed=3).make_lse()
    if decay == 0.0:
        c.mass.fill_(float("nan"))         # old mass is not read
        got = c.run(decay)
        want = c.want(decay)
        for b, n in enumerate(c.lens):
            assert (np.abs(got[b, :n] - want[b, :n]) <= c.tolerance() * want[b, :n]).all()
            assert np.isnan(got[b, n:]).all()
    else:
        check_mass(c, decay)


@pytest.mark.parametrize("shape", [(512, 64), (64, 16)])
def test_mass_lens(shape):
    # tokens from mass_lens on start from nothing, whatever the entry held
    c = Cache([300, 70, 129, 40], 1, 8, *shape, seed=4).make_lse()
    lens = [0, 70, 65, 1000]
    for b, n in enumerate(lens):
        if n < c.width:
            c.mass[b, n : c.lens[b]] = float("nan")
    check_mass(c, 1.0, lens)


@pytest.mark.parametrize("shape", [(512, 64), (64, 16)])
def test_mass_rows_without_keys_and_masked_garbage(shape):
    # rows whose lse is -inf give nothing; NaN and infinity in rows past the end, in spare
    # pages and in tokens later than the query reach no other token
    c = Cache([65, 300, 40], 2, 16, *shape, seed=5, spare=3).make_lse()
    c.lse_host[1, 0, 3:9] = -np.inf
    c.lse_host[2] = -np.inf
    c.lse = torch.from_numpy(c.lse_host).cuda()
    bits = c.pool_bits
    used = np.zeros(bits.shape[:2], dtype=bool)
    for b, n in enumerate(c.lens):
        idx = np.arange(n)
        used[c.table[b][idx // 64], idx % 64] = True
    bits[~used] = np.where(np.arange(c.R) % 2, 0x7FC0, 0xFF80).astype(np.uint16)
    c.pool = dev_bf16(bits)
    got = c.run()
    want = c.want()
    for b, n in enumerate(c.lens):
        assert (np.abs(got[b, :n] - want[b, :n]) <= c.tolerance() * np.abs(want[b, :n])).all()
        assert np.array_equal(got[b, n:], c.mass0[b, n:])
    # a NaN in one token's row stays with that token
    c.pool_bits[c.table[1][2], 5, 0] = 0x7FC0
    c.pool = dev_bf16(c.pool_bits)
    c.mass = torch.from_numpy(c.mass0).cuda()
    again = c.run()
    assert np.isnan(again[1, 133])
    again[1, 133] = got[1, 133]
    assert np.array_equal(again, got)


@pytest.mark.parametrize("shape", [(512, 64), (64, 16), (24, 16, 7)])
@pytest.mark.parametrize("nq,heads", [(1, 5), (3, 100)])
def test_mass_of_one_sequence_is_not_touched_by_another(shape, nq, heads):
    # NaN in the queries of a sequence, whose rows lie behind its neighbour's in memory
    c = Cache([100, 333, 70], nq, heads, *shape, seed=12).make_lse()
    want = c.run()
    c.q[1] = float("nan")
    c.mass = torch.from_numpy(c.mass0).cuda()
    got = c.run()
    assert np.isnan(got[1, :333]).all()
    assert np.array_equal(got[[0, 2]], want[[0, 2]]) and np.array_equal(got[1, 333:], want[1, 333:])


def test_mass_large_scores():
    # scores far from each other: weights from 1 down to nothing
    check_mass(Cache([500, 64], 1, 128, seed=6, spread=4.0).make_lse())


@pytest.mark.parametrize("shape", [(512, 64), (64, 16)])
def test_mass_range_errors(shape):
    c = Cache([200, 300, 100], 2, 8, *shape, seed=8).make_lse()
    want = c.want()
    bad = c.table.copy()
    bad[1, 2] = c.pages                    # tokens 128..191 of sequence 1
    c.page_table = dev_i32(bad)
    lens = c.lens.copy()
    lens[2] = 1                            # below nq
    c.seq_lens = dev_i32(lens)
    got = c.run()
    assert M.mla_status_read(c.status) == M.MLA_ERR_RANGE
    assert np.array_equal(got[2], c.mass0[2])
    assert np.array_equal(got[1, 128:192], c.mass0[1, 128:192])
    tol = c.tolerance()
    for b, sl in ((0, slice(0, 200)), (1, slice(0, 128)), (1, slice(192, 300))):
        assert (np.abs(got[b, sl] - want[b, sl]) <= tol * want[b, sl]).all()
    for v in (-5, c.width + 1, 2**31 - 1):
        M.mla_status_clear(c.status)
        lens[2] = v
        c.seq_lens = dev_i32(lens)
        got = c.run()
        assert M.mla_status_read(c.status) == M.MLA_ERR_RANGE and np.array_equal(got[2], c.mass0[2])


def test_mass_does_not_depend_on_the_batch():
    # one sequence alone, and the same one among others: the same bits
    lens = [700, 64, 1300]
    c = Cache(lens, 2, 128, seed=9).make_lse()
    all_ = c.run()
    for b, n in enumerate(lens):
        mass = torch.from_numpy(c.mass0[b : b + 1].copy()).cuda()
        M.mla_attn_mass(c.dims, c.q[b : b + 1], c.pool, c.page_table[b : b + 1].clone(), dev_i32(lens[b : b + 1]),
                        c.lse[b : b + 1], mass)
        assert np.array_equal(mass.cpu().numpy()[0, :n], all_[b, :n])


def test_mass_of_a_decode_sums_to_its_rows():
    # with the lse that mla_decode_attn returns, the mass of a sequence is nq * H
    w = W.Workload("mass_of_decode", batch=4, nq=2, n_heads=128, d_model=256, d_c=512, d_rope=64, qk_nope=128,
                   v_head=128, context=None, ragged=(1, 1))
    g = GpuStep(W.make_decode_inputs(w, seed=5, lens=[1500, 2, 64, 700])).run()
    mass = torch.full((4, g.page_table.shape[1] * 64), float("nan"), device="cuda")
    M.mla_attn_mass(g.dims, g.q_lat.view(4, 2, 128, 576), g.pool, g.page_table, g.seq_lens, g.lse, mass, decay=0.0,
                    dev_status=g.status)
    assert g.device_status() == 0
    for b, n in enumerate([1500, 2, 64, 700]):
        assert abs(float(mass[b, :n].double().sum()) - 256) <= 256 * 1e-4   # the decode's P is bf16, its lse fp32


# ------------------------------------------------------------------ selection

def run_select(mass, lens, budgets, sink, recent, width=None, batch_lens=None):
    mass = np.ascontiguousarray(mass, dtype=np.float32)
    B = len(lens)
    k = max(1, max(min(int(n), int(m)) for n, m in zip(lens, budgets))) if width is None else width
    keep = torch.full((B, k), -7, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    M.mla_evict_select(torch.from_numpy(mass).cuda(), dev_i32(lens), dev_i32(budgets), keep, new, n_sink=sink,
                       n_recent=recent, dev_status=status)
    return keep.cpu().numpy(), new.cpu().numpy(), M.mla_status_read(status)


def check_select(mass, lens, budgets, sink, recent):
    keep, new, st = run_select(mass, lens, budgets, sink, recent)
    assert st == 0
    want = E.select(mass, lens, budgets, sink, recent)
    for b, w in enumerate(want):
        assert new[b] == len(w)
        assert np.array_equal(keep[b, : len(w)], w), f"sequence {b}"
        assert (keep[b, len(w):] == -7).all(), "entries past the new length changed"


def masses(kind, shape, seed):
    g = np.random.default_rng([seed, 11])
    m = np.exp(2 * g.standard_normal(shape)).astype(np.float32)
    if kind == "zeros":
        m[g.random(shape) < 0.5] = 0.0
    elif kind == "levels":
        m = np.round(4 * m) / 4
    elif kind == "same":
        m[:] = 0.125
    elif kind == "neighbours":                    # keys next to each other, and borders of the bins
        m = (np.float32(1).view(np.uint32) + g.integers(0, 5000, shape)).astype(np.uint32).view(np.float32)
    elif kind == "anything":                      # any bits: NaN, infinities, denormals, both zeros
        m = g.integers(0, 2**32, shape, dtype=np.uint64).astype(np.uint32).view(np.float32)
        m[g.random(shape) < 0.1] = -0.0
        m[g.random(shape) < 0.1] = 0.0
        m[g.random(shape) < 0.05] = np.nan
    return m


@pytest.mark.parametrize("kind", ["spread", "zeros", "levels", "same", "neighbours", "anything"])
@pytest.mark.parametrize("lens,budgets,sink,recent", [
    ([1000], [500], 4, 64), ([1, 2, 33], [1, 1, 32], 0, 0), ([31, 32, 33, 0, 64], [7, 31, 32, 5, 0], 2, 3),
    ([2047, 2049, 4096, 5001], [100, 2048, 4095, 1], 1, 33), ([9000, 70, 12000], [8999, 500, 3], 16, 256),
    ([20000, 131], [64, 130], 4, 4096), ([3000, 9], [70, 8], 2**31 - 1, 2**31 - 1), ([3000, 9], [70, 8], 0, 2**31 - 1),
])
def test_select(kind, lens, budgets, sink, recent):
    check_select(masses(kind, (len(lens), max(lens)), len(lens)), lens, budgets, sink, recent)


@pytest.mark.parametrize("budget", [0, 1, 5, 6, 9, 10, 11, 99, 100, 101])
def test_select_protected_tokens_fill_the_budget(budget):
    check_select(masses("spread", (2, 100), 1), [100, 40], [budget, budget], 6, 4)


@pytest.mark.parametrize("batch", [1, 3, 19, 75, 200])
def test_select_batches(batch):
    # one to eight CTAs per sequence
    g = np.random.default_rng(batch)
    lens = g.integers(1, 30000, batch)
    check_select(masses("spread", (batch, 30000), batch), lens, np.maximum(1, lens // 3), 4, 128)


@pytest.mark.parametrize("kind", ["spread", "zeros"])
def test_select_longer_than_shared_memory(kind):
    # more tokens than a cluster's shared memory holds, and than one CTA's
    check_select(masses(kind, (1, 600001), 2), [600001], [300000], 4, 1000)
    check_select(masses(kind, (150, 60000), 3), [60000 - 37 * b for b in range(150)], [1234] * 150, 4, 100)


@pytest.mark.parametrize("batch", [1, 40])
@pytest.mark.parametrize("equal", [1, 256, 700])
def test_select_plateaus(equal, batch):
    # equal masses spread over the CTAs; the border falls before, inside and behind them
    n = 9000
    g = np.random.default_rng([equal, batch])
    m = np.exp(g.standard_normal((batch, n))).astype(np.float32)
    for b in range(batch):
        m[b, g.permutation(n)[:equal]] = 1.0
    above = int((m[0] > 1.0).sum())
    for k in (above, above + 1, above + equal // 2 + 1, above + equal, above + equal + 1):
        check_select(m, [n] * batch, [k] * batch, 0, 0)
        check_select(m, [n - 13 * b for b in range(batch)], [k] * batch, 5, 77)


@pytest.mark.parametrize("n", [255, 256, 257, 513])
def test_select_short_rows(n):
    for kind in ("spread", "same", "anything"):
        check_select(masses(kind, (3, n), n), [n, n - 1, n - 2], [n // 2, 1, n - 3], 0, 0)
        check_select(masses(kind, (3, n), n), [n, n - 1, n - 2], [n // 2, 3, n - 3], 1, 1)


def test_select_range_errors():
    m = masses("spread", (4, 100), 5)
    lens, budgets = [100, 101, 50, -1], [10, 10, -1, 10]
    keep, new, st = run_select(m, lens, budgets, 0, 0, width=20)
    assert st == M.MLA_ERR_RANGE and new.tolist() == [10, 0, 0, 0]
    assert np.array_equal(keep[0, :10], E.select(m, [100], [10], 0, 0)[0]) and (keep[1:] == -7).all()
    # the kept tokens do not fit a row of keep_idx
    keep, new, st = run_select(m[:2], [100, 20], [30, 30], 0, 0, width=20)
    assert st == M.MLA_ERR_RANGE and new.tolist() == [0, 20]
    assert np.array_equal(keep[1], np.arange(20)) and (keep[0] == -7).all()


# ------------------------------------------------------------------ compaction

def check_compact(c, kept, rerotate=True, theta=0.0, with_mass=True):
    B, k = c.B, max(1, max(len(x) for x in kept))
    idx = np.full((B, k), -1, dtype=np.int32)
    for b, x in enumerate(kept):
        idx[b, : len(x)] = x
    c.dims.rope_theta = theta
    M.mla_cache_compact(c.dims, c.pool, c.page_table, c.seq_lens, dev_i32(idx), dev_i32([len(x) for x in kept]),
                        mass=c.mass if with_mass else None, rerotate=rerotate, dev_status=c.status)
    assert M.mla_status_read(c.status) == 0
    want, mass = E.compact(c.pool64, c.table, kept, c.d_c, mass=c.mass0, rerotate=rerotate,
                           **({"theta": theta} if theta else {}))
    got = bits_of(c.pool)
    exact = W.bf16_bits(want.astype(np.float32))        # the bits of everything that is only moved
    turned = np.zeros(got.shape[:2], dtype=bool)
    if rerotate:
        for b, x in enumerate(kept):
            j = np.nonzero(np.asarray(x, dtype=np.int64) != np.arange(len(x)))[0]
            turned[c.table[b][j // c.pool64.shape[1]], j % c.pool64.shape[1]] = True
    assert np.array_equal(got[..., : c.d_c], exact[..., : c.d_c]), "latent part"
    assert np.array_equal(got[~turned], exact[~turned]), "rows that stay, or do not belong to the sequences"
    g, w = W.bf16_to_f32(got[turned][:, c.d_c:]).astype(np.float64), want[turned][:, c.d_c:]
    length = np.repeat(np.hypot(w[:, 0::2], w[:, 1::2]), 2, axis=1)
    assert (np.abs(g - w) <= 2**-8 * np.abs(w) + 2**-20 * length).all()
    if with_mass:
        assert np.array_equal(c.mass.cpu().numpy(), mass.astype(np.float32))
    else:
        assert np.array_equal(c.mass.cpu().numpy(), c.mass0)


def choose(lens, keep, seed, sink=0):
    g = np.random.default_rng([seed, 13])
    out = []
    for n in lens:
        k = min(n, int(np.ceil(n * keep)))
        s = min(sink, k)
        out.append(np.concatenate([np.arange(s), s + np.sort(g.permutation(n - s)[: k - s])]).astype(np.int64))
    return out


@pytest.mark.parametrize("keep", [0.05, 0.5, 0.95, 1.0])
@pytest.mark.parametrize("shape,page,lens", [
    ((512, 64), 64, [1, 64, 65, 1000]), ((512, 64), 64, [5000]), ((64, 16), 64, [300, 70]), ((192, 24), 16, [333, 2, 47]),
    ((24, 16), 7, [100, 51]), ((8, 8), 1, [40, 9]), ((512, 256), 128, [400] * 3), ((120, 40), 48, [500, 499]),
])
def test_compact(shape, page, lens, keep):
    c = Cache(lens, 1, 1, *shape, page, seed=page + len(lens))
    check_compact(c, choose(lens, keep, 1))


@pytest.mark.parametrize("batch", [1, 2, 3, 5, 8, 17, 40])
def test_compact_batches(batch):
    # the clusters of every size
    lens = [3000 + 711 * b % 1900 for b in range(batch)]
    check_compact(Cache(lens, 1, 1, seed=batch), choose(lens, 0.6, batch, sink=4))


@pytest.mark.parametrize("lens", [[131072], [40000, 9000]])
def test_compact_long(lens):
    # moves over far positions, many tiles per CTA
    check_compact(Cache(lens, 1, 1, 64, 16, seed=3), choose(lens, 0.7, 5))
    check_compact(Cache(lens, 1, 1, 64, 16, seed=3), choose(lens, 0.01, 5))


def test_compact_moves_by_one_and_by_everything():
    # every row moves by one: each is read by its neighbour; only the last row stays: the longest move
    lens = [2000, 2000, 64]
    check_compact(Cache(lens, 1, 1, seed=2), [np.arange(1, 2000), np.array([1999]), np.array([63])])


def test_compact_same_index_twice():
    kept = [np.array([5, 5, 5, 9, 9]), np.array([299] * 200)]
    check_compact(Cache([10, 300], 1, 1, seed=2), kept)


def test_compact_without_turning_and_without_mass():
    lens = [500, 64, 129]
    check_compact(Cache(lens, 1, 1, seed=4), choose(lens, 0.5, 1), rerotate=False)
    check_compact(Cache(lens, 1, 1, seed=4), choose(lens, 0.5, 1), with_mass=False)
    check_compact(Cache(lens, 1, 1, seed=4), choose(lens, 0.5, 1), theta=1234.5)
    check_compact(Cache(lens, 1, 1, seed=4), [[], [], []])


def test_compact_negative_index():
    c = Cache([300], 1, 1, seed=7)
    before = bits_of(c.pool)
    M.mla_cache_compact(c.dims, c.pool, c.page_table, c.seq_lens, dev_i32([[0, -1, -2**31]]), dev_i32([3]), mass=c.mass,
                        dev_status=c.status)
    assert M.mla_status_read(c.status) == M.MLA_ERR_RANGE
    assert np.array_equal(bits_of(c.pool), before) and np.array_equal(c.mass.cpu().numpy(), c.mass0)


def test_compact_range_errors():
    c = Cache([300, 200, 100, 260], 1, 1, seed=6)
    before = bits_of(c.pool)
    idx = np.full((4, 50), -1, dtype=np.int32)
    idx[0, :4] = [2, 0, 300, 7]                 # row 1 would read below itself, row 2 past the end
    idx[1, :50] = np.arange(100, 150)
    idx[3, :3] = [64, 130, 200]                 # pages 1, 2, 3
    table = c.table.copy()
    table[3, 2] = -5                            # page of token 130
    M.mla_cache_compact(c.dims, c.pool, dev_i32(table), dev_i32([300, 200, 5000, 260]), dev_i32(idx),
                        dev_i32([4, 51, 10, 3]), mass=c.mass, rerotate=False, dev_status=c.status)
    assert M.mla_status_read(c.status) == M.MLA_ERR_RANGE
    got = bits_of(c.pool)
    want = before.copy()
    row = lambda b, n: (c.table[b][n // 64], n % 64)
    for b, j, n in ((0, 0, 2), (0, 3, 7), (3, 0, 64), (3, 2, 200)):
        want[row(b, j)] = before[row(b, n)]
    assert np.array_equal(got, want)
    mass = c.mass0.copy()
    mass[0, [0, 3]] = c.mass0[0, [2, 7]]
    mass[3, :3] = c.mass0[3, [64, 130, 200]]    # the mass lies in no page
    assert np.array_equal(c.mass.cpu().numpy(), mass)


# ------------------------------------------------------------------ together

def test_decode_with_a_budget():
    """Steps of append, absorb, decode and mass on a cache that is cut back to its
    budget every third step; each call against the oracle on what it was given."""
    lens = [200, 65, 300]
    w = W.Workload("budget", batch=3, nq=1, n_heads=16, d_model=256, d_c=512, d_rope=64, qk_nope=128, v_head=64,
                   context=None, ragged=(1, 1))
    x = W.make_decode_inputs(w, seed=31, lens=lens, max_pages=6)
    # room for every sequence at its longest
    g = GpuStep(x)
    table, pages = W.make_page_table(np.full(3, 384), 64, 31, True)
    g.pool = dev_bf16(W.bf16_bits(np.random.default_rng(1).standard_normal((pages, 64, 576), dtype=np.float32)))
    g.page_table = dev_i32(table)
    scale = O.softmax_scale(128, 64)
    rng = np.random.default_rng(2)
    mass = torch.zeros(3, 384, device="cuda")
    budgets = dev_i32([150, 150, 96])
    keep = torch.full((3, 150), -1, dtype=torch.int32, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    now = np.array(lens, dtype=np.int32)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    f64 = lambda t: W.bf16_to_f32(bits_of(t)).astype(np.float64)
    for step in range(7):
        h = dev_bf16(W.bf16_bits(rng.standard_normal((3, 256), dtype=np.float32)))
        q = dev_bf16(W.bf16_bits(rng.standard_normal((3, 16, 192), dtype=np.float32)))
        g.seq_lens = dev_i32(now)
        M.mla_append_absorb(g.dims, h, g.w_dkv, dev_i32([0, 1, 2]), dev_i32(now - 1), g.page_table, g.pool, q, g.w_uk,
                            g.q_lat, dev_status=status)
        q_lat = g.q_lat.view(3, 1, 16, 576)
        M.mla_decode_attn(g.dims, q_lat, g.pool, g.page_table, g.seq_lens, g.w_uv, g.ws, g.out, g.lse, dev_status=status)
        before = mass.cpu().numpy()
        M.mla_attn_mass(g.dims, q_lat, g.pool, g.page_table, g.seq_lens, g.lse, mass, decay=0.9, dev_status=status)
        out, lse = O.attend_paged_latents(q_lat=f64(g.q_lat), pool=f64(g.pool), page_table=table, lens=now, nq=1,
                                          w_uv=f64(g.w_uv), scale=scale)
        assert_close(f64_of(g.out).reshape(3, 16, 64), out, "out")
        assert_close(f64_of(g.lse).reshape(3, 16), lse, "lse")
        want = E.attention_mass(f64(g.q_lat).reshape(3, 1, 16, 576), f64(g.pool), table, now, g.lse.cpu().numpy(), scale,
                                before, 0.9)
        got = mass.cpu().numpy()
        for b, n in enumerate(now):
            # scale * A * (R / 16 + 16) * 2^-23 with A = sum |q k| <= 900 here, and the smaller terms
            assert np.allclose(got[b, :n], want[b, :n], rtol=0.072 * 900 * 52 * 2**-23, atol=0)
        if step % 3 == 2:
            pool0 = f64(g.pool)
            M.mla_evict_select(mass, g.seq_lens, budgets, keep, new, n_sink=4, n_recent=16, dev_status=status)
            M.mla_cache_compact(g.dims, g.pool, g.page_table, g.seq_lens, keep, new, mass=mass, dev_status=status)
            kept = E.select(got, now, budgets.cpu().numpy(), 4, 16)
            assert new.cpu().numpy().tolist() == [len(k) for k in kept]
            for b, k in enumerate(kept):
                assert np.array_equal(keep[b, : len(k)].cpu().numpy(), k)
            pool, m = E.compact(pool0, table, kept, 512, mass=got)
            assert (np.abs(f64(g.pool) - pool) <= 2**-8 * np.abs(pool) + 2**-17).all()
            assert np.array_equal(mass.cpu().numpy(), m.astype(np.float32))
            now = new.cpu().numpy().copy()
        now = now + 1
    assert M.mla_status_read(status) == 0
