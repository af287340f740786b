"""The eviction calls as a serving loop uses them: on other streams, captured into
graphs, two at a time, at the largest batch and chunk, in pools whose offsets pass
32 bits, and with the waits cut short."""
import numpy as np
import pytest
import torch

import head_latent_attention_07_b200 as M
import workload as W
from mla_gpu_util import dev_i32
from oracle import eviction as E
from oracle import mla as O
from test_parity_eviction_gpu import Cache, check_mass

pytestmark = pytest.mark.gpu


class Loop:
    """One step's mass, the choice and the compaction of a cache, with buffers of its own."""

    def __init__(self, lens, seed, **kw):
        self.c = Cache(lens, seed=seed, **kw).make_lse()
        self.budgets = dev_i32(np.maximum(1, np.array(lens) // 2))
        self.keep = torch.full((len(lens), max(lens) // 2 + 1), -1, dtype=torch.int32, device="cuda")
        self.new = torch.zeros(len(lens), dtype=torch.int32, device="cuda")

    def calls(self, stream=None):
        c = self.c
        M.mla_attn_mass(c.dims, c.q, c.pool, c.page_table, c.seq_lens, c.lse, c.mass, decay=0.5, dev_status=c.status,
                        stream=stream)
        M.mla_evict_select(c.mass, c.seq_lens, self.budgets, self.keep, self.new, n_sink=2, n_recent=8,
                           dev_status=c.status, stream=stream)
        M.mla_cache_compact(c.dims, c.pool, c.page_table, c.seq_lens, self.keep, self.new, mass=c.mass,
                            dev_status=c.status, stream=stream)

    def state(self):
        torch.cuda.synchronize()
        assert M.mla_status_read(self.c.status) == 0
        return [t.clone() for t in (self.c.pool.view(torch.int16), self.c.mass.view(torch.int32), self.keep, self.new)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


LENS = [700, 64, 1500, 1]


@pytest.mark.parametrize("shape", [dict(nq=1, heads=128), dict(nq=1, heads=8, d_c=64, d_rope=16, nope=32, page=16)])
def test_streams(shape):
    want = Loop(LENS, 1, **shape)
    want.calls()
    want = want.state()
    given, current = Loop(LENS, 1, **shape), Loop(LENS, 1, **shape)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given.calls(stream=s)
    with torch.cuda.stream(torch.cuda.Stream()):
        current.calls()
    assert same(given.state(), want) and same(current.state(), want)


def test_two_loops_at_a_time():
    # two streams, other sizes on each; neither call keeps anything between calls
    a, b = Loop([3000, 2000], 2, nq=2, heads=128), Loop(LENS, 3, nq=1, heads=40)
    a.calls(), b.calls()
    want_a, want_b = a.state(), b.state()
    for _ in range(3):
        a, b = Loop([3000, 2000], 2, nq=2, heads=128), Loop(LENS, 3, nq=1, heads=40)
        torch.cuda.synchronize()
        sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
        a.calls(sa), b.calls(sb)
        assert same(a.state(), want_a) and same(b.state(), want_b)


@pytest.mark.parametrize("shape", [dict(nq=1, heads=128), dict(nq=9, heads=64), dict(nq=1, heads=4, page=7, d_c=24, d_rope=16)])
def test_captured_and_replayed(shape):
    lens = [max(n, 9) for n in LENS]
    eager = Loop(lens, 4, **shape)
    eager.calls()
    first = eager.state()
    eager.calls()
    second = eager.state()
    g = Loop(lens, 4, **shape)
    s = torch.cuda.Stream()
    warm = Loop(lens, 5, **shape)
    warm.calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g.calls()
    graph.replay()
    assert same(g.state(), first)
    graph.replay()                       # the compacted cache once more, lengths as they were
    assert same(g.state(), second)
    graph.reset()


def test_offsets_past_32_bits():
    # the sequences' pages lie at the end of a pool of 5.2 GB; the same cache in a small
    # pool gives the same bits
    pages = 70000
    small = Loop([300, 129, 64], 6, nq=1, heads=16)
    c = small.c
    big = Loop([300, 129, 64], 6, nq=1, heads=16)
    pool = torch.empty((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    shift = pages - c.pages
    pool[shift:] = c.pool
    big.c.pool = pool
    big.c.page_table = torch.where(c.page_table >= 0, c.page_table + shift, c.page_table)
    small.calls()
    big.calls()
    a, b = small.state(), big.state()
    assert torch.equal(a[0], b[0][shift:]) and same(a[1:], b[1:])


def test_largest_batch():
    lens = [1 + (37 * b) % 200 for b in range(1024)]
    c = Cache(lens, 1, 2, 64, 16, 64, 32, seed=7).make_lse()
    check_mass(c)
    mass = c.mass.cpu().numpy()
    budgets = [1 + n // 3 for n in lens]
    keep = torch.full((1024, 68), -1, dtype=torch.int32, device="cuda")
    new = torch.zeros(1024, dtype=torch.int32, device="cuda")
    M.mla_evict_select(c.mass, c.seq_lens, dev_i32(budgets), keep, new, n_sink=1, n_recent=4, dev_status=c.status)
    M.mla_cache_compact(c.dims, c.pool, c.page_table, c.seq_lens, keep, new, mass=c.mass, dev_status=c.status)
    assert M.mla_status_read(c.status) == 0
    kept = E.select(mass, lens, budgets, 1, 4)
    for b, k in enumerate(kept):
        assert new[b] == len(k) and np.array_equal(keep[b, : len(k)].cpu().numpy(), k)
    pool, m = E.compact(c.pool64, c.table, kept, 64, mass=mass)
    got = W.bf16_to_f32(c.pool.view(torch.int16).cpu().numpy().view(np.uint16)).astype(np.float64)
    assert (np.abs(got - pool) <= 2**-8 * np.abs(pool) + 2**-17).all()
    assert np.array_equal(c.mass.cpu().numpy(), m.astype(np.float32))


def test_largest_chunk():
    # 1024 query tokens of 128 heads, the whole sequence new: every token's mass against 64
    # bits, computed on the GPU a query token at a time
    n, nq, H = 1100, 1024, 128
    g = torch.Generator(device="cuda").manual_seed(8)
    pool = torch.randn(20, 64, 576, generator=g, device="cuda").bfloat16()
    q = (0.7 * torch.randn(1, nq, H, 576, generator=g, device="cuda")).bfloat16()
    table = torch.randperm(20, generator=g, device="cuda")[:18].to(torch.int32)[None].contiguous()
    rows = pool[table[0].long()].view(-1, 576)[:n].double()
    dims = M.MlaDims(n_heads=H, d_c=512, d_rope=64, qk_nope=128, v_head=64, d_model=64, page_size=64)
    lse = torch.empty(1, nq, H, device="cuda")
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    largest = 0.0
    for i in range(nq):
        s = q[0, i].double() @ rows[: n - nq + i + 1].T / 192**0.5
        lse[0, i] = torch.logsumexp(s, 1).float()
        want[: n - nq + i + 1] += torch.exp(s - lse[0, i].double()[:, None]).sum(0)
        if i % 64 == 0:
            largest = max(largest, float((q[0, i].double().abs() @ rows.abs().T).max()))
    mass = torch.full((1, 18 * 64), 3.0, device="cuda")
    M.mla_attn_mass(dims, q, pool, table, dev_i32([n]), lse, mass, decay=0.0)
    # a weight's product and exponent as in the parity tests; the sum adds 64 weights to each of
    # four partial sums and 512 of these in turn, each step off by at most half a unit
    tol = 1.3 * largest / 192**0.5 * (576 / 16 + 16) * 2**-23 + 2 * 12 * 1.45 * 2**-23 + 2**-22 + (66 + 512) * 2**-24
    assert float(((mass[0, :n].double() - want).abs() / want).max()) <= tol
    assert (mass[0, n:] == 3.0).all()


def test_waits_run_out(monkeypatch):
    c = Cache([3000, 400], 1, 128, seed=9).make_lse()
    monkeypatch.setenv("MLA_SPIN_LIMIT", "1")
    c.run()
    assert M.mla_status_read(c.status) == M.MLA_ERR_TIMEOUT
    monkeypatch.delenv("MLA_SPIN_LIMIT")
    M.mla_status_clear(c.status)
    c.mass.copy_(torch.from_numpy(c.mass0))
    check_mass(c)


def test_tensors_elsewhere_are_refused():
    # strided views and tensors of the CPU
    c = Cache([100, 50], 2, 4, seed=10).make_lse()
    call = lambda **kw: M.mla_attn_mass(c.dims, kw.get("q", c.q), c.pool, c.page_table, c.seq_lens, kw.get("lse", c.lse),
                                        kw.get("mass", c.mass))
    for kw in (dict(mass=c.mass.cpu()), dict(lse=c.lse.double()), dict(mass=torch.zeros(2, 256, device="cuda")[:, ::2]),
               dict(q=c.q.transpose(0, 1).contiguous().transpose(0, 1)), dict(mass=torch.zeros(2, 64, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(M.MlaError):       # a view whose first element is not 16-byte aligned
        call(mass=torch.zeros(2 * c.width + 1, device="cuda")[1:].view(2, c.width))
