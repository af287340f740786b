"""The eviction calls where their parts have to wait for one another, and at the edges of
what their contract allows."""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import head_latent_attention_07_b200 as M
import workload as W
from mla_gpu_util import bits_of, dev_bf16, dev_i32
from oracle import eviction as E
from test_eviction_use_gpu import Loop, same
from test_parity_eviction_gpu import Cache, check_compact, check_select, choose, masses

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("kind", ["neighbours", "same", "spread"])
@pytest.mark.parametrize("batch,width", [(8, 131072), (16, 20000), (1, 40000)])
def test_select_beside_other_work(kind, batch, width):
    """Clusters whose CTAs run at different speeds: other kernels share the SMs, and sequences
    much shorter than the mass rows leave the higher ranks of their cluster without a token, so
    that they are through with a round at once.  The kinds take one to four rounds."""
    rng = np.random.default_rng([batch, width])
    lens = rng.integers(1, width + 1, batch)
    lens[::2] = rng.integers(200, 3000, len(lens[::2]))
    budgets = np.maximum(1, lens // 3)
    m = masses(kind, (batch, width), 17)
    want = E.select(m, lens, budgets, 2, 50)
    mass, seq_lens, room = torch.from_numpy(m).cuda(), dev_i32(lens), dev_i32(budgets)
    a = torch.randn(1024, 1024, device="cuda")
    other = [torch.cuda.Stream() for _ in range(2)]
    repeats = 40
    keep = [torch.full((batch, int(budgets.max())), -7, dtype=torch.int32, device="cuda") for _ in range(repeats)]
    new = [torch.full((batch,), -7, dtype=torch.int32, device="cuda") for _ in range(repeats)]
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i in range(repeats):
        for s in other:
            with torch.cuda.stream(s):
                a @ a
                a.exp()
        M.mla_evict_select(mass, seq_lens, room, keep[i], new[i], n_sink=2, n_recent=50, dev_status=status)
    torch.cuda.synchronize()
    assert M.mla_status_read(status) == 0
    for i in range(repeats):
        assert torch.equal(new[i], new[0]) and torch.equal(keep[i], keep[0]), f"call {i}"
    for b, w in enumerate(want):
        assert int(new[0][b]) == len(w) and np.array_equal(keep[0][b, : len(w)].cpu().numpy(), w), f"sequence {b}"


@pytest.mark.parametrize("replays", [0, 3])
def test_choices_rewritten_before_each_compaction(replays):
    """Choice after choice into the same buffers, each compacted right behind its selection, whose
    kernel is still at work when the compaction's starts: it must see the new indices and lengths,
    not those of the round before, eager and from a replayed graph."""
    lens, rounds = [900, 64, 3000, 1], 12
    g = np.random.default_rng(41)
    m = np.exp(g.standard_normal((rounds, 4, 3072))).astype(np.float32)
    budgets = [np.minimum(lens, [300 + 17 * i, 1 + 5 * i, 2900 - 211 * i, 1]) for i in range(rounds)]
    table, pages = W.make_page_table(np.asarray(lens, dtype=np.int32), 64, 5, True, 2)
    bits = W.bf16_bits(g.standard_normal((pages, 64, 80), dtype=np.float32))
    dims = M.MlaDims(n_heads=1, d_c=64, d_rope=16, qk_nope=32, v_head=64, d_model=64, page_size=64)
    pools = [dev_bf16(bits) for _ in range(rounds)]
    mass, room = [torch.from_numpy(x).cuda() for x in m], [dev_i32(x) for x in budgets]
    page_table, seq_lens = dev_i32(table), dev_i32(lens)
    keep = torch.full((4, 3000), -1, dtype=torch.int32, device="cuda")
    new = torch.zeros(4, dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")

    def calls():
        for i in range(rounds):
            M.mla_evict_select(mass[i], seq_lens, room[i], keep, new, n_sink=2, n_recent=3, dev_status=status)
            M.mla_cache_compact(dims, pools[i], page_table, seq_lens, keep, new, rerotate=False, dev_status=status)

    if replays == 0:
        calls()
    else:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
    for _ in range(replays):
        for pool in pools:
            pool.copy_(dev_bf16(bits))
        graph.replay()
    torch.cuda.synchronize()
    assert M.mla_status_read(status) == 0
    for i in range(rounds):
        want, _ = E.compact(W.bf16_to_f32(bits), table, E.select(m[i], lens, budgets[i], 2, 3), 64, rerotate=False)
        assert np.array_equal(bits_of(pools[i]), W.bf16_bits(want.astype(np.float32))), f"round {i}"


# ------------------------------------------------------------------ attention mass

@pytest.mark.parametrize("shape", [dict(), dict(d_c=64, d_rope=16, nope=32), dict(d_c=64, d_rope=16, nope=32, page=48)])
@pytest.mark.parametrize("nq,heads", [(1, 8), (2, 40), (2, 128), (4, 128), (11, 128)])
def test_mass_of_padded_queries(nq, heads, shape):
    """Rows with lse = -inf give nothing even where their query is NaN or infinite (slots of a
    batch that hold no query): the bits are those of the same call with ordinary queries there,
    and without such rows nothing changes."""
    lens = [700, 70, 300]
    c = Cache(lens, nq, heads, seed=nq + heads, **shape).make_lse()
    plain = c.run()
    c.lse_host[0, nq // 2, 1 : heads - 1 : 3] = -np.inf
    c.lse_host[1] = -np.inf
    c.lse_host[2, nq - 1, 0] = -np.inf
    c.lse = torch.from_numpy(c.lse_host).cuda()
    none = np.isinf(c.lse_host)
    restart = lambda: setattr(c, "mass", torch.from_numpy(c.mass0).cuda())
    restart()
    want = c.run()
    rows = np.abs(want - c.want())
    for b, n in enumerate(lens):
        assert (rows[b, :n] <= c.tolerance() * np.abs(c.want()[b, :n])).all()
    assert not np.array_equal(want, plain)
    for bits in (0x7FC0, 0x7F80, 0xFF80, 0x7F7F):          # NaN, both infinities, the largest number
        c.q_bits[none] = bits
        c.q = dev_bf16(c.q_bits)
        restart()
        assert np.array_equal(c.run(), want), hex(bits)
    assert M.mla_status_read(c.status) == 0


class LongCache:
    """A cache of many tiles (more than five for each CTA pair of the GPU, in ragged sequences, so
    that shares begin and end inside them), its queries and its mass in 64 bits, all on the GPU."""

    LENS = [33001, 9, 1300, 256, 20011, 257, 700, 25600, 255, 17500, 15003]     # 450 tiles of 256 tokens

    def __init__(self, nq, heads, d_c, d_rope, page, decay):
        g = torch.Generator(device="cuda").manual_seed(1000 * nq + heads + d_c)
        self.lens, self.nq, self.decay = [max(n, nq) for n in self.LENS], nq, decay
        row, B = d_c + d_rope, len(self.lens)
        table, pages = W.make_page_table(np.asarray(self.lens, dtype=np.int32), page, 3, True, 2)
        self.dims = M.MlaDims(n_heads=heads, d_c=d_c, d_rope=d_rope, qk_nope=128, v_head=64, d_model=64, page_size=page)
        self.pool = torch.randn(pages, page, row, generator=g, device="cuda").bfloat16()
        self.q = (0.5 * torch.randn(B, nq, heads, row, generator=g, device="cuda")).bfloat16()
        self.page_table, self.seq_lens = dev_i32(table), dev_i32(self.lens)
        self.mass0 = torch.exp(torch.randn(B, table.shape[1] * page, generator=g, device="cuda"))
        self.lse = torch.empty(B, nq, heads, device="cuda")
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        scale = 1.0 / np.sqrt(128 + d_rope)
        self.want, largest = self.mass0.double(), 0.0
        for b, n in enumerate(self.lens):
            keys = self.pool[self.page_table[b, : -(-n // page)].long()].view(-1, row)[:n].double()
            q = self.q[b].double().view(nq * heads, row)
            s = (q @ keys.T).mul_(scale).view(nq, heads, n)
            seen = torch.arange(n, device="cuda")[None, :] <= (n - nq + torch.arange(nq, device="cuda"))[:, None]
            s.masked_fill_(~seen[:, None, :], -float("inf"))
            self.lse[b] = torch.logsumexp(s, 2).float()
            w = torch.exp(s.sub_(self.lse[b].double()[..., None])).sum(dim=(0, 1))
            w[: n - nq] += decay * self.mass0[b, : n - nq].double()
            self.want[b, :n] = w
            largest = max(largest, float((q.float().abs() @ keys.float().abs().T).max()))
        # the product's, the exponent's and the sum's errors as the parity tests derive them; the old
        # mass is rounded once with its decay and once in the sum
        self.tol = (scale * 1.001 * largest * (row / 16 + 16) * 2**-23 + 2 * float(self.lse.abs().max()) * 1.4427 * 2**-23
                    + 2**-22 + nq * heads * 2**-24 + 2**-23)

    def run(self, only=slice(None)):
        mass = self.mass0[only].clone()
        M.mla_attn_mass(self.dims, self.q[only], self.pool, self.page_table[only].clone(), self.seq_lens[only].clone(),
                        self.lse[only].clone(), mass, decay=self.decay, dev_status=self.status)
        torch.cuda.synchronize()
        return mass


@pytest.mark.parametrize("decay", [0.5, 0.0])
@pytest.mark.parametrize("nq,heads,d_c,d_rope,page", [
    (1, 128, 512, 64, 64),     # 128 query rows, resident; the ring laps, both accumulators are used again
    (1, 5, 512, 64, 256),
    (2, 128, 512, 64, 64),     # 256 rows: one group
    (3, 128, 512, 64, 64),     # two and four groups over tiles in fours; the sums pass through the mass
    (8, 128, 512, 64, 32),
    (9, 128, 512, 64, 64),     # five groups: the keys resident, tile after tile
    (1, 16, 64, 16, 64),       # narrow rows
    (3, 128, 64, 16, 8),
    (9, 128, 64, 16, 128),
])
def test_mass_many_tiles_per_pair(nq, heads, d_c, d_rope, page, decay):
    c = LongCache(nq, heads, d_c, d_rope, page, decay)
    got = c.run()
    assert M.mla_status_read(c.status) == 0
    for b, n in enumerate(c.lens):
        off = ((got[b, :n].double() - c.want[b, :n]).abs() / c.want[b, :n]).max()
        assert float(off) <= c.tol, f"sequence {b}: off by {float(off):.2e} (<= {c.tol:.2e})"
        assert torch.equal(got[b, n:], c.mass0[b, n:]), "mass past the end changed"
    # the same bits from one sequence alone, whose tiles are shared out otherwise
    for b in (0, 4, 10):
        assert torch.equal(c.run(slice(b, b + 1))[0], got[b])
    # tokens of a page outside the pool keep their mass, all others theirs
    c.page_table[0, 2:6] = 2**31 - 1
    again = c.run()
    assert M.mla_status_read(c.status) == M.MLA_ERR_RANGE
    assert torch.equal(again[0, 2 * page : 6 * page], c.mass0[0, 2 * page : 6 * page])
    again[0, 2 * page : 6 * page] = got[0, 2 * page : 6 * page]
    assert torch.equal(again, got)


# ------------------------------------------------------------------ compaction

@pytest.mark.parametrize("batch", [1, 5, 10, 19, 38, 75])
@pytest.mark.parametrize("rerotate", [True, False])
def test_compact_short_sequences_in_wide_tables(batch, rerotate):
    """A page table and mass rows as wide as the longest context of an engine over sequences far
    shorter, at batches between the powers of two: launch shapes come from the width."""
    lens = [1 + (1237 * b + 700) % 2500 for b in range(batch)]
    c = Cache(lens, 1, 1, 64, 16, seed=batch, max_pages=131072 // 64)
    check_compact(c, choose(lens, 0.6, batch, sink=2), rerotate=rerotate)


@pytest.mark.parametrize("batch", [1, 5, 10, 19, 38, 75])
def test_select_short_sequences_in_wide_rows(batch):
    lens = [1 + (1237 * b + 700) % 2500 for b in range(batch)]
    check_select(masses("spread", (batch, 131072), batch), lens, np.maximum(1, np.array(lens) // 3), 2, 40)


# ------------------------------------------------------------------ together

def test_calls_from_several_threads():
    """Loops of other sizes issued by host threads of their own, each on a stream of its own."""
    shapes = [dict(nq=2, heads=128), dict(nq=1, heads=40), dict(nq=9, heads=64),
              dict(nq=1, heads=4, page=48, d_c=64, d_rope=16)]
    lens = [[3000, 2000], [700, 64, 1500], [9, 900], [2500, 300, 77, 4000]]
    make = lambda i: Loop(lens[i], 3 + i, **shapes[i])
    want = []
    for i in range(4):
        loop = make(i)
        loop.calls()
        want.append(loop.state())
    for _ in range(3):
        loops = [make(i) for i in range(4)]
        streams = [torch.cuda.Stream() for _ in loops]
        torch.cuda.synchronize()
        with ThreadPoolExecutor(4) as pool:
            list(pool.map(lambda x: x[0].calls(x[1]), zip(loops, streams)))
        for i, loop in enumerate(loops):
            assert same(loop.state(), want[i]), f"thread {i}"
