"""The eviction calls where their parts have to wait for one another, and at the edges of
what their contract allows."""
import numpy as np
import pytest
import torch

import head_latent_attention_07_b200 as M
from mla_gpu_util import dev_i32
from oracle import eviction as E
from test_parity_eviction_gpu import masses

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
