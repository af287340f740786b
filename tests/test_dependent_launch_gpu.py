"""Calls launched right behind the kernel that writes their input, whose kernels are resident
before it has ended: they must see what it wrote, call after call into the same buffers."""
import dataclasses

import pytest
import torch

import head_latent_attention_07_b200 as M
import workload as W
from mla_gpu_util import dims_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("replays", [0, 3])
def test_query_latent_rewritten_before_each_up_projection(replays):
    # the up-projection reads the compressed latent that the launch just before it wrote
    w, T, r, rounds = dataclasses.replace(W.WORKLOADS["v2"], n_heads=8, d_model=2048), 13, 104, 20
    d = dims_of(w)
    g = torch.Generator(device="cuda").manual_seed(6)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    w_dq, w_uq = randn(r, w.d_model), randn(w.n_heads * (w.qk_nope + w.d_rope), r)
    h = [randn(T, w.d_model) for _ in range(rounds)]
    q = [torch.empty(T, w.n_heads, w.qk_nope + w.d_rope, dtype=torch.bfloat16, device="cuda") for _ in h]
    c_q = torch.zeros(T, r, dtype=torch.bfloat16, device="cuda")

    def calls():
        for x, y in zip(h, q):
            M.mla_query_proj(d, x, w_dq, w_uq, c_q, y)

    if replays == 0:
        calls()
    else:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
    for _ in range(replays):
        for y in q:
            y.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(h, q):
        alone = torch.empty_like(y)
        M.mla_query_proj(d, x, w_dq, w_uq, torch.zeros_like(c_q), alone)
        torch.cuda.synchronize()
        assert torch.equal(alone.view(torch.int16), y.view(torch.int16))
