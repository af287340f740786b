"""Every call from a host thread that has made no CUDA call yet (a server's worker thread), on the
stream it is given and on its current one: the same bits as from the main thread."""
import threading

import pytest
import torch

import head_latent_attention_07_b200 as M
import workload as W
from mla_gpu_util import GpuStep
from test_eviction_use_gpu import Loop

pytestmark = pytest.mark.gpu


def in_thread(f):
    error = []

    def body():
        try:
            f()
        except Exception as e:          # reported in the main thread
            error.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if error:
        raise error[0]


def decode_calls():
    w = W.Workload("thread", batch=2, nq=1, n_heads=16, d_model=256, d_c=512, d_rope=64, qk_nope=128, v_head=64,
                   context=None, ragged=(1, 1))
    g = GpuStep(W.make_decode_inputs(w, seed=1, lens=[100, 200])).run()
    q = g.q_lat.view(2, 1, 16, 576)
    lat = torch.zeros(2, 1, 16, 512, device="cuda")
    given = (g.dims, q, g.pool, g.page_table, g.seq_lens)
    yield "append", lambda s: M.mla_append_latent(g.dims, g.h, g.w_dkv, g.h_seq_idx, g.h_pos, g.page_table, g.pool, stream=s), g.pool
    yield "absorb", lambda s: M.mla_absorb_q(g.dims, g.q, g.q_pos, g.w_uk, g.q_lat, stream=s), g.q_lat
    yield "decode", lambda s: M.mla_decode_attn(*given, g.w_uv, g.ws, g.out, g.lse, stream=s), g.out
    yield "noalloc", lambda s: M.mla_decode_attn_noalloc(*given, g.w_uv, g.out, g.lse, stream=s), g.out
    yield "partial", lambda s: M.mla_decode_attn_partial(*given, 0, 1, g.ws, lat, g.lse, stream=s), lat
    yield "merge", lambda s: M.mla_merge_ranks(g.dims, [lat], [g.lse.clone()], g.w_uv, g.out, stream=s), g.out


def eviction_calls(**shape):
    x = Loop([700, 64, 1500], 4, nq=1, heads=40, **shape)
    c = x.c
    yield "mass", lambda s: M.mla_attn_mass(c.dims, c.q, c.pool, c.page_table, c.seq_lens, c.lse, c.mass, decay=0.0,
                                            stream=s), c.mass
    yield "select", lambda s: M.mla_evict_select(c.mass, c.seq_lens, x.budgets, x.keep, x.new, stream=s), x.keep
    yield "compact", lambda s: M.mla_cache_compact(c.dims, c.pool, c.page_table, c.seq_lens, x.keep, x.new, rerotate=False,
                                                   stream=s), None


@pytest.mark.parametrize("calls", [decode_calls, eviction_calls,
                                   lambda: eviction_calls(page=48, d_c=64, d_rope=16)], ids=["decode", "eviction", "other shape"])
def test_call_from_a_fresh_thread(calls):
    stream = torch.cuda.Stream()
    for name, call, out in calls():
        run = [lambda: call(None), lambda: in_thread(lambda: call(stream)), lambda: in_thread(lambda: call(None))]
        got = []
        for f in run:
            if out is not None and name != "append":
                out.zero_()             # what a call leaves as it was, it leaves alike
            torch.cuda.synchronize()
            f()
            torch.cuda.synchronize()
            got.append(None if out is None else out.view(torch.uint8).clone())
        if out is not None:
            assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0]), name
