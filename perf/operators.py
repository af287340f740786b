"""Cases that measure the cache-eviction operators on a GPU.

Three operators keep a paged latent cache within a budget: the attention mass of the cached tokens
(what a step's queries gave each of them, summed over query tokens and heads), the choice of the
tokens that stay, and the compaction of the cache to those.  Each case runs one of them, either in a
plain form written with elementary torch operations (`own` false) or through the library (`own` true).
"""
import math

import torch

own = False

PAGE = 64
THETA = 10000.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the smallest cache of the tests, one decode step: what a launch costs
        dict(name="mass tiny", op="mass", batch=1, nq=1, heads=4, d_c=64, d_rope=16, nope=32, lo=128, hi=128, decay=1.0),
        # one decode step of 8 short conversations with 32 heads
        dict(name="mass 8x4096 h32", op="mass", batch=8, nq=1, heads=32, d_c=512, d_rope=64, nope=128, lo=4096, hi=4096,
             decay=1.0),
        # one decode step of the serving batch that the benchmark times
        dict(name="mass 16x32768 h128", op="mass", batch=16, nq=1, heads=128, d_c=512, d_rope=64, nope=128, lo=32768,
             hi=32768, decay=1.0),
        # a ragged serving batch, two new tokens for each sequence, older mass fading
        dict(name="mass ragged 64x2 h128", op="mass", batch=64, nq=2, heads=128, d_c=512, d_rope=64, nope=128, lo=1024,
             hi=65536, decay=0.99),
        # the last 32 tokens of two prompts vote on what to keep of them: no earlier mass
        dict(name="mass window 2x32 h128", op="mass", batch=2, nq=32, heads=128, d_c=512, d_rope=64, nope=128, lo=32768,
             hi=32768, decay=0.0),
        # one short conversation, half of it kept: latency
        dict(name="select 1x1000", op="select", batch=1, lo=1000, hi=1000, keep=0.5, sink=4, recent=64),
        # the benchmark's batch, half kept
        dict(name="select 16x32768", op="select", batch=16, lo=32768, hi=32768, keep=0.5, sink=4, recent=512),
        # a ragged batch, a budget of its own for each sequence
        dict(name="select ragged 64", op="select", batch=64, lo=1024, hi=65536, keep=0.3, sink=4, recent=256),
        # long contexts cut to a sixteenth
        dict(name="select 8x131072", op="select", batch=8, lo=131072, hi=131072, keep=0.0625, sink=4, recent=1024),
        # short conversations with half of each kept
        dict(name="compact 8x4096", op="compact", batch=8, d_c=512, d_rope=64, lo=4096, hi=4096, keep=0.5, sink=4),
        # the benchmark's cache, half kept
        dict(name="compact 16x32768", op="compact", batch=16, d_c=512, d_rope=64, lo=32768, hi=32768, keep=0.5, sink=4),
        # one long context alone, most of it kept
        dict(name="compact 1x131072", op="compact", batch=1, d_c=512, d_rope=64, lo=131072, hi=131072, keep=0.9, sink=4),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mass", "mass", "select", "compact"])
    hi = _log_uniform(rng, 40, 131072)
    lo = hi if rng.random() < 0.3 else max(1, int(hi * rng.uniform(0.02, 1.0)))
    if op == "select":
        batch = _log_uniform(rng, 1, max(1, min(128, (1 << 21) // hi)))
        return dict(op=op, batch=batch, lo=lo, hi=hi, keep=round(rng.uniform(0.02, 1.1), 3), sink=rng.choice([0, 1, 4, 16]),
                    recent=rng.choice([0, 1, 33, 256]))
    d_c, d_rope, nope = rng.choice([(512, 64, 128)] * 4 + [(64, 16, 32), (128, 32, 64), (256, 64, 128), (192, 24, 64)])
    if op == "compact":
        batch = _log_uniform(rng, 1, max(1, min(64, (1 << 19) // hi)))
        return dict(op=op, batch=batch, d_c=d_c, d_rope=d_rope, lo=lo, hi=hi, keep=round(rng.uniform(0.02, 0.98), 3),
                    sink=rng.choice([0, 1, 4, 16]))
    heads = rng.choice([1, 4, 12, 16, 32, 40, 64, 128, 128])
    nq = rng.choice([1, 1, 1, 2, 3, 4, 8, 17, 32])
    lo, hi = max(lo, nq), max(hi, nq)
    room = (1 << 27) // (hi * max(16, nq * heads))   # a share of the largest listed case's products
    batch = _log_uniform(rng, 1, max(1, min(64, room)))
    return dict(op=op, batch=batch, nq=nq, heads=heads, d_c=d_c, d_rope=d_rope, nope=nope, lo=lo, hi=hi,
                decay=rng.choice([1.0, 1.0, 0.9, 0.0]))


# ------------------------------------------------------------------ inputs

def _lens(case, g):
    lo, hi = case["lo"], case["hi"]
    if lo == hi:
        return torch.full((case["batch"],), hi, dtype=torch.int32, device="cuda")
    return torch.randint(lo, hi + 1, (case["batch"],), generator=g, device="cuda").to(torch.int32)


def _cache(case, lens, g):
    """A shuffled page table over a pool that could hold every sequence at its longest, with one page
    to spare that no sequence owns."""
    pages = (lens + PAGE - 1) // PAGE
    width = (case["hi"] + PAGE - 1) // PAGE
    total = case["batch"] * width
    ids = torch.randperm(total + 1, generator=g, device="cuda").to(torch.int32)
    first = torch.cumsum(pages, 0) - pages
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j[None, :]).clamp(max=total)
    table = torch.where(j[None, :] < pages[:, None], ids[at], torch.full_like(ids[at], -1)).to(torch.int32).contiguous()
    row = case["d_c"] + case["d_rope"]
    pool = torch.randn(total + 1, PAGE, row, generator=g, device="cuda", dtype=torch.float32)
    pool *= 0.75 + 0.5 * torch.rand(total + 1, PAGE, 1, generator=g, device="cuda")   # some keys stand out
    return table, pool.to(torch.bfloat16), int(ids[total])


def _slots(table, idx):
    """Row of the flattened pool that holds cache index idx [B, n] of each sequence."""
    return torch.gather(table.long(), 1, (idx // PAGE).long()) * PAGE + idx.long() % PAGE


def _old_mass(batch, width, typical, g):
    """Mass of earlier steps, a few times what one step adds."""
    m = 2.0 * typical * torch.exp(1.5 * torch.randn(batch, width, generator=g, device="cuda"))
    some = torch.rand(batch, width, generator=g, device="cuda") < 0.1
    return torch.where(some, torch.zeros_like(m), m)   # tokens that nobody looks at: ties


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    lens = _lens(case, g)
    s = dict(case=case, lens=lens)
    B = case["batch"]
    if case["op"] == "select":
        s["mass"] = _old_mass(B, case["hi"], 128.0 / case["hi"], g)
        s["budgets"] = (lens.double() * case["keep"]).ceil().to(torch.int32)
        k = max(1, min(case["hi"], math.ceil(case["hi"] * case["keep"])))
        s["keep_idx"] = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    s["table"], s["pool"], s["spare"] = _cache(case, lens, g)
    width = s["table"].shape[1] * PAGE
    s["mass"] = _old_mass(B, width, case.get("nq", 1) * case.get("heads", 128) / case["hi"], g)
    if case["op"] == "compact":
        # a choice of the kind that select makes: the first tokens, then a random part in order
        new = (lens.double() * case["keep"]).ceil().to(torch.int32)
        j = torch.arange(width, device="cuda")
        order = torch.rand(B, width, generator=g, device="cuda")
        order[:, : case["sink"]] = 2.0
        order = torch.where(j[None, :] < lens[:, None], order, torch.full_like(order, -1.0))
        rank = torch.argsort(torch.argsort(order, dim=1, descending=True), dim=1)
        idx = torch.where(rank < new[:, None], j[None, :], torch.full_like(rank, width)).sort(dim=1).values
        k = math.ceil(case["hi"] * case["keep"])
        s["keep_idx"] = torch.where(j[None, :k] < new[:, None], idx[:, :k], torch.full_like(idx[:, :k], -1)).to(torch.int32)
        s["new_lens"] = new
        return s
    nq, H, d_c, d_rope = case["nq"], case["heads"], case["d_c"], case["d_rope"]
    q = torch.randn(B, nq, H, d_c + d_rope, generator=g, device="cuda")
    q[..., :d_c] *= math.sqrt(case["nope"] / d_c)    # absorbed queries: W_UK^T of unit rows
    s["q_lat"] = q.to(torch.bfloat16)
    s["lse"] = torch.empty(B, nq, H, dtype=torch.float32, device="cuda")
    for b in range(B):                               # what the step's attention returned
        s["lse"][b] = torch.logsumexp(_scores64(s, b), dim=2).float()
    return s


def _scores64(s, b):
    """Scores [nq, H, len] of sequence b in 64 bits, -inf where a query does not see a key."""
    case, n = s["case"], int(s["lens"][b])
    nq, H = case["nq"], case["heads"]
    idx = torch.arange(n, device="cuda")
    rows = s["pool"].view(-1, s["pool"].shape[2])[_slots(s["table"][b : b + 1], idx[None])[0]].double()
    q = s["q_lat"][b].double().view(nq * H, -1)
    x = (q @ rows.T).view(nq, H, n) / math.sqrt(case["nope"] + case["d_rope"])
    hidden = idx[None, :] > (n - nq + torch.arange(nq, device="cuda"))[:, None]
    return x.masked_fill_(hidden[:, None, :], -math.inf)


# ------------------------------------------------------------------ the operators

def _dims(case):
    import head_latent_attention_07_b200 as mla
    return mla.MlaDims(n_heads=case.get("heads", 1), d_c=case["d_c"], d_rope=case["d_rope"], qk_nope=case.get("nope", 128),
                       v_head=128, d_model=1024, page_size=PAGE)


def _mass(s):
    case = s["case"]
    if own:
        import head_latent_attention_07_b200 as mla
        mla.mla_attn_mass(_dims(case), s["q_lat"], s["pool"], s["table"], s["lens"], s["lse"], s["mass"], decay=case["decay"])
        return {"mass": s["mass"]}
    nq, H, B = case["nq"], case["heads"], case["batch"]
    width = s["mass"].shape[1]
    j = torch.arange(width, device="cuda")
    lens = s["lens"].long()
    rows = s["pool"].view(-1, s["pool"].shape[2])[_slots(s["table"], j[None, :].expand(B, -1)).clamp_(min=0)].float()
    q = s["q_lat"].float().view(B, nq * H, -1)
    p = torch.bmm(q, rows.transpose(1, 2)).view(B, nq, H, width)
    p.mul_(1.0 / math.sqrt(case["nope"] + case["d_rope"])).sub_(s["lse"][..., None])
    last = lens[:, None] - nq + torch.arange(nq, device="cuda")[None, :]
    p.masked_fill_((j[None, None, :] > last[:, :, None])[:, :, None, :], -math.inf)
    w = torch.sum(p.exp_(), dim=(1, 2))
    older = torch.where(j[None, :] < lens[:, None] - nq, s["mass"], torch.zeros_like(s["mass"]))
    new = w if case["decay"] == 0.0 else case["decay"] * older + w
    s["mass"].copy_(torch.where(j[None, :] < lens[:, None], new, s["mass"]))
    return {"mass": s["mass"]}


def _select(s):
    case = s["case"]
    if own:
        import head_latent_attention_07_b200 as mla
        mla.mla_evict_select(s["mass"], s["lens"], s["budgets"], s["keep_idx"], s["new_lens"], n_sink=case["sink"],
                             n_recent=case["recent"])
        return {"keep_idx": s["keep_idx"], "new_lens": s["new_lens"]}
    width, k = s["mass"].shape[1], s["keep_idx"].shape[1]
    j = torch.arange(width, device="cuda")[None, :]
    lens, new = s["lens"].long()[:, None], torch.minimum(s["lens"], s["budgets"]).long()[:, None]
    sink = new.clamp(max=case["sink"])
    recent = torch.minimum(new - sink, torch.full_like(new, case["recent"]))
    value = torch.where((j < sink) | (j >= lens - recent), math.inf, s["mass"])
    value = torch.where(j < lens, value, -1.0)
    order = torch.sort(value, dim=1, descending=True, stable=True).indices
    kept = torch.where(j < new, order, width).sort(dim=1).values[:, :k]
    s["keep_idx"].copy_(torch.where(j[:, :k] < new, kept.to(torch.int32), s["keep_idx"]))
    s["new_lens"].copy_(new[:, 0])
    return {"keep_idx": s["keep_idx"], "new_lens": s["new_lens"]}


def _compact(s):
    case = s["case"]
    if own:
        import head_latent_attention_07_b200 as mla
        mla.mla_cache_compact(_dims(case), s["pool"], s["table"], s["lens"], s["keep_idx"], s["new_lens"], mass=s["mass"])
        return {"pool": s["pool"], "mass": s["mass"]}
    d_c, d_rope, B = case["d_c"], case["d_rope"], case["batch"]
    k = s["keep_idx"].shape[1]
    j = torch.arange(k, device="cuda")[None, :].expand(B, -1)
    valid = j < s["new_lens"][:, None]
    src = torch.where(valid, s["keep_idx"].long(), j)
    spare = s["spare"] * PAGE
    flat = s["pool"].view(-1, d_c + d_rope)
    rows = flat[torch.where(valid, _slots(s["table"], src), spare)]
    inv = THETA ** (-2.0 * torch.arange(d_rope // 2, device="cuda", dtype=torch.float64) / d_rope)
    angle = torch.remainder((j - src).double()[..., None] * inv, 2.0 * math.pi)   # 64 bits: far positions
    c, t = torch.cos(angle).float(), torch.sin(angle).float()
    x, y = rows[..., d_c::2].float(), rows[..., d_c + 1 :: 2].float()
    turned = torch.stack([x * c - y * t, x * t + y * c], dim=-1).flatten(2).to(rows.dtype)
    rows = torch.cat([rows[..., :d_c], torch.where(valid[..., None], turned, rows[..., d_c:])], dim=-1)
    flat[torch.where(valid, _slots(s["table"], j), spare)] = rows
    s["mass"][:, :k] = torch.where(valid, torch.gather(s["mass"], 1, src), s["mass"][:, :k])
    return {"pool": s["pool"], "mass": s["mass"]}


def run(state):
    return {"mass": _mass, "select": _select, "compact": _compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    B = case["batch"]
    tokens = B * (case["lo"] + case["hi"]) / 2
    if case["op"] == "select":
        return {"bytes": 4 * tokens + 4 * tokens * min(1.0, case["keep"]) + 12 * B, "flops": tokens}
    row = case["d_c"] + case["d_rope"]
    if case["op"] == "compact":
        kept = tokens * case["keep"]
        moved = max(0.0, kept - B * case["sink"])    # the first tokens stay where they are
        return {"bytes": 4 * kept + moved * (2 * 2 * row + 8), "flops": moved * 3 * case["d_rope"]}
    nq, H = case["nq"], case["heads"]
    keys = B * nq * ((case["lo"] + case["hi"]) / 2 - (nq - 1) / 2)
    return {"bytes": tokens * (2 * row + 4 + (4 if case["decay"] else 0)) + B * nq * H * (2 * row + 4),
            "flops": keys * H * 2 * row}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return None                                   # whole numbers only
    B = case["batch"]
    mass = s["mass"].double()
    if case["op"] == "mass":
        for b in range(B):
            n = int(s["lens"][b])
            w = torch.exp(_scores64(s, b) - s["lse"][b].double()[..., None]).sum(dim=(0, 1))
            if case["decay"]:
                w[: n - case["nq"]] += case["decay"] * mass[b, : n - case["nq"]]
            mass[b, :n] = w
        return {"mass": mass}
    d_c, d_rope = case["d_c"], case["d_rope"]
    before = s["pool"].view(-1, d_c + d_rope)
    after = before.double()
    i = torch.arange(d_rope // 2, device="cuda", dtype=torch.float64)
    for b in range(B):
        n = int(s["new_lens"][b])
        src = s["keep_idx"][b, :n].long()
        dst = torch.arange(n, device="cuda")
        rows = before[_slots(s["table"][b : b + 1], src[None])[0]].double()
        pairs = torch.view_as_complex(rows[:, d_c:].reshape(n, d_rope // 2, 2).contiguous())
        turn = (dst - src).double()[:, None] * torch.exp(-2.0 * i / d_rope * math.log(THETA))
        rows[:, d_c:] = torch.view_as_real(pairs * torch.polar(torch.ones_like(turn), turn)).reshape(n, d_rope)
        after[_slots(s["table"][b : b + 1], dst[None])[0]] = rows
        mass[b, :n] = s["mass"][b, src].double()
    return {"pool": after.view_as(s["pool"]), "mass": mass}
