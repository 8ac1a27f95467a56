"""What the paged-attention operators with a smaller cache are measured on.

Two ways to hold less than every head's keys and values of every token:

* eviction: `attn_verify_scored` is the decode / verification step that also adds up the attention
  weight every cached key has received; `kv_cache_evict` keeps, per sequence and kv-head, the
  most recent entries and the ones with the largest accumulated weight, and packs them;
* latent attention: a token caches one vector [c (d_c) ; k_r (d_r)] shared by all heads, from which
  head h's key is [W_uk[h] c ; k_r] and its value W_uv[h] c. `attn_latent_decode` is the absorbed
  form (n_q new tokens against the cached vectors), `attn_latent_prefill` the expanded form.

`run` computes the same thing in elementary torch operations (own = False) or by the calls a
user of the package makes (own = True).
"""
import math

import numpy as np
import torch

own = False

PAGE = 64    # tokens per cache page
D_R = 64     # the part of a latent cache row that every head's key takes as it is
DEV = "cuda"
BF = torch.bfloat16


# ---- cases -------------------------------------------------------------------------------------
def _scored(B, Hq, Hkv, d, nq, L):
    return {"op": "scored", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "nq": nq, "L": L}


def _evict(B, Hkv, d, L, budget, recent):
    return {"op": "evict", "B": B, "Hkv": Hkv, "d": d, "nq": 1, "L": L, "budget": budget,
            "recent": recent}


def _latent(B, H, d, d_c, nq, L):
    return {"op": "latent_decode", "B": B, "H": H, "d": d, "d_c": d_c, "nq": nq, "L": L}


def _prefill(B, T, H, d, d_c, prefix):
    return {"op": "latent_prefill", "B": B, "T": T, "H": H, "d": d, "d_c": d_c, "prefix": prefix}


def listed():
    return [
        # one user's chat a few hundred tokens in: launch latency is what counts
        {"name": "scored one sequence", **_scored(1, 16, 4, 64, 1, 517)},
        # a serving batch at the decode benchmark's sizes, sequences of 4k to 8k tokens
        {"name": "scored batch 8192", **_scored(32, 32, 8, 128, 1, 8192)},
        # four drafted tokens checked at once, weights of all four added up
        {"name": "scored verify 4", **_scored(16, 32, 8, 128, 4, 4097)},
        # a short conversation trimmed by a page
        {"name": "evict one page", **_evict(1, 4, 64, 1088, 1024, 64)},
        # a batch whose prompts are cut to half after prefill
        {"name": "evict batch half", **_evict(32, 8, 128, 8192, 4096, 256)},
        # two long documents cut to a small budget: choosing dominates
        {"name": "evict long", **_evict(2, 8, 128, 100033, 8192, 1024)},
        # one user, short context, a small model's heads
        {"name": "latent one sequence", **_latent(1, 16, 64, 256, 1, 517)},
        # a serving batch, sequences of 4k to 8k tokens
        {"name": "latent batch 8192", **_latent(32, 32, 128, 512, 1, 8192)},
        # three new tokens a sequence (two drafts checked), more query rows than one tile holds
        {"name": "latent verify 3", **_latent(16, 32, 128, 512, 3, 4097)},
        # a short first prompt
        {"name": "expanded short", **_prefill(1, 201, 16, 64, 256, 0)},
        # two whole prompts
        {"name": "expanded 4096", **_prefill(2, 4096, 32, 128, 512, 0)},
        # the next part of long prompts, after what is cached already (ragged)
        {"name": "expanded after prefix", **_prefill(3, 1000, 32, 128, 512, 2801)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scored", "evict", "latent", "prefill"])
    d = rng.choice([64, 128])
    if op == "scored":
        nq, Hkv = rng.choice([1, 1, 2, 3, 4]), rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if g * nq <= 16 and g * Hkv <= 64])
        B = _log(rng, 1, 32)
        L = max(nq, min(_log(rng, 1, 40000), 32 * 8 * 8192 // (B * Hkv)))
        return _scored(B, G * Hkv, Hkv, d, nq, L)
    if op == "evict":
        B, Hkv = _log(rng, 1, 32), rng.choice([1, 2, 3, 4, 8])
        L = min(_log(rng, 1, 120000), 32 * 8 * 8192 // (B * Hkv))
        budget = _log(rng, 1, min(L + 100, 16384))
        return _evict(B, Hkv, d, L, budget, rng.randint(0, budget))
    d_c = rng.choice([128, 256, 384, 512])
    if op == "latent":
        nq, H = rng.choice([1, 1, 2, 3, 4]), rng.choice([1, 4, 7, 16, 20, 32, 40])
        B = _log(rng, 1, 32)
        L = max(nq, min(_log(rng, 1, 100000), 32 * 8192 // (B * nq)))
        return _latent(B, H, d, d_c, nq, L)
    B, H, T = _log(rng, 1, 4), rng.choice([1, 3, 4, 8, 16, 32]), _log(rng, 1, 4096)
    prefix = rng.choice([0, _log(rng, 1, 4000)])
    prefix = min(prefix, max(0, 2 * 32 * 4096 * 4096 // (B * H * T) - T))
    return _prefill(B, T, H, d, d_c, prefix)


def _spread(n, L, low):
    """n lengths from L down to about L / 2, odd ones among them, none below `low`."""
    return [max(low, min(L, L - (i * (L // 2)) // max(1, n - 1) - i % 3)) for i in range(n)]


def _lens(c):
    return _spread(c["B"], c["L"], c["nq"])


def _prefill_lens(c):
    """(cached positions, new tokens) of each sequence: both ragged where there is a prefix."""
    if not c["prefix"]:
        return [0] * c["B"], [c["T"]] * c["B"]
    return _spread(c["B"], c["prefix"], 0), _spread(c["B"], c["T"], 1)


# ---- inputs ------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(g, B, per_seq, extra=0):
    """Tables of B sequences over a randomly ordered pool, and the pool's pages."""
    n = B * per_seq
    order = torch.randperm(n + extra, generator=g, device=DEV).to(torch.int32)
    return order[:n].view(B, per_seq).contiguous(), order[n:], n + extra


def _normal_pool(g, *shape):
    """A filled cache pool, made in its own type (a pool can be gigabytes)."""
    return torch.empty(*shape, device=DEV, dtype=BF).normal_(generator=g)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    B, op = c["B"], c["op"]
    if op in ("scored", "evict"):
        L, d, Hkv = c["L"], c["d"], c["Hkv"]
        per = -(-L // PAGE)
        keep = -(-min(L, c.get("budget", 1)) // PAGE) if op == "evict" else 0
        s["table"], rest, n = _pages(g, B, per, B * keep)
        s["k_pool"], s["v_pool"] = _normal_pool(g, n, Hkv, PAGE, d), _normal_pool(g, n, Hkv, PAGE, d)
        s["lens"] = _i32(_lens(c))
        # accumulated weight is skewed: most keys get little, some nothing at all
        w = torch.empty(B, Hkv, per * PAGE, device=DEV).exponential_(generator=g).pow_(3)
        w[torch.rand(w.shape, generator=g, device=DEV) < 0.1] = 0
        s["weights"] = w
        if op == "scored":
            nq, Hq = c["nq"], c["Hq"]
            s["q"] = _randn(g, B, nq, Hq, d)
            s["new_k"], s["new_v"] = _randn(g, B, nq, Hkv, d), _randn(g, B, nq, Hkv, d)
            s["o"] = torch.empty(B, nq, Hq, d, device=DEV, dtype=BF)
        else:
            s["dst"] = rest.view(B, keep).contiguous()
            s["weights_out"] = torch.zeros(B, Hkv, keep * PAGE, device=DEV)
            s["kept"] = torch.empty(B, Hkv, c["budget"], dtype=torch.int32, device=DEV)
            s["new_lens"] = torch.empty(B, dtype=torch.int32, device=DEV)
        return s
    H, d, d_c = c["H"], c["d"], c["d_c"]
    # up-projections of unit gain: keys and values of unit variance from latent ones
    s["w_uk"] = _randn(g, H, d, d_c, scale=d_c ** -0.5)
    s["w_uv"] = _randn(g, H, d, d_c, scale=d_c ** -0.5)
    if op == "latent_decode":
        new, total = c["nq"], c["L"]
        s["lens"] = _i32(_lens(c))
    else:
        new, total = c["T"], c["prefix"] + c["T"]
        pre, cur = _prefill_lens(c)
        s["prefix"], s["prompt"] = (_i32(pre), _i32(cur)) if c["prefix"] else (None, None)
    s["table"], _, n = _pages(g, B, -(-total // PAGE))
    s["pool"] = _normal_pool(g, n, PAGE, d_c + D_R)
    s["q"] = _randn(g, B, new, H, d + D_R)
    s["new_c"] = _randn(g, B, new, d_c + D_R)
    s["o"] = torch.zeros(B, new, H, d, device=DEV, dtype=BF)
    return s


def _workspace(s, size):
    """The scratch a program allocates once for its calls."""
    if "ws" not in s:
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s["ws"]


# ---- one pass ----------------------------------------------------------------------------------
def run(state):
    return {"scored": _run_scored, "evict": _run_evict, "latent_decode": _run_latent,
            "latent_prefill": _run_prefill}[state["case"]["op"]](state)


def _keys(pool, table):
    """A [n, H, PAGE, d] pool's rows in sequence order: [B, H, positions, d] in 32 bits."""
    x = pool[table.long()]  # [B, pages, H, PAGE, d]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, x.shape[4]).float()


def _place(table, pos):
    """(page, slot) of positions [B, n] under each sequence's table."""
    return table.long().gather(1, pos // PAGE), pos % PAGE


def _run_scored(s):
    c = s["case"]
    if own:
        import hybrid_mixer_decoding_b200 as hmd
        ws = _workspace(s, hmd.attn_verify_scored_workspace_size(
            c["nq"], c["B"], c["Hq"], c["Hkv"], c["d"], PAGE, c["L"]))
        hmd.attn_verify_scored(s["q"], s["new_k"], s["new_v"], s["k_pool"], s["v_pool"], s["weights"],
                               s["table"], s["lens"], c["L"], s["o"], ws)
        return {"o": s["o"], "weights": s["weights"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    B, nq, Hkv, d = c["B"], c["nq"], c["Hkv"], c["d"]
    G, lens, w = c["Hq"] // Hkv, s["lens"].long(), s["weights"]
    new = lens[:, None] - nq + torch.arange(nq, device=DEV)  # positions of the new tokens
    page, slot = _place(s["table"], new)
    s["k_pool"][page, :, slot] = s["new_k"]
    s["v_pool"][page, :, slot] = s["new_v"]
    K, V = _keys(s["k_pool"], s["table"]), _keys(s["v_pool"], s["table"])
    q = s["q"].float().view(B, nq, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nq * G, d)
    x = (q @ K.transpose(2, 3)).view(B, Hkv, nq, G, -1) / math.sqrt(d)
    pos = torch.arange(K.shape[2], device=DEV)
    x = x.masked_fill((pos > new[:, :, None])[:, None, :, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, nq * G, -1) @ V).view(B, Hkv, nq, G, d)
    s["o"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, nq, Hkv * G, d))
    old = torch.where((pos < lens[:, None] - nq)[:, None], w, torch.zeros_like(w))
    w.copy_(torch.where((pos < lens[:, None])[:, None], old + p.sum((2, 3)), w))
    return {"o": s["o"], "weights": w, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _run_evict(s):
    c = s["case"]
    out = {k: s[k] for k in ("kept", "new_lens", "weights_out", "k_pool", "v_pool")}
    if own:
        import hybrid_mixer_decoding_b200 as hmd
        hmd.kv_cache_evict(c["budget"], c["recent"], s["k_pool"], s["v_pool"], s["table"], s["lens"],
                           c["L"], s["weights"], s["dst"], s["weights_out"], s["kept"], s["new_lens"])
        return out
    Hkv, n = c["Hkv"], s["weights"].shape[2]
    lens, pos = s["lens"].long()[:, None, None], torch.arange(n, device=DEV)
    rank_of = s["weights"].masked_fill(pos >= lens - c["recent"], math.inf)  # recent ones first
    rank_of = rank_of.masked_fill(pos >= lens, -math.inf)
    best = torch.sort(rank_of, dim=2, descending=True, stable=True).indices
    m = min(n, c["budget"])
    best = best[:, :, :m].masked_fill(pos[:m] >= lens, n)  # fewer entries than the budget
    kept = torch.sort(best, dim=2).values
    live = kept < n
    s["kept"].fill_(-1)
    s["kept"][:, :, :m] = kept.masked_fill(~live, -1).to(torch.int32)
    s["new_lens"].copy_(torch.clamp(s["lens"], max=c["budget"]))
    b, h, j = live.nonzero(as_tuple=True)
    src = kept[b, h, j]
    page, slot = s["table"].long()[b, src // PAGE], src % PAGE
    page_to, slot_to = s["dst"].long()[b, j // PAGE], j % PAGE
    s["k_pool"][page_to, h, slot_to] = s["k_pool"][page, h, slot]
    s["v_pool"][page_to, h, slot_to] = s["v_pool"][page, h, slot]
    s["weights_out"][b, h, j] = s["weights"][b, h, src]
    return out


def _run_latent(s):
    c = s["case"]
    if own:
        import hybrid_mixer_decoding_b200 as hmd
        ws = _workspace(s, hmd.attn_latent_decode_workspace_size(
            c["nq"], c["B"], c["H"], c["d"], c["d_c"], D_R, PAGE, c["L"]))
        hmd.attn_latent_decode(s["q"], s["new_c"], s["w_uk"], s["w_uv"], s["pool"], s["table"],
                               s["lens"], c["L"], s["o"], ws)
        return {"o": s["o"], "pool": s["pool"]}
    B, nq, H, d, d_c = c["B"], c["nq"], c["H"], c["d"], c["d_c"]
    new = s["lens"].long()[:, None] - nq + torch.arange(nq, device=DEV)
    s["pool"][_place(s["table"], new)] = s["new_c"]
    C = s["pool"][s["table"].long()].reshape(B, -1, d_c + D_R).float()
    q = s["q"].float()
    qc = torch.einsum("bihn,hnc->bihc", q[..., :d], s["w_uk"].float())  # the query on the latent
    qc = torch.cat([qc, q[..., d:]], -1).view(B, nq * H, d_c + D_R)
    x = (qc @ C.transpose(1, 2)).view(B, nq, H, -1) / math.sqrt(d + D_R)
    pos = torch.arange(C.shape[1], device=DEV)
    x = x.masked_fill((pos > new[:, :, None])[:, :, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    oc = (p.view(B, nq * H, -1) @ C[..., :d_c]).view(B, nq, H, d_c)
    s["o"].copy_(torch.einsum("bihc,hvc->bihv", oc, s["w_uv"].float()))
    return {"o": s["o"], "pool": s["pool"]}


def _run_prefill(s):
    c = s["case"]
    if own:
        import hybrid_mixer_decoding_b200 as hmd
        ws = _workspace(s, hmd.attn_latent_prefill_workspace_size(
            c["B"], c["T"], c["H"], c["d"], c["d_c"], D_R, PAGE, c["prefix"]))
        hmd.attn_latent_prefill(s["q"], s["new_c"], s["w_uk"], s["w_uv"], s["pool"], s["table"],
                                s["o"], ws, prefix_lens=s["prefix"], max_prefix=c["prefix"],
                                prompt_lens=s["prompt"])
        return {"o": s["o"], "pool": s["pool"]}
    B, T, H, d, d_c = c["B"], c["T"], c["H"], c["d"], c["d_c"]
    tok = torch.arange(T, device=DEV)
    pre = (s["prefix"] if c["prefix"] else torch.zeros(B, device=DEV)).long()[:, None]
    live = tok < (s["prompt"].long()[:, None] if c["prefix"] else T)  # [B, T]
    live = live.expand(B, T)
    b, t = live.nonzero(as_tuple=True)
    at = pre[b, 0] + t
    s["pool"][s["table"].long()[b, at // PAGE], at % PAGE] = s["new_c"][b, t]
    C = s["pool"][s["table"].long()].reshape(B, -1, d_c + D_R).float()
    q = s["q"].float()
    K = torch.einsum("bjc,hnc->bhjn", C[..., :d_c], s["w_uk"].float())
    x = torch.einsum("bthn,bhjn->bhtj", q[..., :d], K)
    x += torch.einsum("bthr,bjr->bhtj", q[..., d:], C[..., d_c:])
    x *= 1 / math.sqrt(d + D_R)
    pos = torch.arange(C.shape[1], device=DEV)
    x.masked_fill_((pos > (pre + tok)[:, :, None])[:, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    x /= x.sum(-1, keepdim=True)
    V = torch.einsum("bjc,hvc->bhjv", C[..., :d_c], s["w_uv"].float())
    o = (x @ V).transpose(1, 2)
    s["o"].copy_(torch.where(live[:, :, None, None], o.to(BF), s["o"]))
    return {"o": s["o"], "pool": s["pool"]}


# ---- what a pass cannot do without -------------------------------------------------------------
def work(case):
    c = dict(case)
    op, B, d = c["op"], c["B"], c["d"]
    if op == "scored":
        keys, Hkv, nq, Hq = sum(_lens(c)), c["Hkv"], c["nq"], c["Hq"]
        old = keys - B * nq
        return {"bytes": old * Hkv * d * 2 * 2                 # cached keys and values
                + 2 * B * nq * Hkv * d * 2 * 2                 # the new ones, read and appended
                + 2 * B * nq * Hq * d * 2                      # q, o
                + (old + keys) * Hkv * 4,                      # weights read and written
                "flops": 4 * keys * nq * Hq * d}
    if op == "evict":
        lens, Hkv = _lens(c), c["Hkv"]
        kept = sum(min(n, c["budget"]) for n in lens)
        return {"bytes": sum(lens) * Hkv * 4                   # every weight
                + kept * Hkv * (2 * d * 2 * 2 + 4)             # kept rows and weights, moved
                + B * Hkv * c["budget"] * 4,
                "flops": sum(lens) * Hkv}
    H, d_c = c["H"], c["d_c"]
    row = (d_c + D_R) * 2
    weights = 2 * H * d * d_c * 2
    if op == "latent_decode":
        keys, nq = sum(_lens(c)), c["nq"]
        return {"bytes": (keys - B * nq) * row + 2 * B * nq * row + weights
                + B * nq * H * (2 * d + D_R) * 2,
                "flops": 2 * keys * nq * H * (2 * d_c + D_R) + 4 * B * nq * H * d * d_c}
    pre, cur = _prefill_lens(c)
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(pre, cur))
    rows = sum(pre) + sum(cur)
    return {"bytes": sum(pre) * row + 2 * sum(cur) * row + weights + sum(cur) * H * (2 * d + D_R) * 2,
            "flops": 2 * pairs * H * (2 * d + D_R) + 4 * rows * H * d * d_c}


# ---- the definitions in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"scored": _exact_scored, "evict": _exact_evict, "latent_decode": _exact_latent,
            "latent_prefill": _exact_prefill}[case["op"]](s)


def _rows(pool, table, n):
    """The first n positions of one sequence: [n, ...] in 64 bits, one page after another."""
    return torch.cat([pool[p] for p in table.tolist()], -2)[..., :n, :].double()


def _softmax64(x, hidden):
    x = torch.where(hidden, torch.full_like(x, -math.inf), x)
    return torch.softmax(x, -1)


def _exact_scored(s):
    c = s["case"]
    nq, Hkv, d = c["nq"], c["Hkv"], c["d"]
    G = c["Hq"] // Hkv
    o = torch.empty(c["B"], nq, c["Hq"], d, dtype=torch.float64, device=DEV)
    w = s["weights"].double()
    for b, L in enumerate(_lens(c)):
        K, V = _rows(s["k_pool"], s["table"][b], L), _rows(s["v_pool"], s["table"][b], L)
        K[:, L - nq:], V[:, L - nq:] = s["new_k"][b].transpose(0, 1), s["new_v"][b].transpose(0, 1)
        w[b, :, L - nq:L] = 0
        for i in range(nq):
            last = L - nq + i
            for h in range(c["Hq"]):
                p = torch.softmax(K[h // G, :last + 1] @ s["q"][b, i, h].double() / d ** 0.5, 0)
                o[b, i, h] = p @ V[h // G, :last + 1]
                w[b, h // G, :last + 1] += p
    return {"o": o, "weights": w, "k_pool": None, "v_pool": None}


def _exact_evict(s):
    c = s["case"]
    w = s["weights"].double().cpu().numpy()
    kept = np.full((c["B"], c["Hkv"], c["budget"]), -1, np.int32)
    out = np.zeros(tuple(s["weights_out"].shape))
    new = []
    for b, L in enumerate(_lens(c)):
        new.append(min(L, c["budget"]))
        first = max(0, L - c["recent"])  # the recent entries start here
        for h in range(c["Hkv"]):
            order = np.lexsort((np.arange(first), -w[b, h, :first]))
            n_old = max(0, min(first, c["budget"] - (L - first)))
            at = np.sort(np.concatenate([order[:n_old], np.arange(max(first, L - c["budget"]), L)]))
            kept[b, h, :len(at)] = at
            out[b, h, :len(at)] = w[b, h, at]
    return {"kept": kept, "new_lens": np.array(new, np.int32), "weights_out": out, "k_pool": None,
            "v_pool": None}


def _exact_latent(s):
    c = s["case"]
    nq, H, d, d_c = c["nq"], c["H"], c["d"], c["d_c"]
    o = torch.empty(c["B"], nq, H, d, dtype=torch.float64, device=DEV)
    for b, L in enumerate(_lens(c)):
        C = _rows(s["pool"], s["table"][b], L)
        C[L - nq:] = s["new_c"][b]
        _expanded(s, b, C, L - nq, nq, o)
    return {"o": o, "pool": None}


def _exact_prefill(s):
    c = s["case"]
    o = torch.zeros(c["B"], c["T"], c["H"], c["d"], dtype=torch.float64, device=DEV)
    for b, (pre, cur) in enumerate(zip(*_prefill_lens(c))):
        C = torch.cat([_rows(s["pool"], s["table"][b], pre), s["new_c"][b, :cur].double()])
        _expanded(s, b, C, pre, cur, o)
    return {"o": o, "pool": None}


def _expanded(s, b, C, first, n, o):
    """Every head's own keys and values from the latent rows C, for the n queries from `first`."""
    c = s["case"]
    d, d_c = c["d"], c["d_c"]
    hidden = torch.arange(len(C), device=DEV)[None] > first + torch.arange(n, device=DEV)[:, None]
    for h in range(c["H"]):
        K = torch.cat([C[:, :d_c] @ s["w_uk"][h].double().T, C[:, d_c:]], 1)
        p = _softmax64(s["q"][b, :n, h].double() @ K.T / (d + D_R) ** 0.5, hidden)
        o[b, :n, h] = p @ (C[:, :d_c] @ s["w_uv"][h].double().T)
