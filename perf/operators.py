"""Cases of the operators around draft-tree verification, and their plain forms.

Four operators of a serving step, on the paged cache and the trees that the
verification calls use:

* ``append``: a ragged batch of new tokens; queries and keys rotated by their
  positions, keys and values written into the cache's pages;
* ``attend``: the attention of those tokens over the cache (prefix and chunk,
  causal, with an optional window and an optional tanh cap on the scores);
* ``logits``: the target model's rows of a draft tree turned into what
  acceptance reads: bias, penalties for tokens of the history and of the
  node's own path, grammar mask, temperature, softmax;
* ``counts``: the per-token history that the penalties read.

``run`` computes them with elementary torch operations, or (``own``) through
the framework's entry points.
"""
import math
import random

import torch

own = False

GB = 1 << 30


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the smallest call: one new token of one short conversation
        dict(name="attend_one_token", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128,
             block=16, batch=1, new_lo=1, new_hi=1, prefix_lo=300, prefix_hi=300, window=0,
             cap=0.0, shape=1),
        # plain decoding of a full batch: every sequence one token, long ragged prefixes
        dict(name="attend_decode_b64", op="attend", dtype="bf16", heads=32, kv_heads=8, dim=128,
             block=16, batch=64, new_lo=1, new_hi=1, prefix_lo=512, prefix_hi=8192, window=0,
             cap=0.0, shape=2),
        # mixed batch: prompt chunks of odd lengths beside sequences that decode
        dict(name="attend_ragged_chunks", op="attend", dtype="bf16", heads=32, kv_heads=8,
             dim=128, block=16, batch=7, new_lo=1, new_hi=1500, prefix_lo=0, prefix_hi=5000,
             window=0, cap=0.0, shape=5),
        # the largest: one chunk of a long prompt over what came before it
        dict(name="attend_long_chunk", op="attend", dtype="bf16", heads=28, kv_heads=4, dim=128,
             block=16, batch=1, new_lo=4096, new_hi=4096, prefix_lo=12281, prefix_hi=12281,
             window=0, cap=0.0, shape=4),
        # layers with a sliding window and capped scores, head size 64, larger pages
        dict(name="attend_window_cap", op="attend", dtype="bf16", heads=16, kv_heads=2, dim=64,
             block=32, batch=3, new_lo=200, new_hi=1200, prefix_lo=1000, prefix_hi=8000,
             window=1024, cap=30.0, shape=5),
        # float32 caches, as the framework's smallest workload has them
        dict(name="attend_f32", op="attend", dtype="f32", heads=2, kv_heads=1, dim=64, block=16,
             batch=4, new_lo=7, new_hi=250, prefix_lo=64, prefix_hi=900, window=0, cap=0.0,
             shape=6),
        # the nodes of a batch of draft trees: rotary positions by depth, half layout
        dict(name="append_trees", op="append", dtype="bf16", heads=32, kv_heads=8, dim=128,
             block=16, batch=32, new_lo=26, new_hi=26, prefix_lo=512, prefix_hi=8192, layout="half",
             rotate=128, scaling="none", factor=1.0, by_depth=True, shape=7),
        # prompt chunks: interleaved pairs in half of the head, scaled for a long context
        dict(name="append_prompts", op="append", dtype="bf16", heads=28, kv_heads=4, dim=128,
             block=16, batch=4, new_lo=1000, new_hi=4100, prefix_lo=0, prefix_hi=90000,
             layout="interleaved", rotate=64, scaling="ramp", factor=8.0, by_depth=False,
             shape=8),
        # probabilities of every node of a batch of draft trees
        dict(name="logits_trees_probs", op="logits", dtype="f32", batch=32, nodes=26,
             vocab=128256, probs=True, bias=True, grammar=True, penalties=True, shape=9),
        # logits of a few chains from half-precision rows, for greedy acceptance
        dict(name="logits_chains", op="logits", dtype="bf16", batch=4, nodes=6, vocab=152064,
             probs=False, bias=False, grammar=True, penalties=True, shape=10),
        # the histories of new prompts
        dict(name="counts_prompts", op="counts", batch=32, vocab=128256, new_lo=200, new_hi=8192,
             prompt=True, shape=11),
        # the tokens that one step accepted
        dict(name="counts_accepted", op="counts", batch=128, vocab=128256, new_lo=1, new_hi=6,
             prompt=False, shape=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "logits", "counts"])
    shape = rng.randrange(1 << 30)
    if op in ("attend", "append"):
        heads, kv_heads = rng.choice([(32, 8), (28, 4), (16, 2), (8, 8), (6, 2), (24, 1), (2, 1)])
        c = dict(op=op, dtype=rng.choice(["bf16"] * 4 + ["f32"]), heads=heads, kv_heads=kv_heads,
                 dim=rng.choice([64, 128, 128]), block=rng.choice([16, 16, 32, 48, 128]),
                 batch=_log_int(rng, 1, 64), shape=shape)
        top = _log_int(rng, 1, 4096)
        c["new_lo"], c["new_hi"] = rng.choice([0, 1, max(1, top // 3)]), top
        far = _log_int(rng, 0, 16000)
        c["prefix_lo"], c["prefix_hi"] = rng.choice([0, far // 4, far]), far
        if op == "attend":
            c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4000)])
            c["cap"] = rng.choice([0.0, 0.0, rng.uniform(5.0, 60.0)])
        else:
            c["layout"] = rng.choice(["half", "interleaved"])
            c["rotate"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 32])
            c["scaling"] = rng.choice(["none", "linear", "ramp", "bands"])
            c["factor"] = 1.0 if c["scaling"] == "none" else rng.uniform(1.5, 16.0)
            c["by_depth"] = rng.choice([False, True])
        # no more work than the largest listed cases of the operator
        while True:
            w = work(c)
            if sum(_lens(c)[0]) == 0:
                c["new_hi"] = c["new_lo"] = 1
            elif c["dtype"] == "f32" and w["flops"] > 4e10 or w["flops"] > 6e11 or w["bytes"] > 0.4 * GB:
                if c["batch"] > 4 or (c["new_hi"] <= 64 and c["batch"] > 1):
                    c["batch"] = c["batch"] // 2
                else:
                    c["new_hi"] = max(1, c["new_hi"] // 2)
                    c["new_lo"] = min(c["new_lo"], c["new_hi"])
            else:
                return c
    if op == "logits":
        c = dict(op="logits", dtype=rng.choice(["f32", "f32", "bf16"]), batch=_log_int(rng, 1, 64),
                 nodes=_log_int(rng, 1, 64),
                 vocab=rng.choice([128256, 152064, _log_int(rng, 1000, 260000)]),
                 probs=rng.choice([True, True, False]), bias=rng.choice([True, False]),
                 grammar=rng.choice([True, False]), penalties=rng.choice([True, True, False]),
                 shape=shape)
        while c["batch"] * c["nodes"] * c["vocab"] > 32 * 26 * 128256:
            if c["batch"] > c["nodes"]:
                c["batch"] //= 2
            else:
                c["nodes"] //= 2
        return c
    prompt = rng.choice([True, False])
    return dict(op="counts", batch=_log_int(rng, 1, 32 if prompt else 200),
                vocab=rng.choice([128256, _log_int(rng, 1000, 128000)]), new_lo=rng.choice([0, 1]),
                new_hi=_log_int(rng, 2, 8000) if prompt else _log_int(rng, 2, 64), prompt=prompt,
                shape=shape)


def _lens(c):
    """New tokens and prefix lengths of the sequences: the case's own, whatever the seed."""
    r = random.Random(c["shape"])
    n = [_log_int(r, c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    p = [_log_int(r, c["prefix_lo"], c["prefix_hi"]) if "prefix_lo" in c else 0 for _ in n]
    return n, p


def _params(c):
    """Penalties and temperatures of the sequences of a logits case."""
    r = random.Random(c["shape"] + 1)
    rep = [r.choice([1.0, 1.1, 1.3]) for _ in range(c["batch"])]
    freq = [r.choice([0.0, 0.2, -0.1]) for _ in rep]
    pres = [r.choice([0.0, 0.5]) for _ in rep]
    temp = [r.choice([0.6, 0.8, 1.0]) for _ in rep]
    return rep, freq, pres, temp


def work(case):
    c = case
    if c["op"] == "logits":
        cells = c["batch"] * c["nodes"] * c["vocab"]
        b = cells * ((4 if c["dtype"] == "f32" else 2) + 4)
        b += c["batch"] * c["vocab"] * 4 * (int(c["bias"]) + int(c["penalties"]))
        b += cells / 8 * int(c["grammar"])
        return {"bytes": b, "flops": cells * (6.0 if c["probs"] else 3.0)}
    n, p = _lens(c)
    if c["op"] == "counts":
        b = sum(n) * 4 + (c["batch"] * c["vocab"] * 4 if c["prompt"] else sum(n) * 8)
        return {"bytes": max(1, b), "flops": 0}
    e = 2 if c["dtype"] == "bf16" else 4
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        return {"bytes": max(1, 2 * sum(n) * (h + 2 * g) * d * e), "flops": sum(n) * (h + g) * c["rotate"] * 3.0}
    pairs = keys = 0
    for ni, pi in zip(n, p):
        if ni == 0:
            continue
        w = c["window"] or pi + ni
        full = max(0, min(ni, pi + ni - w))        # tokens whose window is full
        rest = ni - full
        pairs += full * w + rest * pi + rest * (rest + 1) // 2
        keys += min(pi + ni, w + ni - 1)
    return {"bytes": max(1, 2 * sum(n) * h * d * e + 2 * keys * g * d * e), "flops": 4.0 * pairs * h * d}


# --------------------------------------------------------------------------
# what a user's program has in hand
# --------------------------------------------------------------------------

def _pages(c, n, p, gen):
    """Block table of a paged cache, blocks in shuffled order: attention reads every sequence
    whole; where tokens are only appended, the blocks before them have been given back."""
    last = [max(1, -(-(a + b) // c["block"])) for a, b in zip(n, p)]
    first = [b // c["block"] if c["op"] == "append" else 0 for b in p]
    first = [min(f, t - 1) for f, t in zip(first, last)]
    need = sum(last) - sum(first)
    order = torch.randperm(need, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((len(n), max(last)), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(max(last), device="cuda")
    lo, hi = (torch.tensor(t, device="cuda")[:, None] for t in (first, last))
    table[(at >= lo) & (at < hi)] = order
    return table, need


def _starts(n):
    s = [0]
    for a in n:
        s.append(s[-1] + a)
    return s


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["op"] == "logits":
        s = _prepare_logits(c, gen, i32)
    elif c["op"] == "counts":
        s = _prepare_counts(c, gen, i32)
    else:
        s = _prepare_tokens(c, gen, i32)
    s["status"] = torch.zeros(c["batch"], **i32)
    s["c"] = c
    if own:
        import eagle_speculative_decoding_parent_gb300 as tv
        s["tv"] = tv
        if c["op"] == "attend":
            need = tv.chunk_attention_workspace(s["q"].shape[0], c["batch"], c["heads"],
                                                c["kv_heads"], c["dim"], s["q"].dtype)
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        if c["op"] == "append":
            s["rope"] = tv.rope_table(c["rotate"], theta=500000.0, interleaved=c["layout"] != "half",
                                      scaling=c["scaling"], factor=c["factor"],
                                      original_len=8192)
    return s


def _prepare_tokens(c, gen, i32):
    n, p = _lens(c)
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    table, blocks = _pages(c, n, p, gen)
    starts = _starts(n)
    T = starts[-1]
    s = {"n": n, "p": p, "starts": starts, "table": table, "q_start": torch.tensor(starts, **i32),
         "prefix": torch.tensor(p, **i32)}
    if c["op"] == "attend":
        s["q"] = torch.randn((T, h, d), generator=gen, device="cuda", dtype=dt)
        s["k_cache"] = torch.randn((blocks, g, c["block"], d), generator=gen, device="cuda", dtype=dt)
        s["v_cache"] = torch.randn((blocks, g, c["block"], d), generator=gen, device="cuda", dtype=dt)
        s["out"] = torch.empty((T, h, d), device="cuda", dtype=dt)
        return s
    # queries, keys and values as a fused projection leaves them: views of one row
    qkv = torch.randn((T, h + 2 * g, d), generator=gen, device="cuda", dtype=dt)
    s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
    s["q_out"] = torch.empty((T, h, d), device="cuda", dtype=dt)
    s["k_cache"] = torch.zeros((blocks, g, c["block"], d), device="cuda", dtype=dt)
    s["v_cache"] = torch.zeros((blocks, g, c["block"], d), device="cuda", dtype=dt)
    # position of each token in its sequence, and the sequence it belongs to
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
    at = torch.arange(T, device="cuda") - s["q_start"][:-1].long()[seq]
    slot = s["prefix"].long()[seq] + at
    s["seq"], s["slot"] = seq, slot
    s["positions"] = None
    if c["by_depth"]:
        depth = torch.minimum(at, torch.randint(0, 7, (T,), generator=gen, device="cuda"))
        s["positions"] = (s["prefix"].long()[seq] + depth).to(torch.int32)
    return s


def _prepare_logits(c, gen, i32):
    B, N, V = c["batch"], c["nodes"], c["vocab"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s = {"logits": torch.randn((B, N, V), generator=gen, device="cuda", dtype=dt).mul_(3.0),
         "out": torch.empty((B, N, V), device="cuda"), "mask": None, "tokens": None, "hist": None,
         "bias": None, "grammar": None, "rep": None, "freq": None, "pres": None, "temp": None}
    f32 = dict(dtype=torch.float32, device="cuda")
    rep, freq, pres, temp = _params(c)
    s["temp"] = torch.tensor(temp, **f32)
    if c["penalties"]:
        s["rep"], s["freq"], s["pres"] = (torch.tensor(x, **f32) for x in (rep, freq, pres))
        # random trees in topological order, as ancestor bits; few distinct tokens, so paths repeat
        parent = (torch.rand((B, N), generator=gen, device="cuda") * torch.arange(N, device="cuda")).long()
        rel = torch.eye(N, dtype=torch.bool, device="cuda").expand(B, N, N).clone()
        for i in range(1, N):
            rel[:, i] |= rel[torch.arange(B, device="cuda"), parent[:, i]]
        bits = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(N, device="cuda")
        s["mask"] = (rel * bits).sum(2)
        s["tokens"] = torch.randint(0, V, (B, max(1, N // 2)), generator=gen, device="cuda")
        s["tokens"] = s["tokens"].repeat(1, 3)[:, :N].to(torch.int32).contiguous()
        # history: a few thousand tokens of the prompt (sign bit) and of the output (counts)
        hist = torch.zeros((B, V), **i32)
        some = torch.randint(0, V, (B, 2000), generator=gen, device="cuda")
        hist.scatter_add_(1, some[:, :1200], torch.ones((B, 1200), **i32))
        hist.scatter_add_(1, s["tokens"].long(), torch.ones((B, N), **i32))
        flag = torch.zeros((B, V), dtype=torch.bool, device="cuda").scatter_(1, some[:, 800:], True)
        s["hist"] = torch.where(flag, hist | -(1 << 31), hist)
    if c["bias"]:
        r = torch.rand((B, V), generator=gen, device="cuda")
        s["bias"] = torch.where(r < 0.01, 500.0 * (r - 0.005), torch.zeros((), device="cuda"))
    if c["grammar"]:
        words = (V + 31) // 32
        s["grammar"] = torch.randint(-(1 << 31), 1 << 31, (B, N, words), generator=gen, device="cuda",
                                     dtype=torch.int64).to(torch.int32)
        # every eighth row allows only a few tokens
        few = torch.rand((B, N, words), generator=gen, device="cuda") < 0.001
        tight = (torch.arange(B * N, device="cuda").view(B, N, 1) % 8) == 5
        s["grammar"] = torch.where(tight & ~few, torch.zeros_like(s["grammar"]), s["grammar"])
    return s


def _prepare_counts(c, gen, i32):
    n, _ = _lens(c)
    B, V = c["batch"], c["vocab"]
    s = {"n": n, "hist": torch.zeros((B, V), **i32), "starts": None}
    # token ids lean towards the frequent end of the vocabulary
    if c["prompt"]:
        starts = _starts(n)
        s["starts"] = torch.tensor(starts, **i32)
        r = torch.rand(starts[-1], generator=gen, device="cuda")
        s["tokens"] = (r ** 3 * V).to(torch.int32).clamp_(max=V - 1)
        s["seq"] = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
    else:
        # rows of accepted tokens, padded with -1, as acceptance writes them
        r = torch.rand((B, c["new_hi"]), generator=gen, device="cuda")
        tok = (r ** 3 * V).to(torch.int32).clamp_(max=V - 1)
        live = torch.arange(c["new_hi"], device="cuda") < torch.tensor(n, device="cuda")[:, None]
        s["tokens"] = torch.where(live, tok, torch.full_like(tok, -1))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    if c["op"] == "attend":
        if own:
            s["tv"].chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"],
                                    s["prefix"], s["out"], s["status"], s["workspace"],
                                    softcap=c["cap"], window=c["window"])
            return s["out"]
        return _attend(s, c)
    if c["op"] == "append":
        if own:
            s["tv"].chunk_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"],
                                    s["q_start"], s["prefix"], s["status"], q_out=s["q_out"],
                                    rope=s["rope"], positions=s["positions"])
            return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
        return _append(s, c)
    if c["op"] == "logits":
        if own:
            s["tv"].tree_logits_process(s["logits"], s["out"], s["status"], probs=c["probs"],
                                        mask=s["mask"], draft_tokens=s["tokens"], counts=s["hist"],
                                        bias=s["bias"], grammar=s["grammar"], repetition=s["rep"],
                                        frequency=s["freq"], presence=s["pres"],
                                        temperature=s["temp"])
            return s["out"]
        return _logits(s, c)
    if own:
        s["tv"].token_counts_update(s["hist"], s["tokens"], s["status"], starts=s["starts"],
                                    clear=c["prompt"], prompt=c["prompt"])
        return s["hist"]
    return _counts(s, c)


def _attend_rows(s, c, q, table, prefix):
    """Softmax attention of q [S, n, heads, d] over the pages of S sequences."""
    S, n, h, d = q.shape
    g, w = c["kv_heads"], h // c["kv_heads"]
    pages = table.clamp_min(0).long()
    k = s["k_cache"][pages].transpose(2, 3).flatten(1, 2).float()        # [S, L, g, d]
    v = s["v_cache"][pages].transpose(2, 3).flatten(1, 2).float()
    at = prefix[:, None] + torch.arange(n, device="cuda")                # [S, n]
    keys = torch.arange(k.shape[1], device="cuda")
    hidden = keys > at[..., None]
    if c["window"]:
        hidden = hidden | (keys <= at[..., None] - c["window"])
    qf = q.float().view(S, n, g, w, d).permute(0, 2, 3, 1, 4).reshape(S, g, w * n, d)
    x = (qf @ k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d)).view(S, g, w, n, -1)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    x.masked_fill_(hidden[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = x.view(S, g, w * n, -1) @ v.transpose(1, 2)
    o = o / x.sum(-1).view(S, g, w * n, 1)
    return o.view(S, g, w, n, d).permute(0, 3, 1, 2, 4).reshape(S, n, h, d).to(q.dtype)


def _attend(s, c):
    out = torch.empty_like(s["q"])
    # sequences with one token in one batch, the others one by one
    ones = [b for b, a in enumerate(s["n"]) if a == 1]
    if ones:
        b = torch.tensor(ones, device="cuda")
        rows = s["q_start"][b].long()
        most = max(-(-(s["p"][i] + 1) // c["block"]) for i in ones)
        out[rows] = _attend_rows(s, c, s["q"][rows][:, None], s["table"][b, :most], s["prefix"][b])[:, 0]
    for b, a in enumerate(s["n"]):
        if a > 1:
            lo, most = s["starts"][b], -(-(s["p"][b] + a) // c["block"])
            out[lo:lo + a] = _attend_rows(s, c, s["q"][None, lo:lo + a], s["table"][b:b + 1, :most],
                                          s["prefix"][b:b + 1])[0]
    return out


def _frequencies(c):
    """Radians per position of each rotated pair, in 64 bits, and the factor on cos and sin."""
    dim, theta, old, factor = c["rotate"], 500000.0, 8192, c["factor"]
    j = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
    f = theta ** (-2.0 * j / dim)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "bands":
        # long waves slowed down, short ones kept, a blend between the two borders
        turns = old * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor), 1.0
    if c["scaling"] == "ramp":
        # a linear ramp over the pairs between 32 turns and one turn of the old context
        edge = [dim * math.log(old / (t * 2.0 * math.pi)) / (2.0 * math.log(theta)) for t in (32.0, 1.0)]
        lo, hi = max(0, math.floor(edge[0])), min(dim - 1, math.ceil(edge[1]))
        slow = ((j - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - slow) + f / factor * slow, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotate(x, cos, sin, c):
    m, half = c["rotate"], c["rotate"] // 2
    y = x.float().clone()
    a, b = (slice(0, half), slice(half, m)) if c["layout"] == "half" else (slice(0, m, 2), slice(1, m, 2))
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a] = u * cos - v * sin
    y[..., b] = v * cos + u * sin
    return y.to(x.dtype)


def _append(s, c):
    f, amp = _frequencies(c)
    pos = s["slot"] if s["positions"] is None else s["positions"]
    angle = pos.double()[:, None] * f
    cos, sin = ((t * amp).float()[:, None] for t in (angle.cos(), angle.sin()))
    block = s["table"][s["seq"], s["slot"] // c["block"]].long()
    row = s["slot"] % c["block"]
    s["k_cache"][block, :, row] = _rotate(s["k"], cos, sin, c)
    s["v_cache"][block, :, row] = s["v"]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c))
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _logits(s, c):
    B, N, V = c["batch"], c["nodes"], c["vocab"]
    x = s["logits"].float()
    if s["bias"] is not None:
        x = x + s["bias"][:, None]
    if s["rep"] is not None:
        # output counts: the history's, and the node's path behind the root
        on_path = (s["mask"][:, :, None] >> torch.arange(N, device="cuda")) & 1
        on_path[:, :, 0] = 0
        told = s["tokens"].long()[:, None].expand(B, N, N)
        n_out = (s["hist"] & 0x7FFFFFFF)[:, None].repeat(1, N, 1)
        n_out.scatter_add_(2, told, on_path.to(torch.int32))
        seen = (s["hist"] < 0)[:, None] | (n_out > 0)
        rep, freq, pres = (s[k][:, None, None] for k in ("rep", "freq", "pres"))
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        x = x - freq * n_out - pres * (n_out > 0)
    x = x / s["temp"][:, None, None]
    if s["grammar"] is not None:
        bits = (s["grammar"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = x.masked_fill(bits.view(B, N, -1)[..., :V] == 0, -math.inf)
    if not c["probs"]:
        return x
    top = x.amax(-1, keepdim=True)
    e = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def _counts(s, c):
    V = c["vocab"]
    flat = s["hist"].view(-1)
    if c["prompt"]:
        s["hist"].zero_()
        flat[s["seq"] * V + s["tokens"].long()] = -(1 << 31)
        return s["hist"]
    live = (s["tokens"] >= 0).to(torch.int32)
    s["hist"].scatter_add_(1, s["tokens"].clamp_min(0).long(), live)
    return s["hist"]


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "attend":
        return _attend_exact(s, c)
    if c["op"] == "append":
        return _append_exact(s, c)
    if c["op"] == "logits":
        return _logits_exact(s, c)
    return None


def _attend_exact(s, c):
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    out = torch.zeros((s["starts"][-1], h, d), dtype=torch.float64, device="cuda")
    step = 1024                                            # query rows at once
    for b, n in enumerate(s["n"]):
        p, lo = s["p"][b], s["starts"][b]
        if n == 0:
            continue
        t = torch.arange(p + n, device="cuda")
        block, row = s["table"][b][t // c["block"]].long(), t % c["block"]
        for kv in range(g):
            key, val = s["k_cache"][block, kv, row].double(), s["v_cache"][block, kv, row].double()
            for i in range(0, n, step):
                here = torch.arange(i, min(n, i + step), device="cuda")
                z = torch.einsum("ihd,td->iht", s["q"][lo + here, kv * (h // g):(kv + 1) * (h // g)].double(), key)
                z = z / d ** 0.5
                if c["cap"] > 0:
                    z = torch.tanh(z / c["cap"]) * c["cap"]
                ok = t[None] <= p + here[:, None]
                if c["window"] > 0:
                    ok = ok & (t[None] > p + here[:, None] - c["window"])
                z = torch.where(ok[:, None], z, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                out[lo + here, kv * (h // g):(kv + 1) * (h // g)] = torch.einsum("iht,td->ihd", torch.softmax(z, -1), val)
    return out


def _append_exact(s, c):
    m = c["rotate"]
    old, theta, k = 8192.0, 500000.0, c["factor"]
    rate, amp = [], 1.0
    for j in range(m // 2):
        f = math.pow(theta, -2.0 * j / m)
        if c["scaling"] == "linear":
            f /= k
        elif c["scaling"] == "bands":
            wave = 2.0 * math.pi / f
            if wave > old / 1.0:
                f /= k
            elif wave > old / 4.0:
                mix = (old / wave - 1.0) / 3.0
                f = (1.0 - mix) * f / k + mix * f
        elif c["scaling"] == "ramp":
            first = max(0, math.floor(m * math.log(old / (64.0 * math.pi)) / (2.0 * math.log(theta))))
            last = min(m - 1, math.ceil(m * math.log(old / (2.0 * math.pi)) / (2.0 * math.log(theta))))
            r = min(1.0, max(0.0, (j - first) / (last - first if last > first else 0.001)))
            f = f * (1.0 - r) + r * f / k
            amp = 0.1 * math.log(k) + 1.0
        rate.append(f)
    pos = (s["slot"] if s["positions"] is None else s["positions"].long()).double()
    turn = torch.polar(torch.full((1,), amp, dtype=torch.float64, device="cuda"),
                       torch.outer(pos, torch.tensor(rate, dtype=torch.float64, device="cuda")))[:, None]

    def spun(x):
        x = x.double()
        pairs = x[..., :m].unflatten(-1, (2, m // 2)).transpose(-1, -2) if c["layout"] == "half" else x[..., :m].unflatten(-1, (m // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
        return torch.cat([z, x[..., m:]], -1)

    place = s["table"][s["seq"], torch.div(s["slot"], c["block"], rounding_mode="floor")].long() * c["block"] + s["slot"] % c["block"]
    caches = []
    for name, rows in (("k_cache", spun(s["k"])), ("v_cache", s["v"].double())):
        flat = s[name].double().transpose(1, 2).flatten(0, 1).clone()   # [slots, g, d]
        flat[place] = rows
        caches.append(flat.unflatten(0, (-1, c["block"])).transpose(1, 2).contiguous())
    return {"q": spun(s["q"]), "k": caches[0], "v": caches[1]}


def _logits_exact(s, c):
    B, N, V = c["batch"], c["nodes"], c["vocab"]
    rows = []
    hidden = torch.tensor(-math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        z = s["logits"][b].double()
        if s["bias"] is not None:
            z = z + s["bias"][b].double()
        if s["rep"] is not None:
            hist = s["hist"][b].long()
            # occurrences of each of the path's tokens: ancestors x one-hot tokens
            rel = ((s["mask"][b][:, None] >> torch.arange(N, device="cuda")) & 1).double()
            rel[:, 0] = 0.0
            uniq, which = torch.unique(s["tokens"][b].long(), return_inverse=True)
            occurs = torch.zeros((N, V), dtype=torch.float64, device="cuda")
            occurs[:, uniq] = rel @ torch.nn.functional.one_hot(which, uniq.numel()).double()
            times = occurs + (hist % (1 << 31)).double()
            r, fr, pr = (s[k][b].double() for k in ("rep", "freq", "pres"))
            told = (times > 0) | (hist < 0)
            z = torch.where(told & (z > 0), z / r, torch.where(told, z * r, z))
            z = z - fr * times - torch.where(times > 0, pr, torch.zeros_like(pr))
        z = z / s["temp"][b].double()
        if s["grammar"] is not None:
            ids = torch.arange(V, device="cuda")
            word = s["grammar"][b].long()[:, ids // 32]
            z = torch.where((word >> (ids % 32)) % 2 != 0, z, hidden)
        if c["probs"]:
            z = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
            rows.append(z)
        else:
            rows.append(z)
    return torch.stack(rows)
