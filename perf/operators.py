"""Cases of the serving operators around the packed-state pool, in plain torch and through the library.

Three operators carry a request from its prompt to its beams:

* "plan":   block tables and slot maps of a ragged batch, built on the GPU from the request lengths
            (stepq.RequestPlan.build);
* "prompt": linear attention with a decay, many tokens a request: the gated Delta rule of Gated-DeltaNet and
            KDA, and plain decayed linear attention (stepq.prompt).  Lengths of one token are its recurrent form;
* "beam":   beam search's selection over beams and vocabulary, and the reordering of the states that goes with it
            (stepq.beam_select, PackedStatePool.beam_step).

`own` false: the plain form, elementary torch operations.  `own` true: the library's calls.
"""
import math
import random

import torch

own = False

D = 128          # key and value dimension of a state
BLOCK = 64       # tokens of a block of the plan
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
VARIANTS = {"gdn": 0, "kda": 1, "linear": 2}


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # a handful of requests arrive between two decode steps: latency
        dict(name="plan-few", op="plan", requests=8, longest=512, ragged=1, slots=64, assign=False),
        # a large ragged batch, half of it new requests that take free slots of the pool
        dict(name="plan-many", op="plan", requests=8192, longest=160, ragged=2, slots=12288, assign=True),
        # one token a request, states kept unquantised: batch 64, 32 heads, as the mixed-width pool of the benchmark;
        # query and key heads shared by two value heads
        dict(name="gdn-token", op="prompt", variant="gdn", dtype="bf16", requests=64, longest=1, ragged=0, heads=32, heads_qk=16),
        # the same with a gate per key row, batch 128
        dict(name="kda-token", op="prompt", variant="kda", dtype="f32", requests=128, longest=1, ragged=0, heads=32, heads_qk=32),
        # plain linear attention, one token a request, batch 256
        dict(name="linear-token", op="prompt", variant="linear", dtype="f16", requests=256, longest=1, ragged=0, heads=32, heads_qk=32),
        # four short turns, batch 4 and 16 heads: the smallest prompts, latency again
        dict(name="gdn-short", op="prompt", variant="gdn", dtype="bf16", requests=4, longest=61, ragged=3, heads=16, heads_qk=16),
        # one long document: the only parallel work is over heads, columns and the blocks' own products
        dict(name="gdn-long", op="prompt", variant="gdn", dtype="bf16", requests=1, longest=8192, ragged=0, heads=32, heads_qk=16),
        # a batch of chat prompts, ragged, in the framework's fp32
        dict(name="gdn-ragged", op="prompt", variant="gdn", dtype="f32", requests=16, longest=1023, ragged=5, heads=32, heads_qk=32),
        # the same with a gate per key row
        dict(name="kda-ragged", op="prompt", variant="kda", dtype="bf16", requests=16, longest=1023, ragged=6, heads=32, heads_qk=32),
        # two long prompts without the Delta correction
        dict(name="linear-long", op="prompt", variant="linear", dtype="f16", requests=2, longest=4001, ragged=7, heads=32, heads_qk=32),
        # selection alone, twice as many candidates as beams (a search that sets finished beams aside), odd vocabulary
        dict(name="beam-select", op="beam", groups=1, beams=4, out=8, vocab=32001, dtype="f32", masked=True, heads=0, bits=0),
        # selection and reordering of a 4-bit pool of 512 states of 48 heads, as the benchmark's largest
        dict(name="beam-step", op="beam", groups=64, beams=8, out=8, vocab=100003, dtype="bf16", masked=False, heads=48, bits=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "prompt", "prompt", "prompt", "beam", "beam"])
    ragged = rng.randrange(1, 1 << 20)
    if op == "plan":
        requests, longest = _log(rng, 1, 8192), _log(rng, 1, 4096)
        while requests * longest > 1 << 20:
            longest = max(1, longest // 2)
        assign = rng.random() < 0.5
        return dict(op="plan", requests=requests, longest=longest, ragged=ragged, slots=requests + rng.randrange(1, requests + 64),
                    assign=assign)
    if op == "prompt":
        variant, dtype = rng.choice(sorted(VARIANTS)), rng.choice(sorted(DTYPES))
        heads_qk = rng.choice([1, 2, 3, 4, 8, 16])
        heads = heads_qk * rng.choice([1, 2, 3]) if heads_qk < 16 else heads_qk * rng.choice([1, 2])
        if rng.random() < 0.3:
            requests, longest, ragged = _log(rng, 1, 256), 1, 0
        else:
            requests, longest = _log(rng, 1, 24), _log(rng, 2, 4096)
            while requests * longest * heads > 400000 or longest * requests > 16384:
                longest = max(2, longest // 2)
        return dict(op="prompt", variant=variant, dtype=dtype, requests=requests, longest=longest, ragged=ragged, heads=heads,
                    heads_qk=heads_qk)
    beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
    groups = _log(rng, 1, 512 // beams)
    vocab = _log(rng, 64, 131072)
    while groups * beams * vocab > 48_000_000:
        vocab //= 2
    pool = rng.random() < 0.5
    return dict(op="beam", groups=groups, beams=beams, out=beams if pool else rng.randrange(1, 2 * beams + 1), vocab=vocab,
                dtype=rng.choice(sorted(DTYPES)), masked=rng.random() < 0.5, heads=rng.choice([1, 4, 16, 32]) if pool else 0,
                bits=rng.choice([2, 4, 6, 8]) if pool else 0)


def _lengths(case):
    """The lengths of the requests: all `longest`, or spread by their logarithm, an empty request among them."""
    if not case["ragged"]:
        return [case["longest"]] * case["requests"]
    rng = random.Random(case["ragged"])
    got = [_log(rng, 1, case["longest"]) if rng.random() < 0.5 else rng.randrange(0, case["longest"] + 1) for _ in range(case["requests"])]
    got[-1] = case["longest"]
    return got


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"plan": _prepare_plan, "prompt": _prepare_prompt, "beam": _prepare_beam}[case["op"]](case, seed, g)


def _prepare_plan(case, seed, g):
    rng = random.Random(seed)
    lengths = _lengths(case)
    rng.shuffle(lengths)
    tokens = sum(lengths) + 37  # rows of the padded batch that no request fills
    contexts = [0 if rng.random() < 0.5 else rng.randrange(1, 5000) for _ in lengths]
    s = {"op": "plan", "tokens": tokens, "n_slots": case["slots"]}
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    s["contexts"] = torch.tensor(contexts, dtype=torch.int32, device="cuda")
    perm = rng.sample(range(case["slots"]), case["requests"])
    # a continuing request keeps its slot; with `assign` a new one gets the lowest free slot
    slots = [p if c or not case["assign"] else -1 for p, c in zip(perm, contexts)]
    busy = [0] * case["slots"]
    for p in slots:
        if p >= 0:
            busy[p] = 1
    s["slots"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
    s["busy"] = torch.tensor(busy, dtype=torch.uint8, device="cuda")
    if own:
        from quantized_recurrent_state_sm_b200 import stepq
        s["plan"] = stepq.RequestPlan(case["requests"], tokens, case["slots"])
    return s


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _prepare_prompt(case, seed, g):
    H, Hk, R, dt = case["heads"], case["heads_qk"], case["requests"], DTYPES[case["dtype"]]
    lengths = _lengths(case)
    T = sum(lengths)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    s = {"op": "prompt", "variant": case["variant"], "lengths": lengths}
    s["q"], s["k"] = _unit(normal(T, Hk, D)).to(dt), _unit(normal(T, Hk, D)).to(dt)
    s["v"] = normal(T, H, D).to(dt)
    s["beta"] = torch.sigmoid(normal(T, H))
    # half-lives log-uniform in [1, 4096] tokens for each head (or key row), moved a little from token to token
    gate = (1, H, D) if case["variant"] == "kda" else (1, H)
    half = 12 * torch.rand(gate, device="cuda", generator=g)
    s["alpha"] = torch.exp2(-torch.exp2(-(half + 0.5 * normal(T, *gate[1:])).clamp(min=0)))
    fresh = torch.rand(R, device="cuda", generator=g) < 0.5
    if case["longest"] == 1:
        fresh[:] = False  # a single token continues its request
    s["contexts"] = torch.where(fresh, 0, 1000).to(torch.int32)
    s["S"] = 0.2 * normal(R, H, D, D)
    dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if own:
        from quantized_recurrent_state_sm_b200 import stepq
        s["plan"] = stepq.RequestPlan(R, T, R)  # one plan serves every layer of a model
        s["plan"].build(dev, contexts=s["contexts"], max_length=case["longest"])
    else:
        # the plain form's plan: where each request's tokens lie in a padded [R, L] batch
        L = max(max(lengths), 1)
        C = _chunk(case["variant"], L)
        L = -(-L // C) * C
        at = torch.arange(L, device="cuda").expand(R, L)
        s["there"] = at < dev[:, None]
        s["row"] = torch.where(s["there"], (dev.cumsum(0) - dev)[:, None] + at, T)
        s["back"] = torch.nonzero(s["there"].flatten()).flatten()  # and where each token of the batch lies there
    return s


def _prepare_beam(case, seed, g):
    G, B, V, dt = case["groups"], case["beams"], case["vocab"], DTYPES[case["dtype"]]
    s = {"op": "beam", "n": case["out"]}
    logits = 2.5 * torch.randn((G, B, V), device="cuda", generator=g)
    scores = -20 * torch.rand((G, B), device="cuda", generator=g)
    if case["masked"]:
        # constrained decoding bars most of the vocabulary; some beams are dead, some rows bar every token
        logits.masked_fill_(torch.rand((G, B, V), device="cuda", generator=g) < 0.7, -math.inf)
        dead = torch.rand((G, B), device="cuda", generator=g)
        logits.masked_fill_((dead < 0.1)[:, :, None], -math.inf)
        scores.masked_fill_(dead > 0.85, -math.inf)
    s["logits"], s["scores"] = logits.to(dt), scores
    if case["heads"]:
        import numpy as np
        # packed states of one width: two scale vectors and 128 x 128 codes for each head
        words = case["heads"] * (1024 + 2048 * case["bits"]) // 4
        data = torch.randint(-2 ** 31, 2 ** 31, (G * B, words), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
        if own:
            from quantized_recurrent_state_sm_b200 import stepq
            table = np.full((case["heads"], D), case["bits"], np.uint8)
            s["pool"] = stepq.PackedStatePool(stepq.GDN, G * B, case["heads"], table, np.ones((case["heads"], D), np.float32))
            s["states"] = s["pool"].state.view(torch.int32).view(G * B, words)
            s["states"].copy_(data)
        else:
            s["states"] = data
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"plan": _plain_plan, "prompt": _plain_prompt, "beam": _plain_beam}[s["op"]](s)


def _own(s):
    from quantized_recurrent_state_sm_b200 import stepq
    if s["op"] == "plan":
        busy = s["busy"].clone()  # the pool's map of used slots, updated by the call
        p = s["plan"].build(s["lengths"], contexts=s["contexts"], slots=s["slots"], busy=busy)
        return [p.starts, p.slots, p.token_request, p.token_position, p.block_request, p.block_first, busy.to(torch.int32)]
    if s["op"] == "prompt":
        out = stepq.prompt(VARIANTS[s["variant"]], s["plan"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["S"])
        return [out, s["S"]]
    if "pool" in s:
        scores, parents, tokens = s["pool"].beam_step(s["logits"], s["scores"])
        return [scores, parents, tokens, s["states"]]
    return list(stepq.beam_select(s["logits"], s["scores"], s["n"]))


def _plain_plan(s):
    n, T = s["lengths"].long(), s["tokens"]
    R, dev = n.numel(), n.device
    ends = n.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    # tokens: the request that covers each row, and its place in the request's history
    at = torch.arange(T, device=dev)
    request = torch.searchsorted(ends, at, right=True)
    inside = request < R
    safe = request.clamp(max=R - 1)
    position = torch.where(inside, s["contexts"].long()[safe] + at - starts[safe], -1)
    request = torch.where(inside, request, -1)
    # blocks of 64 tokens, request after request
    blocks = ((n + BLOCK - 1) // BLOCK).cumsum(0)
    b = torch.arange(T // BLOCK + R, device=dev)
    of = torch.searchsorted(blocks, b, right=True)
    real = of < R
    of_safe = of.clamp(max=R - 1)
    first = torch.where(real, (b - blocks[of_safe] + (n[of_safe] + BLOCK - 1) // BLOCK) * BLOCK, -1)
    # slots: the k-th new request with tokens gets the k-th free slot
    new = (s["slots"] < 0) & (n > 0)
    free = s["busy"].argsort(stable=True)  # the free slots, lowest first, and then the others
    rank = (new.long().cumsum(0) - 1).clamp(min=0)
    slots = torch.where(new, free[rank], s["slots"].long())
    used = torch.where((slots >= 0) & (n > 0), slots, s["n_slots"])
    busy = torch.cat([s["busy"], s["busy"].new_zeros(1)]).to(torch.int32).index_fill(0, used, 1)[:-1]
    i32 = torch.int32
    return [starts.to(i32), slots.to(i32), request.to(i32), position.to(i32), torch.where(real, of, -1).to(i32), first.to(i32), busy]


def _chunk(variant, longest):
    """Tokens the plain form takes at once; with a gate per key row every pair of tokens has 128 decays."""
    return min(16 if variant == "kda" else 64, 1 << (longest - 1).bit_length())


def _plain_prompt(s):
    """The chunked form.  With the state S before a chunk, the gates' running products c_t, and decay_ts = c_t / c_s:
    u_t = beta_t (v_t - S^T (c_t k_t) - sum_(s<t) (k_t . decay_ts k_s) u_s), o_t = S^T (c_t q_t) + sum_(s<=t)
    (q_t . decay_ts k_s) u_s, and S becomes c_C S + sum_s (decay_Cs k_s) u_s^T; linear: u_t = beta_t v_t."""
    variant, dt = s["variant"], s["q"].dtype
    T, H = s["v"].shape[:2]
    R, L = s["row"].shape
    C = _chunk(variant, L)
    n = L // C
    share = H // s["q"].shape[1]

    def padded(x, fill, heads):  # [T, heads, ...] -> [R, H, n, C, ...]
        x = torch.cat([x.float(), x.new_full((1, *x.shape[1:]), fill).float()])[s["row"]]
        x = x.reshape(R, n, C, *x.shape[2:]).movedim(3, 1)
        return x if heads == H else x.repeat_interleave(share, dim=1)

    q, k = padded(s["q"], 0, H // share), padded(s["k"], 0, H // share)
    v, beta = padded(s["v"], 0, H), padded(s["beta"], 0, H)
    alpha = padded(s["alpha"], 1, H)
    if variant != "kda":
        alpha = alpha[..., None]
    log = alpha.double().log().cumsum(3)  # long sums of logarithms: 64 bits
    low = torch.ones((C, C), dtype=torch.bool, device=q.device).tril()
    eye = torch.eye(C, device=q.device)
    if variant == "kda":
        pair = (log[:, :, :, :, None] - log[:, :, :, None]).masked_fill(~low[..., None], -math.inf).exp().float()
        pair = pair * k[:, :, :, None]
        P = (pair * q[:, :, :, :, None]).sum(-1)
        A = (pair * k[:, :, :, :, None]).sum(-1)
        del pair
    else:
        decay = (log - log.transpose(3, 4)).masked_fill(~low, -math.inf).exp().float()
        P = q @ k.transpose(3, 4) * decay
        A = k @ k.transpose(3, 4) * decay
    until = log.exp().float()
    after = (log[:, :, :, -1:] - log).exp().float()
    kin, qin, kout, keep = k * until, q * until, k * after, until[:, :, :, -1]
    if variant != "linear":
        A = beta[..., None] * A * (1 - eye)
        solve = eye.expand(A.shape).clone()
        for t in range(1, C):  # (I + A) solve = I, row after row
            solve[..., t, :t] -= (A[..., t, None, :t] @ solve[..., :t, :t])[..., 0, :]
    S = torch.where((s["contexts"] == 0)[:, None, None, None], 0, s["S"])
    out = []
    for c in range(n):
        u = beta[:, :, c, :, None] * v[:, :, c] if variant == "linear" else solve[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - kin[:, :, c] @ S))
        out.append(qin[:, :, c] @ S + P[:, :, c] @ u)
        S = keep[:, :, c].unsqueeze(-1) * S + kout[:, :, c].transpose(2, 3) @ u
    # a request without tokens keeps its state
    some = s["there"][:, 0, None, None, None]
    s["S"] = torch.where(some, S, s["S"])
    o = torch.stack(out, 2).reshape(R, H, L, D).movedim(2, 1).reshape(R * L, H, D)[s["back"]]
    return [o.to(dt), s["S"]]


def _plain_beam(s):
    """score = the beam's score + log_softmax(logits), in 64 bits (candidates of two beams lie close); the best n by
    score, then by beam and token.  A candidate of score -inf is none: parent and token -1."""
    G, B, V = s["logits"].shape
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    scores = s["scores"].double()[..., None] + (x - top - (x - top).exp().sum(-1, keepdim=True).log())
    scores = torch.where(x == -math.inf, -math.inf, scores).reshape(G, B * V)
    # the largest n, ties to the lowest index
    n = s["n"]
    if B * V < n:
        scores = torch.cat([scores, scores.new_full((G, n - B * V), -math.inf)], 1)
    best, at = scores.sort(dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    none = best == -math.inf
    parents = torch.where(none, -1, at // V).to(torch.int32)
    tokens = torch.where(none, -1, at % V).to(torch.int32)
    got = [best.float(), parents, tokens]
    if "states" in s:
        # the state of beam i becomes that of its parent; a beam without one keeps its own
        own_row = torch.arange(B, device=x.device)
        src = torch.where(none, own_row, parents.long()) + B * torch.arange(G, device=x.device)[:, None]
        s["states"] = s["states"][src.flatten()]
        got.append(s["states"])
    return got


# ---- the work and the exact values ---------------------------------------------

def work(case):
    if case["op"] == "plan":
        n = _lengths(case)
        T, R = sum(n) + 37, case["requests"]
        return {"bytes": 4 * (6 * R + 2 * T + 2 * (T // BLOCK + R)) + 2 * case["slots"], "flops": 0}
    if case["op"] == "prompt":
        n = _lengths(case)
        T, H, Hk, e = sum(n), case["heads"], case["heads_qk"], DTYPES[case["dtype"]].itemsize
        gate = D if case["variant"] == "kda" else 1
        some = sum(x > 0 for x in n)
        # half of the requests of a prompt start from nothing and read no state
        states = some * H * D * D * 4 * (2 if case["longest"] == 1 else 1.5)
        return {"bytes": T * (2 * Hk * D * e + 2 * H * D * e + 4 * H * (1 + gate)) + states,
                "flops": T * H * D * D * (4 if case["variant"] == "linear" else 6)}
    G, B, V = case["groups"], case["beams"], case["vocab"]
    moved = 0
    if case["heads"]:
        # beams that change their state: about 1 - 1/B of them, read and written
        moved = 2 * G * (B - 1) * case["heads"] * (1024 + 2048 * case["bits"])
    return {"bytes": G * B * V * DTYPES[case["dtype"]].itemsize + 4 * G * B + 12 * G * case["out"] + moved, "flops": 3 * G * B * V}


def exact(case, seed):
    if case["op"] == "plan":
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_prompt(case, s) if case["op"] == "prompt" else _exact_beam(case, s)


def _exact_prompt(case, s):
    """The recurrence token by token in 64 bits."""
    T, H = s["v"].shape[:2]
    share = H // case["heads_qk"]
    n = torch.tensor(s["lengths"], device="cuda")
    starts = n.cumsum(0) - n
    S = s["S"].double()
    S[s["contexts"] == 0] = 0
    S = torch.where((n == 0)[:, None, None, None], s["S"].double(), S)
    out = torch.zeros((T, H, D), dtype=torch.float64, device="cuda")
    order = sorted(range(len(s["lengths"])), key=lambda r: -s["lengths"][r])
    back = torch.tensor(order, device="cuda")
    S, starts = S[back], starts[back]
    lengths = sorted(s["lengths"], reverse=True)
    live = len(lengths)
    for t in range(lengths[0]):
        while lengths[live - 1] <= t:
            live -= 1
        i = starts[:live] + t
        q, k = (s[x][i].double().repeat_interleave(share, 1) for x in "qk")
        v, a, b = (s[x][i].double() for x in ("v", "alpha", "beta"))
        M = S[:live]
        M.mul_(a[..., None] if a.dim() == 3 else a[..., None, None])
        if case["variant"] != "linear":
            v = v - torch.einsum("rhkv,rhk->rhv", M, k)
        M.add_(k[..., :, None] * (b[..., None] * v)[..., None, :])
        out[i] = torch.einsum("rhkv,rhk->rhv", M, q)
    final = torch.empty_like(S)
    final[back] = S
    return [out, final]


def _exact_beam(case, s):
    G, B, V = s["logits"].shape
    got = []
    for g in range(G):  # a group at a time, from the candidates of each beam
        x = s["logits"][g].double()
        all_ = s["scores"][g].double()[:, None] + torch.log_softmax(x, -1).nan_to_num(nan=-math.inf, neginf=-math.inf)
        best = torch.topk(all_.flatten(), min(case["out"], B * V)).values
        got.append(torch.cat([best, best.new_full((case["out"] - best.numel(),), -math.inf)]))
    return [torch.stack(got), None, None, None][:4 if case["heads"] else 3]
