"""Plans, prompts, packing by request, beam selection and reordering against plain implementations."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from quantized_recurrent_state_sm_b200 import workload as W

from . import serving_reference as ref

GDN, KDA, LINEAR = 0, 1, 2


@pytest.fixture(scope="module")
def S():
    from quantized_recurrent_state_sm_b200 import build
    build.build()
    from quantized_recurrent_state_sm_b200 import stepq
    return stepq


@pytest.fixture(scope="module")
def G(S):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return S


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- refusals, on the host -----------------------------------------------------

def refused(S, status, fragment):
    assert status == S.ERR_INVALID_ARG or status == S.ERR_UNSUPPORTED, status
    assert fragment in S.lib.stepq_last_error().decode()


@pytest.mark.parametrize("bad,fragment", [((-1, 8, 8), "requests"), ((65537, 8, 8), "requests"), ((1, -1, 8), "tokens"),
                                          ((1, (1 << 28) + 1, 8), "tokens"), ((1, 8, -1), "slots"), ((1, 8, (1 << 24) + 1), "slots")])
def test_plan_descriptor_refusals(S, bad, fragment):
    d = S.PlanDesc(*bad)
    assert S.lib.stepq_plan_bytes(C.byref(d)) == 0
    r = S.PlanRegions()
    refused(S, S.lib.stepq_plan_layout(C.byref(d), C.byref(r)), fragment)


def test_plan_layout(S):
    d, r = S.PlanDesc(5, 130, 9), S.PlanRegions()
    assert S.lib.stepq_plan_layout(C.byref(d), C.byref(r)) == 0
    assert r.blocks == 130 // 64 + 5 and S.lib.stepq_plan_bytes(C.byref(d)) == r.total
    order = [(r.head, 16), (r.starts, 24), (r.slot, 20), (r.live, 20), (r.fresh, 20), (r.token_request, 520),
             (r.token_position, 520), (r.block_starts, 24), (r.block_request, 4 * r.blocks), (r.block_first, 4 * r.blocks), (r.scratch, 4 * 14)]
    end = 0
    for at, n in order:
        assert at >= end and at % 16 == 0
        end = at + n
    assert end <= r.total


def test_plan_build_refusals(S):
    d = S.PlanDesc(2, 16, 2)
    n = S.lib.stepq_plan_bytes(C.byref(d))
    build = S.lib.stepq_plan_build
    refused(S, build(C.byref(d), None, n, 1, None, None, None, None, 16, None), "plan is NULL")
    refused(S, build(C.byref(d), None, n - 1, 1, None, None, None, None, 16, None), "required")
    refused(S, build(C.byref(d), None, n, 3, None, None, None, None, 16, None), "the plan holds")
    refused(S, build(C.byref(d), None, n, -1, None, None, None, None, 16, None), "the plan holds")
    refused(S, build(C.byref(d), None, n, 1, None, None, None, None, -1, None), "max_length")
    refused(S, build(None, None, n, 1, None, None, None, None, 1, None), "descriptor")


@pytest.mark.parametrize("change,fragment", [
    (dict(variant=3), "variant"), (dict(variant=-1), "variant"), (dict(dtype=3), "dtype"), (dict(heads=0), "heads"),
    (dict(heads=65536, heads_qk=1), "heads"), (dict(heads_qk=0), "heads_qk"), (dict(heads_qk=3), "heads_qk"),
    (dict(dk=64), "128"), (dict(dv=0), "positive"), (dict(max_length=-1), "max_length"), (dict(stride_q=255), "stride"),
    (dict(stride_k=128), "stride"), (dict(stride_v=511), "stride"), (dict(stride_q=258), "16 bytes"), (dict(stride_v=1 << 41), "stride")])
def test_prompt_descriptor_refusals(S, change, fragment):
    pd = S.PlanDesc(3, 40, 3)
    d = S.PromptDesc(0, 0, 4, 2, 128, 128, 40, 0, 256, 256, 512)
    assert S.lib.stepq_prompt_scratch_bytes(C.byref(pd), C.byref(d)) != C.c_size_t(-1).value
    for f, x in change.items():
        setattr(d, f, x)
    assert S.lib.stepq_prompt_scratch_bytes(C.byref(pd), C.byref(d)) == C.c_size_t(-1).value
    refused(S, S.lib.stepq_prompt(C.byref(pd), None, 1 << 20, C.byref(d), *[None] * 8, 0, None), fragment)


def test_prompt_item_limit(S):
    pd = S.PlanDesc(65536, 40, 3)
    d = S.PromptDesc(0, 0, 257, 1, 128, 128, 40, 0, 128, 128, 257 * 128)
    refused(S, S.lib.stepq_prompt(C.byref(pd), None, 1 << 20, C.byref(d), *[None] * 8, 0, None), "requests * heads")


@pytest.mark.parametrize("args,fragment", [((-1, 2, 9, 1), "groups"), ((1, 0, 9, 1), "beams"), ((1, 65, 9, 1), "beams"),
                                           ((1, 2, 0, 1), "vocab"), ((1, 2, (1 << 30) + 1, 1), "vocab"), ((1, 2, 9, 0), "n 0"),
                                           ((1, 2, 9, 65), "n 65"), ((1 << 24, 2, 9, 1), "groups * beams")])
def test_beam_refusals(S, args, fragment):
    assert S.lib.stepq_beam_scratch_bytes(*args) == 0
    refused(S, S.lib.stepq_beam_select(*args, 0, None, 1 << 31, None, None, None, None, None, 0, None), fragment)


def test_beam_other_refusals(S):
    refused(S, S.lib.stepq_beam_select(1, 2, 9, 1, 3, None, 9, None, None, None, None, None, 0, None), "dtype")
    refused(S, S.lib.stepq_beam_select(1, 2, 9, 1, 0, None, 8, None, None, None, None, None, 0, None), "stride")
    refused(S, S.lib.stepq_beam_select(1, 2, 9, 1, 0, None, 9, None, None, None, None, None, 0, None), "logits is NULL")
    refused(S, S.lib.stepq_reorder_rows(None, 24, 1, 2, None, None), "multiple of 16")
    refused(S, S.lib.stepq_reorder_rows(None, 32, 1, 65, None, None), "beams")
    refused(S, S.lib.stepq_reorder_rows(None, 32, 1, 2, None, None), "base is NULL")
    assert S.lib.stepq_reorder_rows(None, 32, 0, 2, None, None) == 0
    assert S.lib.stepq_pool_reorder(None, 0, 1, 1, None) == S.ERR_INVALID_ARG
    assert S.lib.stepq_pack_requests(None, None, None, 0, None, 0) == S.ERR_INVALID_ARG


def test_host_tensors_are_refused(S):
    x = torch.zeros((1, 2, 9))
    with pytest.raises(TypeError):
        S.beam_select(x, torch.zeros((1, 2)))
    with pytest.raises(TypeError):
        S.reorder_rows(x, torch.zeros((1, 1), dtype=torch.int32))


# ---- plans ---------------------------------------------------------------------

def check_plan(S, requests, tokens, n_slots, lengths, contexts=None, slots=None, busy=None, max_length=None, plan=None):
    want = ref.plan(requests, tokens, n_slots, lengths, contexts, slots, busy, max_length)
    p = plan or S.RequestPlan(requests, tokens, n_slots)
    p.buffer.fill_(0xA5)
    b = None if busy is None else torch.tensor(busy, dtype=torch.uint8, device="cuda")
    p.build(i32(lengths), None if contexts is None else i32(contexts), None if slots is None else i32(slots), b, max_length)
    for f in ("starts", "block_starts", "slots", "live", "fresh", "token_request", "token_position", "block_request", "block_first", "head"):
        assert getattr(p, f).tolist() == want[f], f
    if busy is not None:
        assert b.tolist() == want["busy"]
    if want["head"][0]:
        with pytest.raises(S.StepqError):
            p.check()
    else:
        p.check()
    return p


def spread(rng, n, most):
    return [int(x) for x in np.where(rng.random(n) < 0.2, 0, rng.integers(0, most + 1, n))]


@pytest.mark.gpu
@pytest.mark.parametrize("n,most", [(0, 5), (1, 0), (1, 1), (1, 64), (1, 65), (1, 5000), (2, 2048), (7, 4096), (511, 40), (513, 7),
                                    (4099, 3), (20000, 130)])
def test_plan_token_and_block_tables(G, n, most):
    rng = np.random.default_rng(n * 7 + most)
    lengths = spread(rng, n, most) if n != 1 else [most]
    contexts = [int(x) for x in np.where(rng.random(n) < 0.5, 0, rng.integers(0, 100000, n))]
    check_plan(G, n, sum(lengths), n, lengths)
    check_plan(G, n + 3, sum(lengths) + 77, n + 5, lengths, contexts)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 5, 600, 3001])
@pytest.mark.parametrize("full", [False, True])
def test_plan_slots(G, n, full):
    """Half of the requests bring a slot, the others take free ones; `full` leaves too few."""
    rng = np.random.default_rng(n + full)
    slots_n = n + 40 if not full else n
    lengths = spread(rng, n, 9)
    contexts = [int(x) for x in np.where(rng.random(n) < 0.5, 0, 12)]
    perm = rng.permutation(slots_n)
    slots = [int(perm[r]) if contexts[r] else -1 for r in range(n)]
    busy = [0] * slots_n
    for s in slots:
        if s >= 0:
            busy[s] = 1
    if full:
        for s in range(slots_n):
            busy[s] |= int(rng.random() < 0.7)
    check_plan(G, n, sum(lengths) + 5, slots_n, lengths, contexts, slots, busy)


@pytest.mark.gpu
def test_plan_refusals_of_requests(G):
    # twice the same slot: the first request with tokens has it; a slot out of range; a continuing request without one
    check_plan(G, 6, 40, 4, [0, 5, 5, 5, 5, 5], [1] * 6, [2, 2, 2, 9, -1, 0])
    check_plan(G, 6, 40, 4, [0, 5, 5, 5, 5, 5], [1, 0, 1, 0, 1, 0], [2, 2, 2, -7, -1, -1], [0, 0, 0, 0])
    # a new request may not land in a slot that another names without its being marked as used
    check_plan(G, 3, 40, 2, [4, 4, 4], [0, 9, 0], [-1, 0, -1], [0, 0])
    # negative lengths, lengths above the bound, more tokens than rows
    check_plan(G, 4, 40, 4, [3, -2, 9, 4], None, None, None, 8)
    check_plan(G, 5, 10, 5, [3, 4, 9, 0, 1])
    check_plan(G, 3, 10, 3, [2 ** 31 - 1, 1, 1])
    check_plan(G, 4, 10, 4, [10, 0, 2 ** 31 - 1, 2 ** 31 - 1])
    # more requests than slots
    check_plan(G, 3, 10, 2, [1, 1, 1])
    with pytest.raises(G.StepqError):
        G.RequestPlan(2, 8).build(i32([1, 2, 3]))
    with pytest.raises(G.StepqError):
        G.RequestPlan(2, 8).build(i32([1, 2]), busy=torch.zeros(2, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        G.RequestPlan(2, 8).build(torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError):
        G.RequestPlan(2, 8).build(i32([1, 2]), i32([1]))


@pytest.mark.gpu
def test_plan_rebuilt_in_place_and_replayed(G):
    p = G.RequestPlan(4, 300, 4)
    check_plan(G, 4, 300, 4, [100, 64, 0, 5], plan=p)
    check_plan(G, 4, 300, 4, [1, 299], plan=p)
    lengths = i32([7, 7, 7, 7])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        p.build(lengths)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        p.build(lengths)
    lengths.copy_(i32([0, 130, 2, 0]))
    g.replay()
    want = ref.plan(4, 300, 4, [0, 130, 2, 0])
    assert p.token_position.tolist() == want["token_position"] and p.block_first.tolist() == want["block_first"]


# ---- prompts -------------------------------------------------------------------

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def tolerance(longest, dtype):
    """Relative 2-norm.  A token's fp32 arithmetic leaves at most about 32 half-steps 2^-24 of the state's size (the gate,
    sums over 128 terms, products split to 22 bits, the update), tokens add like independent errors; the output is rounded
    once more to its type, by at most half a step."""
    return 32 * 2.0 ** -24 * (1 + math.sqrt(longest)) + (torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0)


def prompt_inputs(variant, dtype, lengths, H, Hk, seed, pad=0, rows=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lengths) + pad

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    q, k = (torch.nn.functional.normalize(normal(T, Hk, 128), dim=-1).to(dtype) for _ in range(2))
    v = normal(T, H, 128).to(dtype)
    gate = (T, H, 128) if variant == KDA else (T, H)
    alpha = torch.exp2(-torch.exp2(-12 * torch.rand(gate, device="cuda", generator=g)))
    beta = torch.sigmoid(normal(T, H))
    St = 0.2 * normal(rows or len(lengths), H, 128, 128)
    return q, k, v, alpha, beta, St


def rel(x, y):
    y = y.double()
    n = y.norm()
    return float((x.double() - y).norm() / n) if n > 0 else float((x.double() - y).norm())


def run_prompt(S, variant, dtype, lengths, H, Hk, contexts=None, seed=0, max_length=None, change=None):
    q, k, v, alpha, beta, St = prompt_inputs(variant, dtype, lengths, H, Hk, seed)
    if change:
        q, k, v, alpha, beta, St = change(q, k, v, alpha, beta, St)
    contexts = contexts or [7] * len(lengths)
    start = St.clone()
    for r, c in enumerate(contexts):
        if c == 0:
            start[r] = 0
            if lengths[r] > 0:
                St[r] = float("nan")  # not read
    want_o, want_S = ref.recurrence(variant, lengths, q, k, v, alpha, beta, start)
    for r, n in enumerate(lengths):
        if n == 0:
            want_S[r] = St[r]
    p = S.RequestPlan(len(lengths), sum(lengths))
    p.build(i32(lengths), i32(contexts), max_length=max_length)
    p.check()
    out = S.prompt(variant, p, q, k, v, alpha, beta, St)
    assert out.dtype == dtype
    longest = max(lengths)
    assert torch.isfinite(out).all() and torch.isfinite(St).all()
    assert rel(out, want_o) <= tolerance(longest, dtype), rel(out, want_o)
    assert rel(St, want_S) <= tolerance(longest, torch.float32), rel(St, want_S)
    # no single token or request far off either
    for r in range(len(lengths)):
        assert rel(St[r], want_S[r]) <= 4 * tolerance(longest, torch.float32)
    off = (out.double() - want_o).norm(dim=-1).max()
    assert float(off) <= 4 * tolerance(longest, dtype) * float(want_o.norm(dim=-1).max())


@pytest.mark.gpu
@pytest.mark.parametrize("variant", [GDN, KDA, LINEAR])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths,H,Hk", [([1], 1, 1), ([1, 1, 1], 4, 2), ([3, 0, 8, 1], 3, 1), ([5], 6, 6)])
def test_prompt_of_few_tokens(G, variant, dtype, lengths, H, Hk):
    contexts = [0 if r % 3 == 1 else 7 for r in range(len(lengths))]
    run_prompt(G, variant, DT[dtype], lengths, H, Hk, contexts, seed=len(lengths), max_length=8)


@pytest.mark.gpu
@pytest.mark.parametrize("variant", [GDN, KDA, LINEAR])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths,H,Hk", [([64], 1, 1), ([63], 2, 1), ([65], 2, 2), ([1], 3, 1), ([17, 1, 0, 64, 129, 3], 4, 2),
                                          ([200, 0, 40], 6, 2), ([128, 192], 1, 1)])
def test_prompt_in_blocks(G, variant, dtype, lengths, H, Hk):
    contexts = [0 if r % 2 else 7 for r in range(len(lengths))]
    run_prompt(G, variant, DT[dtype], lengths, H, Hk, contexts, seed=sum(lengths))


@pytest.mark.gpu
@pytest.mark.parametrize("variant,dtype", [(GDN, "bf16"), (GDN, "f32"), (KDA, "f16"), (LINEAR, "f32")])
def test_prompt_long(G, variant, dtype):
    run_prompt(G, variant, DT[dtype], [1500], 2, 1, [0], seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["half", "near-half", "one-drop", "first", "last"])
def test_prompt_gates_at_the_border(G, dtype, kind):
    """16 tokens whose gates' product lies at 2^-16, evenly or in one step, with rows of k at the largest mantissa."""
    def change(q, k, v, alpha, beta, St):
        t = torch.arange(len(alpha), device="cuda").reshape(-1, 1, 1) % 16
        one = torch.ones_like(alpha)
        if kind == "half":
            alpha = 0.5 * one
        elif kind == "near-half":
            alpha = 0.5 + 0.02 * (alpha - 0.75)
        elif kind == "one-drop":
            at = torch.arange(alpha.shape[2], device="cuda") % 16
            alpha = torch.where(t == at, 2.0 ** -16, one)
        else:
            alpha = torch.where(t == (1 if kind == "first" else 15), 2.0 ** -16, one)
        k = torch.where(k.float() < 0, -0.1249, 0.1249).to(k.dtype)  # just below 2^-3: rows of norm sqrt 2
        return q, k, v, alpha, 0.5 * beta, St

    run_prompt(G, KDA, DT[dtype], [70, 64, 17], 2, 1, [7, 0, 7], seed=19, change=change)


@pytest.mark.gpu
@pytest.mark.parametrize("variant", [GDN, KDA, LINEAR])
@pytest.mark.parametrize("max_length", [8, None])
@pytest.mark.parametrize("kind", ["open", "quick", "quicker", "shut", "tiny", "mixed", "nobeta", "onebeta", "zero", "small", "large"])
def test_prompt_extreme_gates_and_scales(G, variant, max_length, kind):
    def change(q, k, v, alpha, beta, St):
        if kind == "open":
            alpha = torch.ones_like(alpha)
        elif kind in ("quick", "quicker"):  # about where eight gates' product passes 2^-12
            alpha = 0.2 * (alpha - 0.75) + (0.42 if kind == "quick" else 0.355)
        elif kind == "shut":  # a gate of 0 forgets everything
            alpha = torch.where(torch.arange(len(alpha), device="cuda").reshape(-1, *[1] * (alpha.dim() - 1)) % 3 == 1, 0.0, alpha)
        elif kind == "tiny":
            alpha = alpha * 1e-30
        elif kind == "mixed":
            alpha = torch.where(torch.rand(alpha.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) < 0.3, 1e-20, 1.0)
        elif kind == "nobeta":
            beta = torch.zeros_like(beta)
        elif kind == "onebeta":
            beta = torch.ones_like(beta)
        elif kind == "zero":
            k, q = k * 0, q * 0
        elif kind == "small":
            v, St = v * 2.0 ** -60, St * 2.0 ** -60
        elif kind == "large":
            v, St = v * 2.0 ** 60, St * 2.0 ** 60
        return q, k, v, alpha, beta, St

    run_prompt(G, variant, torch.float32, [8, 5, 1] if max_length else [70, 9, 1], 2, 1, [7, 0, 7], seed=9, max_length=max_length,
               change=change)


@pytest.mark.gpu
@pytest.mark.parametrize("variant", [GDN, KDA, LINEAR])
@pytest.mark.parametrize("lengths,max_length", [([3, 1, 4, 2], 4), ([70, 1, 130, 5], None)])
def test_prompt_leaves_what_is_not_its_own(G, variant, lengths, max_length):
    """Padding rows, requests without tokens, refused requests and their states: neither read (NaN inputs) nor written; token
    strides; states by slot."""
    H, Hk, slots_n = 4, 2, 9
    all_lengths = lengths + [0, 6]
    slots = [5, 2, 7, 0, 3, 2]  # the last request names a slot twice: refused
    T = sum(all_lengths) + 11
    q, k, v, alpha, beta, St = prompt_inputs(variant, torch.bfloat16, all_lengths, H, Hk, 3, pad=11, rows=slots_n)
    used = sum(lengths)
    wide = torch.full((T, (2 * Hk + H) * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    for x, at, n in ((q, 0, Hk), (k, Hk * 128, Hk), (v, 2 * Hk * 128, H)):
        wide[:used, at:at + n * 128] = x[:used].reshape(used, -1)
    qs, ks, vs = (wide[:, at:at + n * 128].unflatten(1, (n, 128)) for at, n in ((0, Hk), (Hk * 128, Hk), (2 * Hk * 128, H)))
    alpha[used:] = float("nan")
    beta[used:] = float("nan")
    others = [s for s in range(slots_n) if s not in slots[:len(lengths)]]
    St[others] = float("nan")
    before = St.clone()
    order = slots[:len(lengths)]
    want_o, want_S = ref.recurrence(variant, lengths, q[:used], k[:used], v[:used], alpha[:used], beta[:used], St[order])
    p = G.RequestPlan(len(all_lengths) + 2, T, slots_n)
    p.build(i32(all_lengths), i32([4] * 6), i32(slots), max_length=max_length)
    out = torch.full((T, H, 128), -3.0, dtype=torch.bfloat16, device="cuda")
    got = G.prompt(variant, p, qs, ks, vs, alpha, beta, St, out, by_slot=True)
    assert got is out
    assert rel(out[:used], want_o) <= tolerance(max(lengths), torch.bfloat16)
    assert rel(St[order], want_S) <= tolerance(max(lengths), torch.float32)
    assert bool((out[used:] == -3.0).all())
    assert torch.equal(St[others].view(torch.int32), before[others].view(torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,max_length", [([2, 8], 8), ([100, 70], None)])
def test_prompt_is_deterministic_across_streams_and_graphs(G, lengths, max_length):
    H = 3
    q, k, v, alpha, beta, S0 = prompt_inputs(GDN, torch.float16, lengths, H, H, 11)
    p = G.RequestPlan(2, sum(lengths)).build(i32(lengths), i32([1, 1]), max_length=max_length)
    St = S0.clone()
    first = G.prompt(GDN, p, q, k, v, alpha, beta, St)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two, S2 = [], [S0.clone(), S0.clone()]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        two.append(G.prompt(GDN, p, q, k, v, alpha, beta, S2[0]))
    two.append(G.prompt(GDN, p, q, k, v, alpha, beta, S2[1]))  # two calls at once, one plan
    torch.cuda.synchronize()
    for o, x in zip(two, S2):
        assert torch.equal(o, first) and torch.equal(x, St)
    Sg, out = S0.clone(), torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.prompt(GDN, p, q, k, v, alpha, beta, Sg, out)
    Sg.copy_(S0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(Sg, St)


@pytest.mark.gpu
@pytest.mark.parametrize("variant", [GDN, KDA, LINEAR])
def test_prompt_split_in_two_continues(G, variant):
    """A prompt in one pass, and in two passes that hand the state on."""
    lengths, cut = [150, 90], [64, 37]
    H = 2
    q, k, v, alpha, beta, S0 = prompt_inputs(variant, torch.float32, lengths, H, 1, 21)
    want_o, want_S = ref.recurrence(variant, lengths, q, k, v, alpha, beta, 0 * S0)
    St = S0
    starts = [0, 150]
    rows = [torch.cat([torch.arange(s, s + c) for s, c in zip(starts, cut)]),
            torch.cat([torch.arange(s + c, s + n) for s, c, n in zip(starts, cut, lengths)])]
    for i, at in enumerate(rows):
        at = at.cuda()
        n = cut if i == 0 else [x - c for x, c in zip(lengths, cut)]
        p = G.RequestPlan(2, len(at)).build(i32(n), i32([0, 0] if i == 0 else cut))
        out = G.prompt(variant, p, *(x[at].contiguous() for x in (q, k, v, alpha, beta)), St)
        assert rel(out, want_o[at]) <= tolerance(150, torch.float32)
    assert rel(St, want_S) <= tolerance(150, torch.float32)


@pytest.mark.gpu
def test_prompt_refusals(G):
    q, k, v, alpha, beta, St = prompt_inputs(GDN, torch.float32, [5], 2, 2, 1)
    p = G.RequestPlan(1, 5).build(i32([5]))
    out = torch.empty_like(v)
    with pytest.raises(TypeError):
        G.prompt(GDN, p, q.double(), k, v, alpha, beta, St)
    with pytest.raises(TypeError):
        G.prompt(GDN, p, q, k.half(), v, alpha, beta, St)
    with pytest.raises(ValueError):
        G.prompt(GDN, p, q[:4], k, v, alpha, beta, St)
    with pytest.raises(ValueError):
        G.prompt(KDA, p, q, k, v, alpha, beta, St)
    with pytest.raises(ValueError):
        G.prompt(GDN, p, q.transpose(0, 1).contiguous().transpose(0, 1), k, v, alpha, beta, St)
    with pytest.raises(ValueError):
        G.prompt(GDN, p, q, k, v, alpha, beta, St, by_slot=True, out=out[:, :1])
    for aliased in (q, v):
        with pytest.raises(G.StepqError, match="overlaps"):
            G.prompt(GDN, p, q, k, v, alpha, beta, St, out=aliased)
    with pytest.raises(G.StepqError):
        G.prompt(7, p, q, k, v, alpha, beta, St)


# ---- packing by request ----------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("ci", [1, 2])
@pytest.mark.parametrize("by_slot", [False, True])
def test_pack_requests_matches_pack(G, ci, by_slot):
    cfg = W.with_overrides(W.CONFIGS[ci], batch=6, heads=6)
    bits, rho = W.bit_table(cfg), W.rho(cfg)
    part, full = (G.PackedStatePool(cfg.variant, 6, 6, bits, rho, cfg.ls_iters) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(ci)
    states = 0.2 * torch.randn((6, 6, 128, 128), device="cuda", generator=g)
    full.pack(states)
    part.state.fill_(0x5C)
    slots, lengths = [4, 1, 0, 5], [3, 0, 7, 2]
    p = G.RequestPlan(5, 12, 6).build(i32(lengths), None, i32(slots))
    part.pack_requests(p, states if by_slot else torch.cat([states[slots], states[:1]]), by_slot)
    torch.cuda.synchronize()
    part.check_guards()
    a, b = part.state.view(6, -1), full.state.view(6, -1)
    for s in range(6):
        if s in (4, 0, 5):
            assert torch.equal(a[s], b[s])
        else:
            assert bool((a[s] == 0x5C).all())


@pytest.mark.gpu
def test_pack_requests_refusals(G):
    pool = G.PackedStatePool(GDN, 3, 2, np.full((2, 128), 6), np.ones((2, 128)))
    p = G.RequestPlan(2, 4, 5).build(i32([1, 1]))
    with pytest.raises(G.StepqError, match="slots"):
        pool.pack_requests(p, torch.zeros((2, 2, 128, 128), device="cuda"))
    p = G.RequestPlan(2, 4, 3).build(i32([1, 1]))
    with pytest.raises(ValueError):
        pool.pack_requests(p, torch.zeros((3, 2, 128, 128), device="cuda"))


# ---- beam search ---------------------------------------------------------------

def check_beam(S, logits, scores, n):
    want = ref.beam(logits.cpu(), scores.cpu(), n)
    got = [x.cpu() for x in S.beam_select(logits, scores, n)]
    for g, rows in enumerate(want):
        for i, (score, b, t) in enumerate(rows):
            assert (got[1][g, i].item(), got[2][g, i].item()) == (b, t), (g, i, rows[i], got[0][g, i].item())
            # one rounding to fp32, and a log-sum of fp32 exponentials: a few of their half-steps at most
            have = got[0][g, i].item()
            assert have == score if math.isinf(score) else abs(have - score) <= 2.0 ** -24 * (abs(score) + 8)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("groups,beams,vocab,n", [(1, 1, 1, 1), (1, 1, 5, 8), (3, 2, 7, 4), (2, 4, 1000, 8), (1, 4, 32001, 4), (5, 3, 8191, 6),
                                                  (2, 16, 8193, 16), (1, 64, 300, 64), (2, 7, 100003, 14), (1, 64, 70001, 64), (70, 8, 20001, 8)])
def test_beam_select(G, dtype, groups, beams, vocab, n):
    """Halves make many equal logits: ties go to the lower token."""
    g = torch.Generator(device="cuda").manual_seed(vocab + beams)
    logits = (3 * torch.randn((groups, beams, vocab), device="cuda", generator=g)).to(DT[dtype])
    scores = -5 * torch.rand((groups, beams), device="cuda", generator=g)
    check_beam(G, logits, scores, n)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["equal", "equal-rows", "rising", "falling", "barred", "all-barred", "nan", "plus-inf", "dead", "all-dead", "lowest",
                                  "zeros", "first"])
@pytest.mark.parametrize("vocab", [33, 9001, 40000])
def test_beam_select_masks_and_ties(G, kind, vocab):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    beams, n = 4, 8
    x = torch.randn((2, beams, vocab), device="cuda", generator=g)
    s = -torch.rand((2, beams), device="cuda", generator=g)
    if kind == "equal":
        x = torch.full_like(x, 1.25)
    elif kind == "equal-rows":
        x, s = x[:, :1].expand(2, beams, vocab).contiguous(), torch.full_like(s, -2.5)
    elif kind == "rising":
        x = torch.arange(vocab, device="cuda").float().div(vocab).expand(2, beams, vocab).contiguous()
    elif kind == "falling":
        x = -torch.arange(vocab, device="cuda").float().div(vocab).expand(2, beams, vocab).contiguous()
    elif kind == "barred":  # fewer tokens left than candidates wanted
        keep = torch.zeros((2, beams, vocab), dtype=torch.bool, device="cuda")
        keep[0, 1, vocab // 2] = keep[0, 3, vocab - 1] = keep[1, 0, 0] = True
        x = torch.where(keep, x, -math.inf)
    elif kind == "all-barred":
        x[0] = -math.inf
    elif kind == "nan":
        x[:, :, ::3] = math.nan
        x[1, 2] = math.nan
    elif kind == "plus-inf":
        x[0, 1, 5] = x[0, 1, vocab - 1] = x[1, 0, 7] = math.inf
    elif kind == "dead":
        s[0, 0] = s[1, 1] = -math.inf
        s[1, 2] = math.nan
    elif kind == "all-dead":
        s[1] = -math.inf
    elif kind == "lowest":  # masks of the type's lowest value are values
        x[:, :, vocab // 4:] = torch.finfo(torch.float32).min
        x[1, 1] = torch.finfo(torch.float32).min
    elif kind == "zeros":
        x = torch.where(torch.arange(vocab, device="cuda") % 2 == 0, -0.0, 0.0).expand(2, beams, vocab).contiguous()
    elif kind == "first":  # the first step: all beams alike, one alive
        s[:, 1:] = -math.inf
    check_beam(G, x, s, n)


@pytest.mark.gpu
def test_beam_select_strided_and_unaligned_rows(G):
    g = torch.Generator(device="cuda").manual_seed(4)
    for dtype in DT.values():
        big = torch.randn((2 * 3, 5000), device="cuda", generator=g).to(dtype)
        big[:, :3] = big[:, 4000:] = math.inf  # not part of the rows
        s = torch.zeros((2, 3), device="cuda")
        check_beam(G, big.view(2, 3, 5000)[:, :, 3:4000], s, 4)
        one = big.view(6, 1, 5000)[:, :, 3:4000]
        check_beam(G, one, torch.zeros((6, 1), device="cuda"), 4)
    with pytest.raises(ValueError):
        G.beam_select(big.view(3, 2, 5000).transpose(0, 1), s)
    with pytest.raises(ValueError):
        G.beam_select(big.view(2, 3, 5000)[:, :, ::2], s)
    with pytest.raises(G.StepqError):
        G.beam_select(big[:1].expand(6, 5000).view(2, 3, 5000), s)
    assert all(t.shape == (0, 3) for t in G.beam_select(big.view(2, 3, 5000)[:0], s[:0]))


@pytest.mark.gpu
@pytest.mark.parametrize("variant", [GDN, KDA, LINEAR])
def test_calls_behind_one_another(G, variant):
    """Prompts and selections without a wait between them, which get the same scratch in turn: each as if alone."""
    sets = []
    for seed, lengths in enumerate([[130, 5, 64], [1, 200, 70]]):
        q, k, v, alpha, beta, St = prompt_inputs(variant, torch.bfloat16, lengths, 4, 2, seed)
        p = G.RequestPlan(3, sum(lengths))
        p.build(i32(lengths), i32([7, 0, 7]))
        x = torch.randn((3, 4, 9001), device="cuda")
        sets.append((p, q, k, v, alpha, beta, St, x, -torch.rand((3, 4), device="cuda")))

    def both(p, q, k, v, alpha, beta, St, x, s):
        St = St.clone()
        return [G.prompt(variant, p, q, k, v, alpha, beta, St), St, *G.beam_select(x, s)]

    alone = []
    for x in sets:
        alone.append(both(*x))
        torch.cuda.synchronize()
    got = [both(*sets[i % 2]) for i in range(24)]
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, alone[i % 2]))
    # and captured: a graph of the same calls, replayed twice without a wait
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(*sets[0])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [both(*sets[i % 2]) for i in range(4)]
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for i, outs in enumerate(kept):
        assert all(torch.equal(a, b) for a, b in zip(outs, alone[i % 2]))


@pytest.mark.gpu
@pytest.mark.parametrize("groups,beams,row", [(1, 1, 16), (3, 2, 48), (2, 5, 1040), (4, 8, 33 * 1024), (1, 64, 4112), (7, 3, 5 * 16)])
def test_reorder_rows(G, groups, beams, row):
    rng = np.random.default_rng(beams)
    rows = torch.from_numpy(rng.integers(0, 256, (groups * beams, row), dtype=np.uint8)).cuda()
    cases = [rng.integers(0, beams, (groups, beams)), np.tile(np.arange(beams), (groups, 1)), np.tile(np.arange(beams)[::-1], (groups, 1)),
             np.zeros((groups, beams)), rng.integers(-2, beams + 2, (groups, beams)), np.full((groups, beams), -1)]
    for parents in cases:
        parents = parents.astype(np.int32)
        want = rows.clone()
        for g in range(groups):
            for i in range(beams):
                p = int(parents[g, i])
                want[g * beams + i] = rows[g * beams + (p if 0 <= p < beams else i)]
        got = rows.clone()
        assert G.reorder_rows(got, torch.from_numpy(parents).cuda()) is got
        assert torch.equal(got, want)


@pytest.mark.gpu
def test_reorder_refusals(G):
    rows = torch.zeros((6, 8), device="cuda")
    par = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    G.reorder_rows(rows, par)
    with pytest.raises(ValueError):
        G.reorder_rows(rows[:5], par)
    with pytest.raises(ValueError):
        G.reorder_rows(rows.t(), par.view(2, 3, 1))
    with pytest.raises(TypeError):
        G.reorder_rows(rows, par.long())
    with pytest.raises(G.StepqError, match="16"):
        G.reorder_rows(torch.zeros((6, 3), device="cuda"), par)
    pool = G.PackedStatePool(GDN, 5, 1, np.full((1, 128), 4), np.ones((1, 128)))
    with pytest.raises(G.StepqError, match="pass the pool"):
        pool.reorder(par)
    with pytest.raises(G.StepqError, match="pass the pool"):
        pool.reorder(par[:1], first=3)
    with pytest.raises(ValueError):
        pool.beam_step(torch.zeros((2, 3, 9), device="cuda"), torch.zeros((2, 3), device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("ci", [1, 2])
def test_pool_beam_step(G, ci):
    """Selection and reordering of a pool's mixed-width states; requests outside the groups stay."""
    cfg = W.with_overrides(W.CONFIGS[ci], batch=8, heads=6)
    pool = G.PackedStatePool(cfg.variant, 8, 6, W.bit_table(cfg), W.rho(cfg), cfg.ls_iters)
    g = torch.Generator(device="cuda").manual_seed(ci)
    pool.pack(0.2 * torch.randn((8, 6, 128, 128), device="cuda", generator=g))
    before = pool.state.clone().view(8, -1)
    logits = torch.randn((2, 3, 501), device="cuda", generator=g)
    scores = torch.zeros((2, 3), device="cuda")
    scores[1, 1:] = -math.inf
    got_s, parents, tokens = pool.beam_step(logits, scores, first=1)
    want = G.beam_select(logits, scores)
    assert torch.equal(got_s, want[0]) and torch.equal(parents, want[1]) and torch.equal(tokens, want[2])
    src = [0] + [1 + 3 * i + (p if p >= 0 else j) for i, ps in enumerate(parents.tolist()) for j, p in enumerate(ps)] + [7]
    torch.cuda.synchronize()
    pool.check_guards()
    assert torch.equal(pool.state.view(8, -1), before[src])


# ---- together --------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("variant", [GDN, KDA])
def test_prompts_to_beams(G, variant):
    """Two prompts into slots the plan finds, packed into a pool of 8-bit states, decoded, spread over beams by a first
    selection, decoded again, reordered by a second: against the float64 recurrence of the surviving beams, within the drift
    of 8-bit states."""
    H, B, V = 2, 3, 400
    lengths = [70, 9]
    q, k, v, alpha, beta, _ = prompt_inputs(variant, torch.float32, lengths, H, H, 31)
    St = torch.full((2, H, 128, 128), float("nan"), device="cuda")
    pool = G.PackedStatePool(variant, 2 * B, H, np.full((H, 128), 8), np.ones((H, 128)))
    pool.pack(torch.zeros((2 * B, H, 128, 128), device="cuda"))
    # slots 0 and 3 are free: the first beams of the two groups
    busy = torch.tensor([0, 1, 1, 0, 1, 1], dtype=torch.uint8, device="cuda")
    plan = G.RequestPlan(2, sum(lengths), 2 * B).build(i32(lengths), None, i32([-1, -1]), busy)
    plan.check()
    assert plan.slots.tolist() == [0, 3] and busy.tolist() == [1] * 6
    out = G.prompt(variant, plan, q, k, v, alpha, beta, St)
    want_o, want_S = ref.recurrence(variant, lengths, q, k, v, alpha, beta, torch.zeros_like(St))
    assert rel(out, want_o) <= tolerance(70, torch.float32)
    pool.pack_requests(plan, St)
    g = torch.Generator(device="cuda").manual_seed(2)
    state = [want_S[0]] + [torch.zeros_like(want_S[0])] * 2 + [want_S[1]] + [torch.zeros_like(want_S[0])] * 2
    scores = torch.tensor([[0.0] + [-math.inf] * (B - 1)] * 2, device="cuda")
    for step in range(3):
        x = prompt_inputs(variant, torch.float32, [1] * (2 * B), H, H, 40 + step)
        got = pool.decode_step(*(t.contiguous() for t in x[:5]))
        want = []
        for b in range(2 * B):
            o, s = ref.recurrence(variant, [1], *(t[b:b + 1] for t in x[:5]), state[b][None])
            want.append(o[0])
            state[b] = s[0]
        live = [b for b in range(2 * B) if scores.flatten()[b] > -math.inf]
        assert rel(got[live], torch.stack(want)[live]) <= 0.02 * (step + 1)
        logits = torch.randn((2, B, V), device="cuda", generator=g)
        new_scores, parents, tokens = pool.beam_step(logits, scores)
        picked = ref.beam(logits.cpu(), scores.cpu(), B)
        assert parents.tolist() == [[c[1] for c in p] for p in picked] and tokens.tolist() == [[c[2] for c in p] for p in picked]
        state = [state[(b // B) * B + picked[b // B][b % B][1]] for b in range(2 * B)]
        scores = new_scores
    full = pool.unpack()
    assert rel(full, torch.stack(state)) <= 0.06
    pool.check()
    pool.check_guards()
