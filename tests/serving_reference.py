"""Plain implementations of the serving operators for the tests: the plan request by request in Python, the recurrence token
by token and the beam selection in float64.  They share nothing with the library."""
import math

import torch

BAD_LENGTH, TOO_MANY, BAD_SLOT, SLOT_TWICE, NO_SLOT = 1, 2, 4, 8, 16
BLOCK = 64


def plan(requests, tokens, n_slots, lengths, contexts=None, slots=None, busy=None, max_length=None):
    n = len(lengths)
    max_length = tokens if max_length is None else max_length
    contexts = contexts or [0] * n
    busy = None if busy is None else list(busy)
    p = dict(starts=[0], block_starts=[0], slots=[-1] * requests, live=[-1] * requests, fresh=[0] * requests, token_request=[-1] * tokens,
             token_position=[-1] * tokens, block_request=[], block_first=[], status=0)
    over = False
    used = 0
    want = {}
    lens = []
    for r in range(n):
        ln = lengths[r]
        if ln < 0:
            p["status"] |= BAD_LENGTH
            ln = 0
        if not over and used + ln > tokens:
            over = True
        if over:
            p["status"] |= TOO_MANY
            ln = 0
        lens.append(ln)
        for i in range(ln):
            p["token_request"][used + i] = r
            p["token_position"][used + i] = contexts[r] + i
        for b in range(0, ln, BLOCK):
            p["block_request"].append(r)
            p["block_first"].append(b)
        used += ln
        p["starts"].append(used)
        p["block_starts"].append(len(p["block_first"]))
        p["fresh"][r] = int(contexts[r] == 0)
        s = r if slots is None else slots[r]
        good = 0 <= s < n_slots
        p["slots"][r] = s if good else -1
        if ln == 0:
            continue
        if lengths[r] > max_length:
            p["status"] |= BAD_LENGTH
        elif good:
            if s in want:
                p["status"] |= SLOT_TWICE
            else:
                want[s] = r
                p["live"][r] = s
                if busy is not None:
                    busy[s] = 1
        elif not (s == -1 and contexts[r] == 0 and busy is not None):
            p["status"] |= BAD_SLOT
        else:
            p["live"][r] = -2
    for r in range(n):
        if p["live"][r] == -2:
            free = next((s for s in range(n_slots) if busy[s] == 0), None)
            if free is None:
                p["status"] |= NO_SLOT
                p["live"][r] = -1
            else:
                busy[free] = 1
                p["live"][r] = p["slots"][r] = free
    p["starts"] += [used] * (requests - n)
    p["block_starts"] += [len(p["block_first"])] * (requests - n)
    blocks = tokens // BLOCK + requests
    for f in ("block_request", "block_first"):
        p["head_blocks"] = len(p[f])
        p[f] += [-1] * (blocks - len(p[f]))
    p["busy"] = busy
    p["head"] = [p.pop("status"), n, used, p.pop("head_blocks")]
    return p


def recurrence(variant, lengths, q, k, v, alpha, beta, S):
    """variant 0 (one gate a head), 1 (one a key row), 2 (no Delta correction).  S [requests, H, 128, 128].  Returns (out of
    the token rows, S after) in float64."""
    H = v.shape[1]
    share = H // q.shape[1]
    S = S.double().clone()
    q, k = (x.double().repeat_interleave(share, 1) for x in (q, k))
    v, alpha, beta = v.double(), alpha.double(), beta.double()
    out = torch.zeros((q.shape[0], H, 128), dtype=torch.float64, device=q.device)
    t = 0
    for r, n in enumerate(lengths):
        for _ in range(n):
            a = alpha[t][:, :, None] if variant == 1 else alpha[t][:, None, None]
            S[r] = S[r] * a
            u = v[t]
            if variant != 2:
                u = u - torch.einsum("hkv,hk->hv", S[r], k[t])
            S[r] += k[t][:, :, None] * (beta[t][:, None] * u)[:, None, :]
            out[t] = torch.einsum("hkv,hk->hv", S[r], q[t])
            t += 1
    return out, S


def beam(logits, scores, n):
    """Lists of (score, parent, token) of each group, best first."""
    got = []
    for g in range(logits.shape[0]):
        cand = []
        for b in range(logits.shape[1]):
            x = logits[g, b].double()
            x = torch.where(x.isnan(), -math.inf, x)
            top = x.max().item()
            s = scores[g, b].item()
            if top == -math.inf or not s > -math.inf:
                continue
            d = torch.where(x == top, 0.0, x - top)
            total = s + (d - d.exp().sum().log())
            val, at = total.sort(descending=True, stable=True)
            keep = val > -math.inf
            cand += [(-v, b, t) for v, t in zip(val[keep][:n].tolist(), at[keep][:n].tolist())]
        cand.sort()
        got.append([(-v, b, t) for v, b, t in cand[:n]] + [(-math.inf, -1, -1)] * max(0, n - len(cand)))
    return got
