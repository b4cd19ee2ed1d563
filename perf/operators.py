"""Cases for measuring the generation operators around the packed decode step.

Four operators take a request from its prompt to its beams:

* ``prefill``  linear attention with one decay per head over ragged prompts, for
  the additive rule  M_t = a_t M_{t-1} + k_t v_t^T  and for the delta rule
  M_t = a_t M_{t-1} + b_t k_t (v_t - a_t M_{t-1}^T k_t)^T,  o_t = M_t^T q_t;
* ``step``     the same recurrence for one token of every request;
* ``select``   beam search's selection: the best num_out continuations of a
  request over its beams and the vocabulary;
* ``reorder``  the survivors' states stay where they are, and the states of
  beams that split are copied into the slots of beams that ended.

Heads, head sizes and batches are those of the repository's workloads (48 heads
of 128 under a per-head gate, 32 heads of 128, batch 512, 6-bit slots); prompt
lengths, beam counts and vocabularies are generic.

With ``own`` false, ``run`` computes the plain form with elementary torch
operations in 32 bits; with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
CHUNK = 64           # of the plain form
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EOS = 2


def listed():
    return [
        # one short prompt: a chat turn, where the call's latency is what the user waits for
        dict(name="prefill delta short", op="prefill", rule="delta", dtype="bf16", batch=1, tokens=37,
             heads=48, qk_heads=16, dim=128, resume=False),
        # a batch of prompts admitted together, half of them continuing an earlier chunk of the prompt
        dict(name="prefill delta batch", op="prefill", rule="delta", dtype="bf16", batch=8, tokens=8192,
             heads=48, qk_heads=16, dim=128, resume=True),
        # the largest admission: a full token budget, shared key heads
        dict(name="prefill delta largest", op="prefill", rule="delta", dtype="bf16", batch=16, tokens=32768,
             heads=48, qk_heads=16, dim=128, resume=False),
        # a few prompts of a half-precision model with a key head for every value head
        dict(name="prefill delta f16", op="prefill", rule="delta", dtype="f16", batch=3, tokens=5001,
             heads=32, qk_heads=32, dim=128, resume=False),
        # one long document: few rows, a long axis
        dict(name="prefill additive long", op="prefill", rule="additive", dtype="bf16", batch=1, tokens=16384,
             heads=32, qk_heads=32, dim=128, resume=False),
        # a small model in single precision, odd lengths
        dict(name="prefill additive f32", op="prefill", rule="additive", dtype="f32", batch=5, tokens=3001,
             heads=12, qk_heads=12, dim=64, resume=True),
        # one request's next token: latency
        dict(name="step additive one", op="step", rule="additive", dtype="bf16", batch=1, tokens=1,
             heads=48, qk_heads=16, dim=128, resume=True),
        # the serving batch's next token, states in binary32
        dict(name="step delta serving", op="step", rule="delta", dtype="f32", batch=512, tokens=512,
             heads=48, qk_heads=48, dim=128, resume=True),
        # one request, four beams
        dict(name="select one", op="select", dtype="f32", batch=1, beams=4, vocab=32000, num_out=4, finished=False),
        # a batch of beam searches that keeps twice as many candidates as beams, some beams finished
        dict(name="select batch", op="select", dtype="bf16", batch=32, beams=8, vocab=131072, num_out=16, finished=True),
        # the first step of a search: the prompt's state is forked into its beams
        dict(name="reorder fork", op="reorder", batch=1, beams=4, dead=3, heads=32, dim=128, bits=6),
        # a step of 64 searches, three beams in eight ending
        dict(name="reorder batch", op="reorder", batch=64, beams=8, dead=3, heads=48, dim=128, bits=6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "step", "select", "reorder"])
    if op in ("prefill", "step"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        dim = rng.choice([32, 64, 128, 128])
        qk_heads = rng.choice([4, 8, 16])
        heads = qk_heads * rng.choice([1, 2, 3])
        batch = _log_int(rng, 1, 24) if op == "prefill" else _log_int(rng, 1, 500)
        tokens = batch if op == "step" else max(batch, _log_int(rng, 20, 30000 if dtype == "bf16" else 9000))
        return dict(op=op, rule=rng.choice(["delta", "additive"]), dtype=dtype, batch=batch, tokens=tokens,
                    heads=heads, qk_heads=qk_heads, dim=dim, resume=op == "step" or rng.random() < 0.5)
    if op == "select":
        beams = rng.randint(1, 12)
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), batch=_log_int(rng, 1, 24), beams=beams,
                    vocab=_log_int(rng, 1000, 120000), num_out=rng.randint(beams, 2 * beams), finished=rng.random() < 0.5)
    beams = rng.randint(2, 10)
    return dict(op=op, batch=_log_int(rng, 1, 50), beams=beams, dead=rng.randint(1, beams - 1),
                heads=rng.randint(1, 48), dim=rng.choice([32, 64, 128]), bits=rng.choice([4, 6, 8]))


def _lengths(batch, tokens, g):
    """Ragged lengths that add up to `tokens`; an empty prompt and one of a single token where there are many."""
    if batch == 1:
        return np.array([tokens], dtype=np.int64)
    w = g.uniform(0.25, 1.75, size=batch)
    special = batch >= 4 and tokens >= 4 * batch
    if special:
        w[1] = w[2] = 0.0
    rest = tokens - (1 if special else 0)
    cuts = np.floor(np.cumsum(w) / w.sum() * rest + 0.5).astype(np.int64)
    n = np.diff(np.r_[0, cuts])
    if special:
        n[2] = 1
    assert n.sum() == tokens and n.min() >= 0
    return n


def _slot_bytes(case):
    """A slot's codes and scales: dim * dim fields of `bits` bits and 2 * dim binary16 scales for every head."""
    d, h = case["dim"], case["heads"]
    words = (d * case["bits"] + 31) // 32
    pool = (4 * words * d * h + 255) // 256 * 256
    return pool, 4 * d * h


def prepare(case, seed):
    g = np.random.default_rng(seed)
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    s = dict(case=dict(case), keep={})
    if case["op"] in ("prefill", "step"):
        t, h, hk, d, b = (case[n] for n in ("tokens", "heads", "qk_heads", "dim", "batch"))
        dtype = TYPES[case["dtype"]]
        # q and k have unit norm, v is normal, half-lives are spread over 1 to 1000 tokens
        s["q"] = unit(normal(t, hk, d)).to(dtype)
        s["k"] = unit(normal(t, hk, d)).to(dtype)
        s["v"] = normal(t, h, d).to(dtype)
        s["beta"] = torch.sigmoid(normal(t, h)) if case["rule"] == "delta" else None
        half_life = 10.0 ** torch.from_numpy(g.uniform(0.0, 3.0, size=h)).to(DEVICE, torch.float32)
        s["gate"] = torch.exp2(-(1.0 + 0.2 * torch.rand(t, h, generator=gen, device=DEVICE)) / half_life)
        s["o"] = torch.empty(t, h, d, dtype=dtype, device=DEVICE)
        s["num_slots"] = b + 3
        s["slots"] = torch.from_numpy(g.permutation(b + 3)[:b].astype(np.int32)).to(DEVICE)
        s["state"] = 0.1 * normal(b + 3, h, d, d)
        if case["op"] == "prefill":
            n = _lengths(b, t, g)
            s["max_len"] = int(n.max())
            s["cu"] = torch.from_numpy(np.r_[0, np.cumsum(n)].astype(np.int32)).to(DEVICE)
            s["resume"] = torch.from_numpy((g.random(b) < 0.5).astype(np.uint8)).to(DEVICE) if case["resume"] else None
    elif case["op"] == "select":
        rows, v = case["batch"] * case["beams"], case["vocab"]
        # a language model's logits: a broad bulk and a few dozen likely tokens
        x = 2.0 * normal(rows, v)
        at = torch.randint(0, v // 40, (rows, 40), generator=gen, device=DEVICE) + torch.arange(40, device=DEVICE) * (v // 40)
        x.scatter_(1, at, 8.0 + 2.0 * normal(rows, 40))
        x[:, 0] = -math.inf                                        # a banned token
        s["logits"] = x.to(TYPES[case["dtype"]])
        s["scores"] = -3.0 * torch.rand(rows, generator=gen, device=DEVICE) - 4.0
        s["finished"] = (torch.rand(rows, generator=gen, device=DEVICE) < 0.15).to(torch.uint8) if case["finished"] else None
    else:
        b, k = case["batch"], case["beams"]
        pool, scales = _slot_bytes(case)
        s["num_slots"] = b * k + 5
        s["pool"] = torch.randint(0, 256, (s["num_slots"], pool), generator=gen, device=DEVICE, dtype=torch.uint8)
        s["scales"] = torch.randint(0, 256, (s["num_slots"], scales), generator=gen, device=DEVICE, dtype=torch.uint8)
        s["slots"] = torch.from_numpy(g.permutation(s["num_slots"])[:b * k].astype(np.int32)).to(DEVICE)
        s["new_slots"] = torch.empty_like(s["slots"])
        parents = np.empty((b, k), dtype=np.int32)
        for i in range(b):                       # `dead` beams end; the others have one child or more
            alive = g.permutation(k)[:k - case["dead"]]
            parents[i] = g.permutation(np.r_[alive, g.choice(alive, size=case["dead"])])
        s["parents"] = torch.from_numpy(parents.reshape(-1)).to(DEVICE)
    return s


def work(case):
    if case["op"] in ("prefill", "step"):
        t, h, hk, d, b = (case[n] for n in ("tokens", "heads", "qk_heads", "dim", "batch"))
        e = 4 if case["dtype"] == "f32" else 2
        delta = case["rule"] == "delta"
        reads = 1.0 if case["op"] == "step" else 0.5 if case["resume"] else 0.0
        states = b * h * d * d * 4
        byts = 2 * t * hk * d * e + 2 * t * h * d * e + t * h * 4 * (2 if delta else 1) + states * (1 + reads)
        return {"bytes": byts, "flops": t * h * d * d * (6 if delta else 4)}
    if case["op"] == "select":
        rows = case["batch"] * case["beams"]
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": rows * (case["vocab"] * e + 4) + case["batch"] * case["num_out"] * 12,
                "flops": 3 * rows * case["vocab"]}
    pool, scales = _slot_bytes(case)
    n = case["batch"] * case["beams"]
    return {"bytes": case["batch"] * case["dead"] * 2 * (pool + scales) + 12 * n, "flops": 0}


# ---------------------------------------------------------------- plain forms

def _expand(x, heads):
    """Value head h reads key head h // (heads / key heads)."""
    return x.repeat_interleave(heads // x.shape[-2], dim=-2)


def _plain_prefill(s):
    """Chunks of 64 tokens: with G_t the product of the chunk's retentions up to t,
    (I + B) U = diag(b) (V - diag(G) K M),  B_ij = b_i (G_i / G_j) k_i.k_j  for j < i  (additive rule: U = V),
    O = diag(G) Q M + A U,  A_ij = (G_i / G_j) q_i.k_j  for j <= i,   M <- G_C M + (K diag(G_C / G))^T U."""
    q, k, v, gate, beta, cu = (s[n] for n in ("q", "k", "v", "gate", "beta", "cu"))
    t, h, d = v.shape
    b = cu.numel() - 1
    n = max(1, -(-s["max_len"] // CHUNK))
    pos = torch.arange(n * CHUNK, device=v.device)
    real = pos[None, :] < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + pos[None, :]).clamp(max=t - 1)

    def chunks(x, fill):                                     # [T, H, ...] -> [B, H, n, C, ...]
        y = x.float()[at]
        y = torch.where(real.reshape(real.shape + (1,) * (y.dim() - 2)), y, fill)
        y = y.reshape((b, n, CHUNK) + y.shape[2:])
        return y.movedim(3, 1)

    qc, kc, vc = chunks(_expand(q, h), 0.0), chunks(_expand(k, h), 0.0), chunks(v, 0.0)
    log_g = chunks(gate, 1.0).log().cumsum(-1)               # [B, H, n, C]
    lower = torch.ones(CHUNK, CHUNK, device=v.device, dtype=torch.bool).tril()
    ratio = torch.where(lower, log_g[..., :, None] - log_g[..., None, :], -math.inf).exp()
    a = (qc @ kc.transpose(-1, -2)) * ratio
    if beta is not None:
        bc = chunks(beta, 0.0)[..., None]
        low = ((kc @ kc.transpose(-1, -2)) * ratio * bc).tril(-1)
        inv = torch.eye(CHUNK, device=v.device).expand_as(low).clone()
        for i in range(1, CHUNK):                            # rows of (I + B)^-1, by substitution
            inv[..., i, :i] = -(low[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    grow, left = log_g.exp()[..., None], (log_g[..., -1:] - log_g).exp()[..., None]
    m = s["state"][s["slots"].long()]
    m = torch.zeros_like(m) if s["resume"] is None else m * s["resume"].float()[:, None, None, None]
    out = torch.empty_like(vc)
    for c in range(n):
        u = vc[:, :, c]
        if beta is not None:
            u = inv[:, :, c] @ (bc[:, :, c] * (u - grow[:, :, c] * (kc[:, :, c] @ m)))
        out[:, :, c] = grow[:, :, c] * (qc[:, :, c] @ m) + a[:, :, c] @ u
        m = grow[:, :, c, -1:] * m + (left[:, :, c] * kc[:, :, c]).transpose(-1, -2) @ u
    out = out.movedim(1, 3).reshape(b, n * CHUNK, h, d)
    s["o"][at[real]] = out[real].to(s["o"].dtype)
    s["state"][s["slots"].long()] = m
    return {"o": s["o"], "state": s["state"]}


def _plain_step(s):
    h = s["v"].shape[1]
    q, k, v = _expand(s["q"].float(), h), _expand(s["k"].float(), h), s["v"].float()
    m = s["state"][s["slots"].long()] * s["gate"][:, :, None, None]
    u = v if s["beta"] is None else s["beta"][..., None] * (v - (m * k[..., None]).sum(-2))
    m = m + k[..., None] * u[:, :, None, :]
    s["state"][s["slots"].long()] = m
    return {"o": (m * q[..., None]).sum(-2).to(s["v"].dtype), "state": s["state"]}


def _plain_select(s):
    """A beam's own order is by logit, then token; candidates of different beams
    are ordered by score, then beam.  A finished beam has one continuation: the
    end token, at its own score."""
    c = s["case"]
    b, k, n = c["batch"], c["beams"], c["num_out"]
    x = s["logits"].float()
    top, token = x.sort(dim=-1, descending=True, stable=True)
    top, token = top[:, :n], token[:, :n]
    most = top[:, :1]
    lse = (x - most).exp().sum(-1, keepdim=True).log()
    score = s["scores"][:, None] + ((top - most) - lse)
    if s["finished"] is not None:
        done, first = s["finished"].bool()[:, None], torch.arange(n, device=x.device)[None, :] == 0
        score = torch.where(done, torch.where(first, s["scores"][:, None], -math.inf), score)
        token = torch.where(done, EOS, token)
    score, token = score.reshape(b, -1), token.reshape(b, -1)
    best, at = score.sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    none = best == -math.inf
    return {"tokens": torch.where(none, -1, token.gather(1, at)).int(),
            "parents": torch.where(none, -1, at // n).int(), "scores": best}


def _plain_reorder(s):
    """A beam's first child keeps its slot; the others take the slots of beams without children, in order."""
    k = s["case"]["beams"]
    slots, parents = s["slots"].reshape(-1, k).long(), s["parents"].reshape(-1, k).long()
    child = parents[:, None, :] == torch.arange(k, device=slots.device)[None, :, None]          # [B, beam, child]
    first = (child & (child.cumsum(-1) == 1)).any(1)
    dead = ~child.any(-1)
    order = dead.to(torch.int32).sort(dim=-1, descending=True, stable=True).indices              # dead beams, ascending
    rank = (~first).cumsum(-1) - 1
    source = slots.gather(1, parents)
    new = torch.where(first, source, slots.gather(1, order.gather(1, rank.clamp(min=0))))
    for buf in (s["pool"], s["scales"]):
        buf[new.reshape(-1)] = buf[source.reshape(-1)]
    s["new_slots"].copy_(new.reshape(-1))
    return {"new_slots": s["new_slots"], "pool": s["pool"], "scales": s["scales"]}


# ------------------------------------------------------------------- run

def _run_own(s):
    c, keep = s["case"], s["keep"]
    if c["op"] in ("prefill", "step"):
        from quantized_recurrent_state_packed_amd import linear
        att = keep.get("att")
        if att is None:      # the handle and its workspace, which a program keeps
            att = keep["att"] = linear.LinearAttention(c["heads"], c["dim"], num_qk_heads=c["qk_heads"],
                                                       rule=c["rule"], dtype=TYPES[c["dtype"]])
        if c["op"] == "step":
            att.step(s["slots"], s["q"], s["k"], s["v"], s["beta"], s["gate"], s["state"], s["o"])
            return {"o": s["o"], "state": s["state"]}
        if "ws" not in keep:
            keep["ws"] = att.workspace(c["batch"], c["tokens"], device=DEVICE)
        att.prefill(s["cu"], s["q"], s["k"], s["v"], s["beta"], s["gate"], s["slots"], s["state"], s["o"],
                    resume=s["resume"], workspace=keep["ws"])
        return {"o": s["o"], "state": s["state"]}
    from quantized_recurrent_state_packed_amd import beam
    if c["op"] == "select":
        sel = keep.get("select")
        if sel is None:
            sel = keep["select"] = beam.BeamSelect(c["batch"], c["beams"], c["vocab"], c["num_out"],
                                                   TYPES[c["dtype"]], eos_token=EOS, device=DEVICE)
        tokens, parents, scores = sel(s["logits"], s["scores"], finished=s["finished"])
        return {"tokens": tokens, "parents": parents, "scores": scores}
    beam.reorder(c["beams"], s["slots"], s["parents"], [s["pool"], s["scales"]], s["new_slots"])
    return {"new_slots": s["new_slots"], "pool": s["pool"], "scales": s["scales"]}


def run(state):
    if own:
        return _run_own(state)
    return {"prefill": _plain_prefill, "step": _plain_step, "select": _plain_select,
            "reorder": _plain_reorder}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    if case["op"] == "reorder":
        return None                                           # whole numbers only
    if case["op"] == "select":
        s = prepare(case, seed)
        b, n = case["batch"], case["num_out"]
        x = s["logits"].double()
        score = s["scores"].double()[:, None] + torch.log_softmax(x, dim=-1)
        if s["finished"] is not None:
            done = s["finished"].bool()
            score[done] = -math.inf
            score[done, EOS] = s["scores"].double()[done]
        best = torch.topk(score.reshape(b, -1), n, dim=-1).values
        return {"tokens": None, "parents": None, "scores": best}
    t, h, d, b = case["tokens"], case["heads"], case["dim"], case["batch"]
    rep = h // case["qk_heads"]
    s = prepare(case, seed)
    if case["op"] == "step":
        cu, keep_state = list(range(b + 1)), torch.ones(b, device=DEVICE, dtype=torch.float64)
    else:
        cu = s["cu"].tolist()
        keep_state = (torch.zeros(b, device=DEVICE) if s["resume"] is None else s["resume"]).double()
    state = s["state"].double()
    out = torch.zeros(t, h, d, device=DEVICE, dtype=torch.float64)
    m = state[s["slots"].long()] * keep_state[:, None, None, None]
    # token by token, the requests that still have one at a time
    order = sorted(range(b), key=lambda i: cu[i] - cu[i + 1])
    start = torch.tensor([cu[i] for i in order], device=DEVICE)
    length = [cu[i + 1] - cu[i] for i in order]
    index = torch.tensor(order, device=DEVICE)
    m = m[index]
    live = b
    for p in range(max(length)):
        while length[live - 1] <= p:
            live -= 1
        at = start[:live] + p
        kt = s["k"][at].double().repeat_interleave(rep, 1)
        qt = s["q"][at].double().repeat_interleave(rep, 1)
        vt = s["v"][at].double()
        mt = m[:live]
        mt *= s["gate"][at].double()[:, :, None, None]
        if case["rule"] == "delta":
            vt = s["beta"][at].double()[:, :, None] * (vt - torch.matmul(kt[:, :, None, :], mt)[:, :, 0])
        mt += kt[:, :, :, None] * vt[:, :, None, :]
        out[at] = torch.matmul(qt[:, :, None, :], mt)[:, :, 0]
    state[s["slots"].long()[index]] = m
    return {"o": out, "state": state}
