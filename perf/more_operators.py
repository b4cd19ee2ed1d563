"""Cases for measuring the operators of a gated recurrent block and of drafted tokens.

* ``scan``    the gated linear recurrence over ragged prompts, channel by channel:
  a_t = exp(-rate s(ga_t) softplus(decay)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(gx_t) x_t,
  y_t = h_t, s the logistic function, decay a parameter of the channel; the
  states of requests lie in slots;
* ``train``   the same and its backward pass: gradients of x, ga, gx, decay and of the states
  that requests start from;
* ``step``    the recurrence for one token of every request;
* ``norm``    n = rms_norm(block) post,  t = residual + scale n act(gate),  y = rms_norm(t) pre,
  or n act(gate) alone, the norm behind a readout, head by head;
* ``norm_backward``  gradients of the former's inputs and weights, from t and the gradients of t and y;
* ``verify``  drafted tokens against the target's logits: which are accepted, and the token
  after them, from given random numbers.

Widths are those of the repository's workloads (48 heads of 128, 32 heads of 128), the serving
batch of 512 among them; prompt lengths, numbers of drafts and vocabularies are generic.

With ``own`` false, ``run`` computes the plain form with elementary torch
operations in 32 bits (choices between tokens in 64); with ``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
RATE = 8.0
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SCAN_OPS = ("scan", "train", "step")


def listed():
    return [
        # one short prompt: a chat turn, where the call's latency is what the user waits for
        dict(name="scan prompt short", op="scan", dtype="bf16", batch=1, tokens=37, width=4096, resume=False),
        # a batch of prompts admitted together, half of them continuing an earlier part of the prompt
        dict(name="scan prompts batch", op="scan", dtype="bf16", batch=8, tokens=8192, width=6144, resume=True),
        # one long document: a single chain of tokens
        dict(name="scan long document", op="scan", dtype="bf16", batch=1, tokens=32768, width=4096, resume=False),
        # a training step of packed documents
        dict(name="scan training step", op="train", dtype="bf16", batch=6, tokens=12288, width=4096, resume=False),
        # a small model in single precision, odd sizes, states carried over from the part before
        dict(name="scan training f32 odd", op="train", dtype="f32", batch=5, tokens=3001, width=1001, resume=True),
        # the serving batch's next token
        dict(name="scan step serving", op="step", dtype="bf16", batch=512, tokens=512, width=6144, resume=True),
        # the norms around a block for one request's next token: latency
        dict(name="norm one token", op="norm", dtype="bf16", tokens=1, heads=1, width=4096, form="block", act="silu"),
        # the gated norm behind linear attention's readout, head by head
        dict(name="norm gated heads", op="norm", dtype="bf16", tokens=8192, heads=48, width=128, form="gated", act="silu"),
        # the norms around a block, prompts of a batch
        dict(name="norm block prompts", op="norm", dtype="bf16", tokens=8192, heads=1, width=4096, form="block", act="sigmoid"),
        # the same in training, backward
        dict(name="norm block backward", op="norm_backward", dtype="bf16", tokens=8192, heads=1, width=4096, form="block",
             act="silu"),
        # one request, four drafted tokens
        dict(name="verify one", op="verify", dtype="f32", batch=1, drafts=4, vocab=32000, given="logits"),
        # a batch of requests with up to five drafts each, some of them decoded greedily
        dict(name="verify batch", op="verify", dtype="bf16", batch=64, drafts=5, vocab=131072, given="logits"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "step", "norm", "norm_backward", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "step":
        batch = _log_int(rng, 1, 512)
        return dict(op=op, dtype=dtype, batch=batch, tokens=batch, width=_log_int(rng, 60, 6000), resume=True)
    if op in SCAN_OPS:
        width = rng.choice([_log_int(rng, 60, 4096), 128 * rng.randint(1, 32)])
        most = min(30000, (20_000_000 if op == "train" else 50_000_000) // width)
        tokens = _log_int(rng, 20, most)
        return dict(op=op, dtype=dtype, batch=min(tokens, _log_int(rng, 1, 64)), tokens=tokens, width=width,
                    resume=rng.random() < 0.5)
    if op == "verify":
        return dict(op=op, dtype=dtype, batch=_log_int(rng, 1, 48), drafts=rng.randint(1, 7), vocab=_log_int(rng, 1000, 100000),
                    given=rng.choice(["logits", "logits", "tokens"]))
    form = rng.choice(["block", "block", "gated"])
    heads = rng.choice([4, 16, 32, 48]) if form == "gated" else 1
    width = rng.choice([32, 64, 96, 128, 256]) if form == "gated" else rng.choice([_log_int(rng, 100, 8192), 128 * rng.randint(1, 64)])
    tokens = _log_int(rng, 1, min(8192, 30_000_000 // (heads * width)))
    return dict(op=op, dtype=dtype, tokens=tokens, heads=heads, width=width, form=form, act=rng.choice(["silu", "sigmoid"]))


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
    return n


def prepare(case, seed):
    g = np.random.default_rng(seed)
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEVICE)

    s = dict(case=dict(case), keep={})
    op, dtype = case["op"], TYPES[case["dtype"]]
    if op in SCAN_OPS:
        t, d, b = case["tokens"], case["width"], case["batch"]
        # slices of one fused projection, as a model has them
        s["x"], s["ga"], s["gx"] = normal(t, 3, d).to(dtype).unbind(1)
        # half-lives at an open gate's middle of 1 to 1000 tokens
        half_life = 10.0 ** (3.0 * uniform(d).double())
        s["decay"] = torch.log(torch.expm1(math.log(2.0) / (0.5 * RATE * half_life))).float()
        s["y"] = torch.empty(t, d, dtype=dtype, device=DEVICE)
        s["slots"] = torch.from_numpy(g.permutation(b + 3)[:b].astype(np.int32)).to(DEVICE)
        s["state"] = 0.5 * normal(b + 3, d)
        if op != "step":
            n = _lengths(b, t, g)
            s["longest"] = int(n.max())
            s["cu"] = torch.from_numpy(np.r_[0, np.cumsum(n)].astype(np.int32)).to(DEVICE)
            s["resume"] = torch.from_numpy((g.random(b) < 0.5).astype(np.uint8)).to(DEVICE) if case["resume"] else None
        if op == "train":
            s["dy"] = normal(t, d).to(dtype)
            s["dstate"] = normal(b + 3, d)         # of the states that requests end with, then of those that they start from
            s["dx"], s["dga"], s["dgx"] = torch.empty(t, 3, d, dtype=dtype, device=DEVICE).unbind(1)
            s["ddecay"] = torch.empty(d, device=DEVICE)
    elif op in ("norm", "norm_backward"):
        t, h, d = case["tokens"], case["heads"], case["width"]
        block = case["form"] == "block"
        s["block"] = (normal(t, h * d) * (0.3 + uniform(t, 1))).to(dtype)
        s["gate"] = normal(t, h * d).to(dtype)
        s["post"] = 1.0 + 0.2 * normal(d)
        s["residual"] = (2.0 * normal(t, h * d)).to(dtype) if block else None
        s["scale"] = 0.5 + 0.1 * normal(d) if block else None
        s["pre"] = 1.0 + 0.2 * normal(d) if block else None
        if op == "norm":
            s["t"] = torch.empty(t, h * d, dtype=dtype, device=DEVICE)
            s["y"] = torch.empty(t, h * d, dtype=dtype, device=DEVICE) if block else None
        else:
            # what the forward pass left: the residual stream after the block
            s["t"] = (s["residual"].float() + 0.4 * normal(t, h * d)).to(dtype) if block else None
            s["dt"] = normal(t, h * d).to(dtype)
            s["dy"] = normal(t, h * d).to(dtype) if block else None
            for name in ("dblock", "dgate") + (("dresidual",) if block else ()):
                s[name] = torch.empty(t, h * d, dtype=dtype, device=DEVICE)
            for name in ("dpost",) + (("dscale", "dpre") if block else ()):
                s[name] = torch.empty(d, device=DEVICE)
    else:
        b, k, v = case["batch"], case["drafts"], case["vocab"]
        # a language model's logits: a broad bulk and a few dozen likely tokens; the draft is a noisy copy
        x = 2.0 * normal(b * (k + 1), v)
        at = torch.randint(0, v // 40, (b * (k + 1), 40), generator=gen, device=DEVICE) + torch.arange(40, device=DEVICE) * (v // 40)
        x.scatter_(1, at, 8.0 + 2.0 * normal(b * (k + 1), 40))
        x[:, 0] = -math.inf                                        # a banned token
        z = x.view(b, k + 1, v)[:, :k].reshape(b * k, v) + 0.5 * normal(b * k, v)
        s["logits"] = x.to(dtype)
        s["temperature"] = 0.6 + 0.6 * uniform(b)
        if b >= 4:
            s["temperature"][uniform(b) < 0.2] = 0.0               # greedy requests
        s["draft_logits"] = z.to(dtype) if case["given"] == "logits" else None
        # the drafted tokens: chosen by the draft's probabilities, or its most likely ones where they are given as such
        noise = -torch.log(-torch.log(uniform(b * k, v).clamp(1e-20, 1.0 - 6e-8)))
        warm = s["temperature"].repeat_interleave(k)[:, None]
        s["drafts"] = (z + (warm * noise if case["given"] == "logits" else 0.0)).argmax(-1).int().view(b, k)
        s["num_drafts"] = torch.from_numpy(g.integers(0, k + 1, size=b).clip(min=k - 2).astype(np.int32)).to(DEVICE)
        s["uniforms"] = uniform(b, k + 1)
    return s


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op in SCAN_OPS:
        n = case["tokens"] * case["width"]
        starts = 1.0 if op == "step" else 0.5 if case["resume"] else 0.0
        states = case["batch"] * case["width"] * 4 * (1 + starts)
        if op == "train":
            return {"bytes": n * 11 * e + 2 * states + case["width"] * 12, "flops": 60 * n}
        return {"bytes": n * 4 * e + states + case["width"] * 4, "flops": 20 * n}
    if op in ("norm", "norm_backward"):
        n, block = case["tokens"] * case["heads"] * case["width"], case["form"] == "block"
        if op == "norm":
            return {"bytes": n * e * (5 if block else 3) + case["width"] * 4 * (3 if block else 1), "flops": n * (16 if block else 10)}
        return {"bytes": n * e * (8 if block else 5) + case["width"] * 8 * (3 if block else 1), "flops": n * (40 if block else 24)}
    b, k, v = case["batch"], case["drafts"], case["vocab"]
    rows = b * (2 * k + 1) if case["given"] == "logits" else b * (k + 1)
    return {"bytes": rows * v * e + b * (8 * k + 4 * (k + 1) + 12), "flops": 4 * rows * v}


# ---------------------------------------------------------------- plain forms

def _gates(s):
    """log a, sqrt(1 - a^2) and the two gates, [T, D]."""
    sa, sx = torch.sigmoid(s["ga"].float()), torch.sigmoid(s["gx"].float())
    log_a = -RATE * sa * torch.nn.functional.softplus(s["decay"])
    return log_a, torch.sqrt(-torch.expm1(2.0 * log_a)), sa, sx


def _scan(a, u, longest):
    """h_t = a_t h_{t-1} + u_t along the tokens, by doubling; a is 0 at a request's first token."""
    n = 1
    while n < longest:
        u = torch.cat([u[:n], torch.addcmul(u[n:], a[n:], u[:-n])])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return u


def _starts(s):
    start = s["state"][s["slots"].long()]
    return torch.zeros_like(start) if s["resume"] is None else start * s["resume"].float()[:, None]


def _plain_scan(s):
    log_a, b, sa, sx = _gates(s)
    first, last = s["cu"][:-1].long(), s["cu"][1:].long() - 1
    some = last >= first
    a, u, start = log_a.exp(), b * sx * s["x"].float(), _starts(s)
    before = torch.zeros_like(a)                  # the state that a request's first token finds
    before[first[some]] = start[some]
    inside = torch.ones(a.shape[0], 1, device=a.device)
    inside[first[some]] = 0.0
    h = _scan(a * inside, torch.addcmul(u, a, before), s["longest"])
    end = start.clone()
    end[some] = h[last[some]]
    s["y"].copy_(h)
    s["state"][s["slots"].long()] = end
    if s["case"]["op"] == "scan":
        return {"y": s["y"], "state": s["state"]}
    # backward: g_t = dy_t + a_{t+1} g_{t+1}, the last token also takes what the final state gets
    grad_end = s["dstate"][s["slots"].long()]
    dy = s["dy"].float()
    dy[last[some]] += grad_end[some]
    ahead = torch.cat([a[1:], torch.zeros_like(a[:1])])
    ahead[last[some]] = 0.0
    g = _scan(ahead.flip(0), dy.flip(0), s["longest"]).flip(0)
    prior = torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * inside + before
    gain = sx * s["x"].float()
    slope = torch.where(b > 0, log_a / b, 0.0)                     # log a / sqrt(1 - a^2)
    d_log_a = g * (a * prior * log_a - a * a * gain * slope)       # times log a
    s["dga"].copy_(d_log_a * (1.0 - sa))
    sp = torch.nn.functional.softplus(s["decay"])
    s["ddecay"].copy_(d_log_a.sum(0) * torch.sigmoid(s["decay"]) / sp)
    s["dx"].copy_(g * b * sx)
    s["dgx"].copy_(g * b * gain * (1.0 - sx))
    grad_end[some] = (g * a)[first[some]]
    s["dstate"][s["slots"].long()] = grad_end * (0.0 if s["resume"] is None else s["resume"].float()[:, None])
    return _gradients(s)


def _gradients(s):
    return {k: s[k] for k in ("y", "state", "dx", "dga", "dgx", "ddecay", "dstate")}


def _plain_step(s):
    log_a, b, _, sx = _gates(s)
    h = log_a.exp() * s["state"][s["slots"].long()] + b * sx * s["x"].float()
    s["state"][s["slots"].long()] = h
    s["y"].copy_(h)
    return {"y": s["y"], "state": s["state"]}


def _rows(s, name):
    c = s["case"]
    return s[name].float().view(c["tokens"] * c["heads"], c["width"])


def _rstd(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    x, z = _rows(s, "block"), _rows(s, "gate")
    act = torch.sigmoid(z) * (z if s["case"]["act"] == "silu" else 1.0)
    p = x * _rstd(x) * s["post"] * act
    if s["residual"] is None:
        s["t"].copy_(p.view_as(s["t"]))
        return {"t": s["t"]}
    t = _rows(s, "residual") + s["scale"] * p
    s["t"].copy_(t)
    s["y"].copy_(t * _rstd(t) * s["pre"])
    return {"t": s["t"], "y": s["y"]}


def _plain_norm_backward(s):
    x, z, g = _rows(s, "block"), _rows(s, "gate"), _rows(s, "dt")
    sig = torch.sigmoid(z)
    silu = s["case"]["act"] == "silu"
    act, slope = (sig * z, sig * (1.0 + z * (1.0 - sig))) if silu else (sig, sig * (1.0 - sig))
    r = _rstd(x)
    n = x * r * s["post"]
    if s["residual"] is not None:
        t, dy = _rows(s, "t"), _rows(s, "dy")
        rt = _rstd(t)
        s["dpre"].copy_((dy * t * rt).sum(0))
        v = s["pre"] * dy
        g = g + rt * v - t * rt.pow(3) * (t * v).mean(-1, keepdim=True)
        s["dresidual"].copy_(g)
        s["dscale"].copy_((g * n * act).sum(0))
        g = g * s["scale"]
    s["dgate"].copy_((g * n * slope).view_as(s["dgate"]))
    m = g * act
    s["dpost"].copy_((m * x * r).sum(0))
    v = s["post"] * m
    s["dblock"].copy_((r * v - x * r.pow(3) * (x * v).mean(-1, keepdim=True)).view_as(s["dblock"]))
    return {k: s[k] for k in ("dblock", "dgate", "dresidual", "dpost", "dscale", "dpre") if k in s}


def _chances(logits, temperature):
    """softmax(logits / temperature) in 64 bits; at temperature 0 all of it is the first of the largest."""
    x = logits.double()
    most = x.max(-1, keepdim=True).values
    warm = torch.where(temperature > 0, temperature.double(), 1.0)
    e = torch.exp((x - most) / warm)
    best = torch.zeros_like(e).scatter_(-1, (x == most).to(torch.int32).argmax(-1, keepdim=True), 1.0)
    return torch.where(temperature > 0, e / e.sum(-1, keepdim=True), best)


def _plain_verify(s):
    b, k, v = (s["case"][n] for n in ("batch", "drafts", "vocab"))
    warm = s["temperature"].view(b, 1, 1)
    p = _chances(s["logits"].view(b, k + 1, v), warm)
    drafts = s["drafts"].long()
    sharp = torch.zeros(b, k, v, device=p.device, dtype=p.dtype).scatter_(-1, drafts[..., None], 1.0)
    # greedy requests take a drafted token where it is the target's choice, whatever drafted it
    q = sharp if s["draft_logits"] is None else torch.where(warm > 0, _chances(s["draft_logits"].view(b, k, v), warm), sharp)
    u, count = s["uniforms"].double(), s["num_drafts"].long()
    place = torch.arange(k + 1, device=p.device)
    pd, qd = (t[:, :k].gather(-1, drafts[..., None])[..., 0] for t in (p, q))
    good = (u[:, :k] * qd < pd) & (place[:k] < count[:, None])
    n = good.long().cumprod(-1).sum(-1)
    at = n[:, None, None].expand(b, 1, v)
    pn = p.gather(1, at)[:, 0]
    qn = torch.cat([q, torch.zeros_like(q[:, :1])], 1).gather(1, at)[:, 0] * (n < count).double()[:, None]
    rest = (pn - qn).clamp(min=0.0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, pn)
    run_sum = rest.cumsum(-1)
    beyond = (run_sum > u[:, k:] * rest.sum(-1, keepdim=True)) & (rest > 0)
    last = v - 1 - (rest > 0).flip(-1).to(torch.int32).argmax(-1)
    token = torch.where(beyond.any(-1), beyond.to(torch.int32).argmax(-1), last).int()
    padded = torch.cat([s["drafts"], s["drafts"][:, :1]], 1)
    tokens = torch.where(place < n[:, None], padded, torch.where(place == n[:, None], token[:, None], -1))
    return {"accepted": n.int(), "tokens": tokens.int()}


# ------------------------------------------------------------------- run

def _own_scan(s):
    from quantized_recurrent_state_packed_amd import recurrence
    c, keep = s["case"], s["keep"]
    rec = keep.get("rec")
    if rec is None:          # the handle and its workspaces, which a program keeps
        rec = keep["rec"] = recurrence.GatedRecurrence(c["width"], dtype=TYPES[c["dtype"]], rate=RATE)
        if c["op"] != "step":
            keep["ws"] = rec.workspace(c["batch"], c["tokens"], device=DEVICE)
            keep["saved"] = rec.saved(c["batch"], c["tokens"], device=DEVICE) if c["op"] == "train" else None
    if c["op"] == "step":
        rec.step(s["slots"], s["x"], s["ga"], s["gx"], s["decay"], s["state"], s["y"])
        return {"y": s["y"], "state": s["state"]}
    rec.prefill(s["cu"], s["x"], s["ga"], s["gx"], s["decay"], s["slots"], s["state"], s["y"], resume=s["resume"],
                saved=keep["saved"], workspace=keep["ws"])
    if c["op"] == "scan":
        return {"y": s["y"], "state": s["state"]}
    # The plain form works on a binary32 dy in place and leaves the last states' gradients added to it; a second
    # pass on the same state has to meet the same dy here.
    single = c["dtype"] == "f32"
    if single:
        if "last" not in keep:
            some = s["cu"][1:] > s["cu"][:-1]
            keep["last"], keep["ended"] = s["cu"][1:].long()[some] - 1, s["slots"].long()[some]
        grad_end = s["dstate"].index_select(0, keep["ended"])
    rec.backward(s["cu"], s["x"], s["ga"], s["gx"], s["decay"], keep["saved"], s["dy"], s["dx"], s["dga"], s["dgx"],
                 s["ddecay"], slot_ids=s["slots"], dstate=s["dstate"], resume=s["resume"], workspace=keep["ws"])
    if single:
        s["dy"].index_add_(0, keep["last"], grad_end)
    return _gradients(s)


def _own_norm(s):
    from quantized_recurrent_state_packed_amd import norm
    c, keep = s["case"], s["keep"]
    op = keep.get("norm")
    if op is None:
        op = keep["norm"] = norm.BlockNorm(c["width"], heads=c["heads"], dtype=TYPES[c["dtype"]], activation=c["act"],
                                           pre=c["form"] == "block", eps=EPS)
        keep["ws"] = op.workspace(c["tokens"], device=DEVICE) if c["op"] == "norm_backward" else None
    if c["op"] == "norm":
        op.forward(s["block"], s["t"], normed=s["y"], gate=s["gate"], residual=s["residual"], post_weight=s["post"],
                   scale=s["scale"], pre_weight=s["pre"])
        return {"t": s["t"]} if s["y"] is None else {"t": s["t"], "y": s["y"]}
    op.backward(s["block"], s["t"], s["dt"], s["dblock"], d_normed=s["dy"], gate=s["gate"], d_gate=s["dgate"],
                d_residual=s.get("dresidual"), post_weight=s["post"], d_post_weight=s["dpost"], scale=s["scale"],
                d_scale=s.get("dscale"), pre_weight=s["pre"], d_pre_weight=s.get("dpre"), workspace=keep["ws"])
    return {k: s[k] for k in ("dblock", "dgate", "dresidual", "dpost", "dscale", "dpre") if k in s}


def _own_verify(s):
    from quantized_recurrent_state_packed_amd import draft
    c, keep = s["case"], s["keep"]
    op = keep.get("verify")
    if op is None:
        op = keep["verify"] = draft.DraftVerify(c["batch"], c["drafts"], c["vocab"], TYPES[c["dtype"]], device=DEVICE)
    accepted, tokens = op(s["logits"], s["drafts"], s["uniforms"], draft_logits=s["draft_logits"], num_drafts=s["num_drafts"],
                          temperature=s["temperature"])
    return {"accepted": accepted, "tokens": tokens}


def run(state):
    op = state["case"]["op"]
    if own:
        return (_own_scan if op in SCAN_OPS else _own_verify if op == "verify" else _own_norm)(state)
    return {"scan": _plain_scan, "train": _plain_scan, "step": _plain_step, "norm": _plain_norm,
            "norm_backward": _plain_norm_backward, "verify": _plain_verify}[op](state)


# ------------------------------------------------------------------- exact

def _exact_scan(case, s):
    """Token by token, the requests that still have one at a time, forward and then backward."""
    op, b = case["op"], case["batch"]
    x, ga, gx, decay = (s[n].double() for n in ("x", "ga", "gx", "decay"))
    i, r = 1.0 / (1.0 + torch.exp(-gx)), 1.0 / (1.0 + torch.exp(-ga))
    speed = RATE * torch.log1p(torch.exp(decay))
    la = -(speed * r)
    a = torch.exp(la)
    b2 = -torch.expm1(la) * (1.0 + a)
    bb = torch.sqrt(b2)
    u = bb * i * x
    slots = s["slots"].long()
    h0 = s["state"].double()[slots]
    cu = list(range(b + 1)) if op == "step" else s["cu"].tolist()
    if op != "step":
        h0 = h0 * (torch.zeros(b, 1, device=DEVICE).double() if s["resume"] is None else s["resume"].double()[:, None])
    order = sorted(range(b), key=lambda n: cu[n] - cu[n + 1])
    start = torch.tensor([cu[n] for n in order], device=DEVICE)
    length = [cu[n + 1] - cu[n] for n in order]
    index = torch.tensor(order, device=DEVICE)
    h = h0[index]
    y, prior = torch.zeros_like(u), torch.zeros_like(u)
    lives, live = [], b
    for p in range(max(length)):
        while length[live - 1] <= p:
            live -= 1
        lives.append(live)
        at = start[:live] + p
        prior[at] = h[:live]
        h[:live] = a[at] * h[:live] + u[at]
        y[at] = h[:live]
    state = s["state"].double()
    state[slots[index]] = h
    if op != "train":
        return {"y": y, "state": state}
    g = s["dstate"].double()[slots[index]]
    dy, total = s["dy"].double(), torch.zeros_like(u)
    for p in range(max(length) - 1, -1, -1):
        live = lives[p]
        at = start[:live] + p
        now = g[:live] + dy[at]
        total[at] = now
        g[:live] = a[at] * now
    # h = a h' + sqrt(1 - a^2) i x, with a = exp(-speed r)
    d_a = total * (prior - a / bb * i * x)
    d_r = d_a * a * -speed
    d_speed = (d_a * a * -r).sum(0)
    dstate = s["dstate"].double()
    kept = torch.zeros_like(g) if s["resume"] is None else g * s["resume"].double()[index][:, None]
    dstate[slots[index]] = kept
    return {"y": y, "state": state, "dx": total * bb * i, "dga": d_r * r * (1.0 - r), "dgx": total * bb * x * i * (1.0 - i),
            "ddecay": d_speed * RATE / (1.0 + torch.exp(-decay)), "dstate": dstate}


def _exact_norm(case, s):
    """The gradients are those that differentiation of the definition gives."""
    shape = (case["tokens"], case["heads"], case["width"])
    o, z = s["block"].double().view(shape), s["gate"].double().view(shape)
    post = s["post"].double()
    backward, full = case["op"] == "norm_backward", s["residual"] is not None

    def normed(v, w):
        return v * w / torch.sqrt((v * v).sum(-1, keepdim=True) / shape[-1] + EPS)

    def gated(o, z, post):
        return normed(o, post) * (z if case["act"] == "silu" else 1.0) / (1.0 + torch.exp(-z))

    if not backward:
        p = gated(o, z, post)
        if not full:
            return {"t": p.reshape(s["t"].shape)}
        t = s["residual"].double().view(shape) + s["scale"].double() * p
        return {"t": t.reshape(s["t"].shape), "y": normed(t, s["pre"].double()).reshape(s["t"].shape)}
    leaves = [v.clone().requires_grad_(True) for v in (o, z, post)]
    g = s["dt"].double().view(shape)
    out = {}
    if full:
        t, pre = (s[n].double().clone().requires_grad_(True) for n in ("t", "pre"))
        normed(t, pre).backward(s["dy"].double())
        g = g + t.grad.view(shape)
        leaves.append(s["scale"].double().clone().requires_grad_(True))
        (leaves[3] * gated(*leaves[:3])).backward(g)
        out = {"dresidual": g.reshape(s["dt"].shape), "dscale": leaves[3].grad, "dpre": pre.grad}
    else:
        gated(*leaves).backward(g)
    return {"dblock": leaves[0].grad.reshape(s["dt"].shape), "dgate": leaves[1].grad.reshape(s["dt"].shape),
            "dpost": leaves[2].grad, **out}


def exact(case, seed):
    if case["op"] == "verify":
        return None                                           # whole numbers only
    s = prepare(case, seed)
    return _exact_scan(case, s) if case["op"] in SCAN_OPS else _exact_norm(case, s)
