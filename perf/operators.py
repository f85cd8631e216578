"""Timed cases of the gated delta rule and of draft verification, with their plain forms.

The gated delta rule keeps, per value head, a state S of [dk, dv]; token t does
    S <- e^{g_t} S;   u = beta_t (v_t - S^T k_t);   S <- S + k_t u^T;   o_t = scale S^T q_t
with ONE log-decay g_t per token and value head, and query and key heads shared by groups of
value heads.  Its forms: the chunked prefill over packed sequences, the same with its
gradients, and the recurrent step over one or a few tokens with the state updated in place.

Draft verification takes the target's and the draft's probabilities, the drafted tokens and
uniform random numbers: draft j is kept while u_j q_j(x_j) < p_j(x_j); the token after the
kept ones is drawn from max(p - q, 0) at the first rejected place, or from p after the last.

`own` is false: the plain forms, in elementary torch operations.  True: the package's calls.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
C = 64  # tokens per chunk of the plain chunked form


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one short prompt of a small model: latency of a single prefill call
        dict(name="prefill_short", op="prefill", dtype=BF16, lens="17", hk=2, hv=4, dk=64, dv=64, s0=False),
        # a training or serving batch of equal lengths, states carried in and out
        dict(name="prefill_b4_h16_t4096", op="prefill", dtype=BF16, lens="4096,4096,4096,4096", hk=16, hv=16, dk=128, dv=128, s0=True),
        # a packed serving batch of ragged prompts, an empty one among them, keys shared by 4 value heads
        dict(name="prefill_ragged_grouped", op="prefill", dtype=BF16,
             lens="1,511,2049,0,63,1000,4097,129,3333,64,777,15,2500,1291,65,3001,190,2222,1,640,4000,333,1777", hk=8, hv=32, dk=128, dv=128, s0=True),
        # one long document: few chains, many chunks
        dict(name="prefill_b1_h32_t131072", op="prefill", dtype=BF16, lens="131072", hk=16, hv=32, dk=128, dv=128, s0=False),
        # 32-bit inputs, ragged, dk != dv
        dict(name="prefill_f32", op="prefill", dtype=F32, lens="1000,1,333,2050", hk=4, hv=4, dk=64, dv=128, s0=True),
        # one user's next token
        dict(name="step_n1", op="step", dtype=BF16, n=1, k=1, pool=1, hk=16, hv=32, dk=128, dv=128, mode="decode"),
        # a full decode batch whose states lie in a pool under slot numbers
        dict(name="step_n256_h32", op="step", dtype=BF16, n=256, k=1, pool=288, hk=16, hv=32, dk=128, dv=128, mode="decode"),
        # speculative decoding: outputs of 4 drafts from the stored state, then the kept ones written
        dict(name="step_verify_commit", op="step", dtype=BF16, n=96, k=4, pool=96, hk=32, hv=32, dk=128, dv=128, mode="drafts"),
        # a small ragged training batch with shared keys
        dict(name="backward_ragged", op="backward", dtype=BF16, lens="300,1,64,517", hk=2, hv=4, dk=64, dv=128, s0=True),
        # the training batch
        dict(name="backward_b4_h16_t4096", op="backward", dtype=BF16, lens="4096,4096,4096,4096", hk=16, hv=16, dk=128, dv=128, s0=True),
        # verification for one user, and for a batch with a large odd vocabulary
        dict(name="accept_n1", op="accept", dtype=F32, n=1, k=4, vocab=32000, onehot=False, ragged=False),
        dict(name="accept_n128", op="accept", dtype=F32, n=128, k=8, vocab=151669, onehot=False, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; no dearer than the largest listed."""
    op = rng.choice(["prefill", "prefill", "step", "backward", "accept"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    if op == "accept":
        return dict(op=op, dtype=rng.choice([F32, F32, BF16]), n=_log(rng, 1, 128), k=rng.randint(1, 8),
                    vocab=_log(rng, 500, 151669), onehot=rng.random() < 0.25, ragged=rng.random() < 0.5)
    hk = _log(rng, 1, 16)
    heads = dict(hk=hk, hv=hk * rng.choice([1, 1, 2, 3, 4]), dk=rng.choice([64, 128]), dv=rng.choice([64, 128]))
    if op == "step":
        n = _log(rng, 1, 256)
        mode = rng.choice(["decode", "drafts"])
        return dict(op=op, dtype=dtype, n=n, k=1 if mode == "decode" else rng.randint(2, 16), pool=n + rng.randint(0, 9), mode=mode, **heads)
    # prefill and backward: ragged lengths around a mean, total tokens x heads bounded
    most = (1 << 20 if op == "prefill" else 1 << 17) // heads["hv"]
    if dtype == F32:
        most = min(most, 1 << 13)
    total, seqs = _log(rng, 40, max(64, most)), _log(rng, 1, 32)
    mean = max(1, total // seqs)
    lens = [max(0, min(2 * mean, int(mean * rng.uniform(0, 2)))) for _ in range(seqs)]
    lens[0] = max(1, lens[0])
    return dict(op=op, dtype=dtype, lens=",".join(map(str, lens)), s0=rng.random() < 0.6, **heads)


# ------------------------------------------------------------------------------ the inputs

def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)


def _unit(shape, g, dt):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dt)


def _gates(shape, g):
    """log-decay and write strength as a model forms them: g = -A softplus(x + b), A per head
    in [1, 16], softplus(b) in [1e-3, 1e-1] per head; beta = sigmoid(x)."""
    hv = shape[-1]
    a = 1 + 15 * torch.rand(hv, generator=g, device="cuda")
    dt = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(hv, generator=g, device="cuda"))
    x = torch.randn(shape, generator=g, device="cuda") + torch.log(torch.expm1(dt))
    la = -a * torch.nn.functional.softplus(x)
    return la, torch.sigmoid(torch.randn(shape, generator=g, device="cuda"))


def prepare(case, seed):
    g, dt = _gen(case, seed), TYPES[case["dtype"]]
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "accept":
        n, k, vocab = case["n"], case["k"], case["vocab"]
        z = 2.5 * randn(n, k + 1, vocab)
        p = torch.softmax(z, -1).to(dt)
        if case["onehot"]:  # a draft without probabilities: the likeliest token, or some other one
            x = torch.where(torch.rand((n, k), generator=g, device="cuda") < 0.6, z[:, :k].argmax(-1),
                            torch.randint(vocab, (n, k), generator=g, device="cuda"))
            q = None
        else:
            q = torch.softmax(z[:, :k] + 0.5 * randn(n, k, vocab), -1).to(dt)
            at = torch.rand((n, k, 1), generator=g, device="cuda", dtype=torch.float64)
            c = q.double().cumsum(-1)
            x = (c <= at * c[..., -1:]).sum(-1).clamp_max(vocab - 1)
        counts = torch.randint(0, k + 1, (n,), generator=g, device="cuda").int() if case["ragged"] else None
        return dict(case=case, p=p, q=q, x=x.int(), u=torch.rand((n, k + 1), generator=g, device="cuda"), counts=counts)
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    if case["op"] == "step":
        n, k = case["n"], case["k"]
        la, be = _gates((n, k, hv), g)
        slots = torch.randperm(case["pool"], generator=g, device="cuda")[:n].int()
        return dict(case=case, q=_unit((n, k, hk, dk), g, dt), k=_unit((n, k, hk, dk), g, dt), v=randn(n, k, hv, dv).to(dt), la=la, be=be,
                    pool=0.05 * randn(case["pool"], hv, dk, dv), slots=slots,
                    kept=torch.randint(0, k + 1, (n,), generator=g, device="cuda").int())
    lens = [int(x) for x in case["lens"].split(",")]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    t, n = cu[-1], len(lens)
    la, be = _gates((t, hv), g)
    s = dict(case=case, q=_unit((t, hk, dk), g, dt), k=_unit((t, hk, dk), g, dt), v=randn(t, hv, dv).to(dt), la=la, be=be,
             cu=cu, cu_dev=torch.tensor(cu, device="cuda"), s0=0.02 * randn(n, hv, dk, dv) if case["s0"] else None)
    if case["op"] == "backward":
        s["do"], s["dsf"] = randn(t, hv, dv).to(dt), 0.1 * randn(n, hv, dk, dv)
    return s


# ------------------------------------------------------------------------------ the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"prefill": _own_prefill, "step": _own_step, "backward": _own_backward, "accept": _own_accept}[op](state)
    return {"prefill": _prefill, "step": _step, "backward": _backward, "accept": _accept}[op](state)


def _own_prefill(s):
    import linear_attention_sequence_chunked_amd as kda
    return kda.gdn_chunk_prefill(s["q"], s["k"], s["v"], s["la"], s["be"], cu_seqlens=s["cu"], initial_state=s["s0"])


def _own_step(s):
    import linear_attention_sequence_chunked_amd as kda
    x = (s["q"], s["k"], s["v"], s["la"], s["be"], s["pool"])
    if s["case"]["mode"] == "decode":
        return kda.gdn_recurrent(*x, state_indices=s["slots"]), s["pool"]
    o = kda.gdn_recurrent(*x, state_indices=s["slots"], update_state=False)
    kda.gdn_recurrent(*x, state_indices=s["slots"], steps=s["kept"], output=False)
    return o, s["pool"]


def _own_backward(s):
    import linear_attention_sequence_chunked_amd as kda
    return kda.gdn_prefill_backward(s["q"], s["k"], s["v"], s["la"], s["be"], s["do"], cu_seqlens=s["cu"], initial_state=s["s0"], d_final_state=s["dsf"])


def _own_accept(s):
    import linear_attention_sequence_chunked_amd as kda
    return kda.spec_accept(s["p"], s["q"], s["x"], s["u"], num_drafts=s["counts"])


# ------------------------------------------------------------------------------ the plain forms

def _inverse(a):
    """(I + a)^-1 of strictly lower triangular blocks, joined from their halves' inverses."""
    n = a.shape[-1]
    if n == 1:
        return torch.ones_like(a)
    h = n // 2
    t = _inverse(torch.stack([a[..., :h, :h], a[..., h:, h:]], -3))
    t0, t1 = t[..., 0, :, :], t[..., 1, :, :]
    low = -t1 @ (a[..., h:, :h] @ t0)
    return torch.cat([torch.cat([t0, torch.zeros_like(t0)], -1), torch.cat([low, t1], -1)], -2)


def _chunked(q, k, v, la, be, s, scale=1.0):
    """The rule over [n, t, heads, *] inputs in 32 bits, t a multiple of C; rows past a
    sequence's end have k = 0, beta = 0 and no decay.  Sums of log-decays are in 64 bits."""
    n, t, h, _ = v.shape
    cut = lambda x: x.reshape(n, t // C, C, h, -1).transpose(2, 3)  # noqa: E731  [n, chunk, h, C, *]
    q, k, v, be = cut(q) * scale, cut(k), cut(v), cut(be[..., None])
    g = cut(la[..., None]).double().cumsum(-2)
    e, last = torch.exp(g).float(), torch.exp(g[..., -1:, :]).float()
    rest = torch.exp(g[..., -1:, :] - g).float()
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    d = torch.exp((g - g.transpose(-1, -2)).masked_fill(~low, -math.inf)).float()
    inv = _inverse((be * d * (k @ k.transpose(-1, -2))).tril(-1))
    w, u0 = inv @ (be * e * k), inv @ (be * v)
    p, qe, kr = d * (q @ k.transpose(-1, -2)), e * q, (rest * k).transpose(-1, -2)
    out = []
    for c in range(t // C):
        u = u0[:, c] - w[:, c] @ s
        out.append(qe[:, c] @ s + p[:, c] @ u)
        s = last[:, c] * s + kr[:, c] @ u
    return torch.stack(out, 1).transpose(2, 3).reshape(n, t, h, -1), s


def _padded(s, names):
    """Packed rows laid out as [n, t, *], zeros past each end; and the index that takes them back."""
    lens = s["cu_dev"][1:] - s["cu_dev"][:-1]
    t = max(b - a for a, b in zip(s["cu"], s["cu"][1:]))
    t = max(C, -(-t // C) * C)
    at = torch.arange(t, device="cuda")
    inside = at < lens[:, None]
    idx = (s["cu_dev"][:-1, None] + at).clamp_max(s["cu"][-1] - 1)
    back = inside.reshape(-1).nonzero()[:, 0]
    take = lambda x: x.float()[idx] * inside.reshape(inside.shape + (1,) * (x.dim() - 1))  # noqa: E731
    return [take(s[n]) for n in names], back


def _heads(x, s):
    """Query and key heads repeated for the value heads that share them."""
    return x.repeat_interleave(s["case"]["hv"] // s["case"]["hk"], dim=-2)


def _start(s):
    c = s["case"]
    return s["s0"].float() if s["s0"] is not None else torch.zeros(len(s["cu"]) - 1, c["hv"], c["dk"], c["dv"], device="cuda")


def _prefill(s):
    (q, k, v, la, be), back = _padded(s, ("q", "k", "v", "la", "be"))
    o, sf = _chunked(_heads(q, s), _heads(k, s), v, la, be, _start(s))
    return o.flatten(0, 1)[back].to(s["v"].dtype), sf


def _backward(s):
    names = ("q", "k", "v", "la", "be")
    leaves = {n: s[n].float().requires_grad_() for n in names}
    s0 = _start(s).clone().requires_grad_()
    with torch.enable_grad():
        (q, k, v, la, be), back = _padded({**s, **leaves}, names)
        o, sf = _chunked(_heads(q, s), _heads(k, s), v, la, be, s0)
        got = torch.autograd.grad([o.flatten(0, 1)[back], sf], [leaves[n] for n in names] + [s0], [s["do"].float(), s["dsf"]])
    got = [x.to(s[n].dtype) for x, n in zip(got, names)] + [got[-1]]
    return dict(zip(("dq", "dk", "dv", "dlog_alpha", "dbeta", "d_initial_state"), got))


def _step(s):
    """All tokens as one chunk, with the state taken from and written back to its slot; of
    drafts, the kept ones alone write (the others' keys and decays are zero for the state)."""
    n, k = s["case"]["n"], s["case"]["k"]
    pad = lambda x: torch.nn.functional.pad(x.float(), (0, 0) * (x.dim() - 2) + (0, C - k))  # noqa: E731
    q, kk, v, la, be = (pad(s[x]) for x in ("q", "k", "v", "la", "be"))
    q, kk, slots = _heads(q, s), _heads(kk, s), s["slots"].long()
    o, new = _chunked(q, kk, v, la, be, s["pool"][slots])
    if s["case"]["mode"] == "drafts":
        keep = (torch.arange(C, device="cuda") < s["kept"][:, None])[..., None]
        new = _chunked(q, kk * keep[..., None], v, la * keep, be * keep, s["pool"][slots])[1]
    s["pool"][slots] = new
    return o[:, :k].to(s["v"].dtype), s["pool"]


def _accept(s):
    """Products, differences and sums over the vocabulary in 64 bits: a draw lies next to a border."""
    p, q, u, k = s["p"], s["q"], s["u"].double(), s["case"]["k"]
    n, x = p.shape[0], s["x"].long()
    rows, at = torch.arange(n, device="cuda"), torch.arange(k + 1, device="cuda")
    counts = s["counts"].long() if s["counts"] is not None else torch.full((n,), k, device="cuda")
    px = p[:, :k].gather(-1, x[..., None])[..., 0].double()
    qx = q.gather(-1, x[..., None])[..., 0].double() if q is not None else torch.ones_like(px)
    keep = (u[:, :k] * qx < px) & (at[:k] < counts[:, None])
    kept = keep.long().cumprod(-1).sum(-1)
    full = p[rows, kept].double()
    if q is None:
        minus = torch.zeros_like(full)
        minus[rows, x[rows, kept.clamp_max(k - 1)]] = math.inf
    else:
        minus = q[rows, kept.clamp_max(k - 1)].double()
    left = torch.where((kept < counts)[:, None], (full - minus).clamp_min(0), full)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, full)
    c = left.cumsum(-1)
    drawn = (c <= u[:, k:] * c[:, -1:]).sum(-1)
    tokens = torch.cat([x, x[:, :1]], -1).masked_fill(at >= kept[:, None], -1)
    tokens[rows, kept] = drawn
    return kept.int(), tokens.int()


# ------------------------------------------------------------------------------ 64 bits, apart

def exact(case, seed):
    """The recurrence itself, token by token in 64 bits, and its reverse."""
    if case["op"] == "accept":
        return None  # whole numbers: compared as they are
    s = prepare(case, seed)
    r = case["hv"] // case["hk"]
    f = lambda x: x.double()  # noqa: E731
    if case["op"] == "step":
        q, k = (f(s[x]).repeat_interleave(r, 2) for x in ("q", "k"))
        v, la, be, pool = f(s["v"]), f(s["la"]), f(s["be"]), f(s["pool"])
        st = pool[s["slots"].long()]
        history, out = [st], []
        for t in range(case["k"]):
            st = st * torch.exp(la[:, t])[..., None, None]
            w = (st * k[:, t, :, :, None]).sum(-2)
            st = st + k[:, t, :, :, None] * (be[:, t, :, None] * (v[:, t] - w))[:, :, None]
            out.append((st * q[:, t, :, :, None]).sum(-2))
            history.append(st)
        kept = s["kept"].long() if case["mode"] == "drafts" else torch.full((case["n"],), case["k"], device="cuda")
        pool[s["slots"].long()] = torch.stack(history, 1)[torch.arange(case["n"], device="cuda"), kept]
        return torch.stack(out, 1), pool
    lens = [b - a for a, b in zip(s["cu"], s["cu"][1:])]
    longest, n, t_all = max(lens), len(lens), s["cu"][-1]
    hv, dk, dv = case["hv"], case["dk"], case["dv"]
    if case["op"] == "backward" and 8 * t_all * hv * dk * dv > 60e9:
        return None
    st = f(s["s0"]) if s["s0"] is not None else torch.zeros(n, hv, dk, dv, device="cuda", dtype=torch.float64)
    o = torch.zeros(t_all, hv, dv, device="cuda", dtype=torch.float64)
    before, active = [], []
    order = sorted(range(n), key=lambda i: -lens[i])  # the longest first: the running ones lead
    st = st[torch.tensor(order, device="cuda")]
    starts = torch.tensor([s["cu"][i] for i in order], device="cuda")
    rows_of = lambda m, t: starts[:m] + t  # noqa: E731
    running = [sum(x > t for x in lens) for t in range(longest)]
    vec = lambda x, rows: f(x[rows]).repeat_interleave(r, 1)  # noqa: E731
    for t in range(longest):
        m = running[t]
        rows = rows_of(m, t)
        q, k, v = vec(s["q"], rows), vec(s["k"], rows), f(s["v"][rows])
        if case["op"] == "backward":
            before.append(st[:m].clone())
        a = st[:m] * torch.exp(f(s["la"][rows]))[..., None, None]
        w = (k[:, :, None] @ a)[:, :, 0]
        a += k[..., None] * (f(s["be"][rows])[..., None] * (v - w))[:, :, None]
        st[:m] = a
        o[rows] = (q[:, :, None] @ a)[:, :, 0]
    sf = torch.empty_like(st)
    sf[torch.tensor(order, device="cuda")] = st
    if case["op"] == "prefill":
        return o, sf
    ds = f(s["dsf"])[torch.tensor(order, device="cuda")]
    dq, dk_ = (torch.zeros(t_all, hv, dk, device="cuda", dtype=torch.float64) for _ in range(2))
    dv_ = torch.zeros_like(o)
    dla, dbe = (torch.zeros(t_all, hv, device="cuda", dtype=torch.float64) for _ in range(2))
    for t in reversed(range(longest)):
        m = running[t]
        rows = rows_of(m, t)
        q, k, v = vec(s["q"], rows), vec(s["k"], rows), f(s["v"][rows])
        do, b, al = f(s["do"][rows]), f(s["be"][rows])[..., None], torch.exp(f(s["la"][rows]))[..., None, None]
        a = before.pop() * al  # the decayed state
        err = v - (k[:, :, None] @ a)[:, :, 0]
        u = b * err
        new = a + k[..., None] * u[:, :, None]
        d = ds[:m] + q[..., None] * do[:, :, None]
        dq[rows] = (new @ do[..., None])[..., 0]
        du = (k[:, :, None] @ d)[:, :, 0]
        dk_[rows] = (d @ u[..., None])[..., 0] - (a @ (b * du)[..., None])[..., 0]
        dbe[rows] = (du * err).sum(-1)
        dv_[rows] = b * du
        d = d - k[..., None] * (b * du)[:, :, None]
        dla[rows] = (d * a).sum((-1, -2))
        ds[:m] = d * al
    ds0 = torch.empty_like(ds)
    ds0[torch.tensor(order, device="cuda")] = ds
    shared = lambda x: x.reshape(t_all, case["hk"], r, dk).sum(2)  # noqa: E731
    return dict(dq=shared(dq), dk=shared(dk_), dv=dv_, dlog_alpha=dla, dbeta=dbe, d_initial_state=ds0)


# ------------------------------------------------------------------------------ what it cannot do without

def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "accept":  # the target's row of the drawn token, the draft's where one was rejected
        rows = case["n"] * (1 if case["onehot"] else 1 + (0.5 if case["ragged"] else 0.8))
        return {"bytes": rows * case["vocab"] * es + 16 * case["n"] * (case["k"] + 1), "flops": 3 * rows * case["vocab"]}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    row = 2 * hk * dk * es + 2 * hv * dv * es + 8 * hv  # q, k, v, o, log-decay, beta
    mac = 2 * hv * dk * dv  # one product with the state
    if case["op"] == "step":
        t, moved = case["n"] * case["k"], 2 * case["n"]
        if case["mode"] == "drafts":  # read for the outputs, read and written for the kept ones (all but those that keep none)
            moved = case["n"] * (1 + 2 * case["k"] / (case["k"] + 1))
        return {"bytes": t * row + moved * hv * dk * dv * 4, "flops": 3 * mac * t}
    lens = [int(x) for x in case["lens"].split(",")]
    t, st = sum(lens), len(lens) * hv * dk * dv * 4
    if case["op"] == "prefill":
        return {"bytes": t * row + st * (2 if case["s0"] else 1), "flops": 3 * mac * t}
    # q, k, v, d_out, gates in; dq, dk, dv and the gates' gradients out; the states' gradients
    return {"bytes": t * (4 * hk * dk * es + 3 * hv * dv * es + 16 * hv) + st * (3 if case["s0"] else 2), "flops": 8 * mac * t}
