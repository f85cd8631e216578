"""GPU tests of the gated delta rule's forward forms against the 64-bit token loop."""
import pytest
import torch

import gdn_reference as ref
import linear_attention_sequence_chunked_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = torch.float32


def prefill(x, cu, **kw):
    return kda.gdn_chunk_prefill(x["q"], x["k"], x["v"], x["la"], x["be"], cu_seqlens=cu,
                                 initial_state=x["s0"], **kw)


def check_prefill(x, cu, dtype, **kw):
    o, sf = prefill(x, cu, **kw)
    torch.cuda.synchronize()
    ro, rs = ref.forward(x["q"], x["k"], x["v"], x["la"], x["be"], cu, x["s0"], kw.get("scale", 1.0))
    ref.close("o", o, ro, dtype)
    ref.close("S", sf, rs, F32)
    return o, sf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_prefill_shapes(dtype, dk, dv):
    x, cu = ref.inputs([200, 1, 0, 65], 2, 4, dk, dv, DT[dtype], seed=dk + dv)
    check_prefill(x, cu, DT[dtype], scale=0.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 96, 127, 128, 129, 191, 193, 321])
def test_prefill_lengths(dtype, n):
    x, cu = ref.inputs([n], 1, 2, 128, 128, DT[dtype], seed=n, s0=n % 2 == 0)
    check_prefill(x, cu, DT[dtype])


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 7), (3, 3), (5, 10), (2, 64)])
def test_prefill_heads(hk, hv):
    x, cu = ref.inputs([70, 129], hk, hv, 128, 64, torch.bfloat16, seed=hk * hv)
    check_prefill(x, cu, torch.bfloat16)


def test_prefill_many_chains_full_width():
    """Enough chains that every workgroup takes the full width of the state."""
    x, cu = ref.inputs([130, 66, 3, 64], 16, 80, 128, 128, torch.bfloat16, seed=5)
    check_prefill(x, cu, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_more_sequences_than_one_launch(dtype):
    lens = [(7 * i) % 19 for i in range(300)]
    x, cu = ref.inputs(lens, 1, 2, 64, 64, DT[dtype], seed=9)
    check_prefill(x, cu, DT[dtype])


@pytest.mark.parametrize("dk,dv,n", [(64, 128, 70), (128, 64, 130), (128, 128, 70)])
def test_prefill_f32_of_many_states(dk, dv, n):
    """More states than one column per lane would fill the card with."""
    x, cu = ref.inputs([(11 * i) % 37 for i in range(n)], 1, 1, dk, dv, torch.float32, seed=n)
    check_prefill(x, cu, torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_all_empty(dtype):
    x, cu = ref.inputs([0, 0], 1, 2, 64, 64, DT[dtype], seed=3)
    o, sf = prefill(x, cu)
    assert o.shape == (0, 2, 64) and torch.equal(sf, x["s0"])
    x["s0"] = None
    assert not prefill(x, cu)[1].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["reset", "no_decay_same_key", "strong_decay", "no_write", "zero_keys"])
def test_prefill_gates(dtype, what):
    x, cu = ref.inputs([150, 33], 1, 2, 128, 128, DT[dtype], seed=21)
    if what == "reset":  # a log-decay of -inf forgets the state; a huge one too
        x["la"][40] = -float("inf")
        x["la"][90] = -1e30
        x["la"][91] = torch.finfo(F32).min
    elif what == "no_decay_same_key":  # the chunk's triangular system at its worst
        x["la"].zero_()
        x["be"].fill_(1.0)
        x["k"][:] = x["k"][:1]
    elif what == "strong_decay":
        x["la"].fill_(-20.0)
    elif what == "no_write":
        x["be"].zero_()
    else:
        x["k"].zero_()
    check_prefill(x, cu, DT[dtype])


@pytest.mark.parametrize("amp", [1e-3, 100.0])
def test_prefill_value_scale(amp):
    """The rule is linear in v and the state: small and large values keep the accuracy of the
    outputs.  (fp32 states of values below 1e-2 lose it gradually: halves of fp16 operands end
    at 2^-25, an eighth of that behind the prescale, so 2^-28 / 1e-3 = 4e-6 of v per product,
    times sqrt(128) of a sum: 4.2e-5.)"""
    x, cu = ref.inputs([140], 1, 2, 128, 128, torch.bfloat16, seed=4, amp=amp)
    o, sf = prefill(x, cu)
    ro, rs = ref.forward(x["q"], x["k"], x["v"], x["la"], x["be"], cu, x["s0"])
    ref.close("o", o, ro, torch.bfloat16)
    assert ref.rel(sf, rs) <= (ref.TOL_F32 if amp > 1 else ref.TOL_F32 + 4.2e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_nan_stays_in_its_sequence_and_head(dtype):
    x, cu = ref.inputs([80, 70], 2, 2, 64, 64, DT[dtype], seed=8)
    clean = prefill(x, cu)
    x["v"][20, 1] = float("nan")
    x["la"][100, 0] = float("nan")
    o, sf = prefill(x, cu)
    assert torch.equal(o[:80, 0], clean[0][:80, 0]) and torch.equal(o[80:, 1], clean[0][80:, 1])
    assert torch.isnan(o[20:80, 1]).all() and torch.isnan(o[100:, 0]).all()
    assert torch.isnan(sf[0, 1]).all() and torch.isnan(sf[1, 0]).all()
    assert torch.equal(sf[0, 0], clean[1][0, 0]) and torch.equal(sf[1, 1], clean[1][1, 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_strided_projection(dtype):
    """q, k and v as slices of one projection give the dense call's bits."""
    x, cu = ref.inputs([100, 29], 2, 4, 64, 128, DT[dtype], seed=2)
    T = cu[-1]
    w = torch.full((T, 2 * 2 * 64 + 4 * 128 + 64), float("nan"), dtype=DT[dtype], device="cuda")
    w[:, :128] = x["q"].reshape(T, -1)
    w[:, 128:256] = x["k"].reshape(T, -1)
    w[:, 256:768] = x["v"].reshape(T, -1)
    y = dict(x, q=w[:, :128].view(T, 2, 64), k=w[:, 128:256].view(T, 2, 64), v=w[:, 256:768].view(T, 4, 128))
    assert not y["v"].is_contiguous()
    a, b = prefill(x, cu), prefill(y, cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_writes_its_rows_alone_and_the_state_in_place(dtype):
    x, cu = ref.inputs([77, 0, 64], 2, 2, 128, 128, DT[dtype], seed=6)
    want = prefill(x, cu)
    T = cu[-1]
    buf = torch.full((T + 40, 2, 128), 7.0, dtype=DT[dtype], device="cuda")
    st = torch.full((5, 2, 128, 128), 7.0, device="cuda")
    st[1:4] = x["s0"]
    o, sf = kda.gdn_chunk_prefill(x["q"], x["k"], x["v"], x["la"], x["be"], cu_seqlens=cu,
                                  initial_state=st[1:4], final_state=st[1:4], out=buf[20:20 + T])
    assert torch.equal(o, want[0]) and torch.equal(sf, want[1])
    assert (buf[:20] == 7).all() and (buf[20 + T:] == 7).all() and (st[0] == 7).all() and (st[4] == 7).all()


def test_prefill_fixed_batch_and_split_resume():
    x, cu = ref.inputs([128, 128], 2, 2, 128, 128, torch.bfloat16, seed=12)
    want = prefill(x, cu)
    b = lambda t: t.view(2, 128, *t.shape[1:])  # noqa: E731
    o, sf = kda.gdn_chunk_prefill(b(x["q"]), b(x["k"]), b(x["v"]), b(x["la"]), b(x["be"]), initial_state=x["s0"])
    assert torch.equal(o.view_as(want[0]), want[0]) and torch.equal(sf, want[1])
    cut = lambda t, i: b(t)[:, 64 * i:64 * i + 64].contiguous()  # noqa: E731
    s = x["s0"]
    for i in range(2):
        o, s = kda.gdn_chunk_prefill(*(cut(x[n], i) for n in ("q", "k", "v", "la", "be")), initial_state=s)
        assert torch.equal(o, cut(want[0], i))
    assert torch.equal(s, want[1])


def test_prefill_same_bits_every_run_and_on_another_stream():
    x, cu = ref.inputs([300, 65, 700], 2, 4, 128, 128, torch.bfloat16, seed=13)
    want = prefill(x, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [prefill(x, cu) for _ in range(3)]
    side.synchronize()
    for o, s in got:
        assert torch.equal(o, want[0]) and torch.equal(s, want[1])


# ------------------------------------------------------------------------------ recurrent form

def step_inputs(N, K, hk, hv, dk, dv, dtype, seed, slots=None):
    x, _ = ref.inputs([K] * N, hk, hv, dk, dv, dtype, seed)
    y = {n: x[n].view(N, K, *x[n].shape[1:]) for n in ("q", "k", "v", "la", "be")}
    g = torch.Generator().manual_seed(seed + 1)
    y["state"] = (0.3 * torch.randn(slots or N, hv, dk, dv, generator=g)).cuda()
    return y


def call(y, state, **kw):
    return kda.gdn_recurrent(y["q"], y["k"], y["v"], y["la"], y["be"], state, **kw)


def loop(y, state, steps=None, scale=1.0):
    N, K = y["q"].shape[:2]
    flat = [y[n].reshape(N * K, *y[n].shape[2:]) for n in ("q", "k", "v", "la", "be")]
    cu = [K * i for i in range(N + 1)]
    o, sf = ref.forward(*flat, cu, state, scale)
    if steps is not None:
        sf = ref.f64(state).clone()
        for n, m in enumerate(steps):
            rows = [t[n * K:n * K + m] for t in flat]
            sf[n] = ref.forward(*rows, [0, m], state[n:n + 1], scale)[1][0]
    return o.view(N, K, *o.shape[1:]), sf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("K", [1, 3, 16])
def test_recurrent_shapes(dtype, dk, dv, K):
    y = step_inputs(3, K, 2, 4, dk, dv, DT[dtype], seed=dk + dv + K)
    s = y["state"].clone()
    o = call(y, s, scale=1.3)
    ro, rs = loop(y, y["state"], scale=1.3)
    ref.close("o", o, ro, DT[dtype])
    ref.close("S", s, rs, F32)


def test_recurrent_wide_batch():
    """Enough (sequence, head) pairs that a workgroup takes whole rows of the state."""
    y = step_inputs(40, 2, 8, 16, 128, 128, torch.bfloat16, seed=77)
    s = y["state"].clone()
    o = call(y, s)
    ro, rs = loop(y, y["state"])
    ref.close("o", o, ro, torch.bfloat16)
    ref.close("S", s, rs, F32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_recurrent_drafts_verify_then_commit(dtype):
    N, K = 9, 5
    y = step_inputs(N, K, 2, 2, 128, 128, DT[dtype], seed=31)
    s = y["state"].clone()
    steps = [0, 1, 2, 3, 4, 5, 9, -3, 2]  # clamped to [0, K]
    kept = [min(max(m, 0), K) for m in steps]
    dev = torch.tensor(steps, dtype=torch.int32, device="cuda")
    o = call(y, s, update_state=False)
    assert torch.equal(s, y["state"])
    both = call(y, s.clone(), steps=dev)
    assert torch.equal(both, o)
    assert call(y, s, steps=dev, output=False) is None
    ro, rs = loop(y, y["state"], kept)
    ref.close("o", o, ro, DT[dtype])
    ref.close("S", s, rs, F32)
    for n, m in enumerate(kept):
        if m == 0:
            assert torch.equal(s[n], y["state"][n])
    t = y["state"].clone()  # the same bits as one token after another
    for j in range(K):
        one = {n: y[n][:, j].contiguous() for n in ("q", "k", "v", "la", "be")}
        assert torch.equal(call(one, t), o[:, j])
    assert torch.equal(t[5], s[5])


def test_recurrent_slots_padding_and_repeats():
    N, slots = 7, 9
    y = step_inputs(N, 2, 1, 3, 64, 128, torch.bfloat16, seed=41, slots=slots)
    idx = torch.tensor([4, -1, 8, 4, 0, 9, 2], dtype=torch.int32, device="cuda")
    s = y["state"].clone()
    o = call(y, s, state_indices=idx)
    assert not o[[1, 3, 5]].any(), "padded rows, and a repeated slot's later rows, are zero"
    use = [0, 2, 4, 6]
    z = {n: y[n][use].contiguous() for n in ("q", "k", "v", "la", "be")}
    at = idx[use].long()
    ro, rs = loop(z, y["state"][at])
    ref.close("o", o[use], ro, torch.bfloat16)
    ref.close("S", s[at], rs, F32)
    rest = [i for i in range(slots) if i not in at.tolist()]
    assert torch.equal(s[rest], y["state"][rest])
    # where nothing is written every row reads its slot, repeated or not
    o = call(y, s.copy_(y["state"]), state_indices=idx, update_state=False)
    alone = {n: y[n][3:4].contiguous() for n in ("q", "k", "v", "la", "be")}
    assert torch.equal(o[3:4], call(alone, y["state"][4:5].clone()))
    assert not o[[1, 5]].any()


def test_recurrent_continues_the_prefill():
    x, cu = ref.inputs([90, 33], 2, 4, 128, 128, torch.bfloat16, seed=51, s0=False)
    first = [0, 89, 89 + 32]
    cut = {n: torch.cat([x[n][:89], x[n][90:122]]).contiguous() for n in ("q", "k", "v", "la", "be")}
    _, s = kda.gdn_chunk_prefill(cut["q"], cut["k"], cut["v"], cut["la"], cut["be"], cu_seqlens=first)
    one = {n: x[n][[89, 122]].contiguous() for n in ("q", "k", "v", "la", "be")}
    o = call(one, s)
    ro, rs = ref.forward(x["q"], x["k"], x["v"], x["la"], x["be"], cu)
    ref.close("o", o, ro[[89, 122]], torch.bfloat16)
    ref.close("S", s, rs, F32)


def test_recurrent_captured_and_replayed():
    y = step_inputs(4, 1, 2, 4, 128, 128, torch.bfloat16, seed=61, slots=6)
    idx = torch.tensor([5, 0, -1, 2], dtype=torch.int32, device="cuda")
    s, eager, out = y["state"].clone(), y["state"].clone(), torch.empty_like(y["v"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(y, s.clone(), state_indices=idx)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y, s, state_indices=idx, out=out)
    for i in range(4):
        y["v"].mul_(1.25)
        if i == 2:
            idx.copy_(torch.tensor([1, 0, 3, -1], dtype=torch.int32))
        g.replay()
        want = call(y, eager, state_indices=idx)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(s, eager)
