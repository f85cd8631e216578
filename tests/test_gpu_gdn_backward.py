"""GPU tests of the gated delta rule's gradients against the 64-bit reverse token loop and
against differences of the forward."""
import pytest
import torch

import gdn_reference as ref
import linear_attention_sequence_chunked_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = torch.float32
NAMES = ("dq", "dk", "dv", "dlog_alpha", "dbeta", "d_initial_state")

# fp32 gradients pass through two chains of the forward's kind (the states, and their
# gradients, whose operands are bf16 pairs: 2^-16 a side): five products in a row with sums that
# grow a term's error by up to sqrt(128): 5 * 2 * 11 * 2^-22 with exact operands, and
# 3 * 11 * 2^-16 * 2^-2 (the rounding of a pair is uniform below its bound, a quarter of it in
# the mean square) with pairs: 1.3e-4 is their bound; what a chain measures is far below.
TOL_GRAD = 1.3e-4
TOL_GRAD_BF16 = 2.0 ** -8 + TOL_GRAD


def run(x, cu, do, dsf, **kw):
    return kda.gdn_prefill_backward(x["q"], x["k"], x["v"], x["la"], x["be"], do, cu_seqlens=cu, initial_state=x["s0"],
                                    d_final_state=dsf, **kw)


def upstream(x, cu, dtype, seed, final=True, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    hv, dk, dv = x["v"].shape[1], x["k"].shape[2], x["v"].shape[2]
    do = (amp * torch.randn(cu[-1], hv, dv, generator=g)).to(dtype).cuda()
    return do, (amp * torch.randn(len(cu) - 1, hv, dk, dv, generator=g)).cuda() if final else None


def check(x, cu, dtype, seed=1, final=True, amp=1.0, scale=1.0):
    do, dsf = upstream(x, cu, dtype, seed, final, amp)
    got = run(x, cu, do, dsf, scale=scale)
    torch.cuda.synchronize()
    want = ref.backward(x["q"], x["k"], x["v"], x["la"], x["be"], cu, x["s0"], do, dsf, scale)
    for n in NAMES:
        assert torch.isfinite(got[n]).all(), n
        e, low = ref.rel(got[n], want[n]), got[n].dtype == torch.bfloat16
        print(f"  {n}: {e:.2e}", flush=True)
        assert got[n].shape == want[n].shape
        assert e <= (TOL_GRAD_BF16 if low else TOL_GRAD), f"{n}: {e:.3e}"
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_backward_shapes(dtype, dk, dv):
    x, cu = ref.inputs([140, 1, 0, 65], 2, 4, dk, dv, DT[dtype], seed=dk + dv)
    check(x, cu, DT[dtype], scale=0.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200])
def test_backward_lengths(dtype, n):
    x, cu = ref.inputs([n], 1, 1, 128, 128, DT[dtype], seed=n, s0=n % 2 == 0)
    check(x, cu, DT[dtype], final=n % 3 == 0)


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 5), (3, 3), (2, 8), (3, 6)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_heads(dtype, hk, hv):
    x, cu = ref.inputs([70, 33], hk, hv, 64, 64, DT[dtype], seed=hk * hv)
    check(x, cu, DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_many_sequences(dtype):
    lens = [(5 * i) % 17 for i in range(270)]
    x, cu = ref.inputs(lens, 1, 2, 64, 64, DT[dtype], seed=9)
    check(x, cu, DT[dtype])


@pytest.mark.parametrize("dk,dv,n", [(64, 128, 132), (128, 64, 260), (128, 128, 132)])
def test_backward_f32_of_many_states(dk, dv, n):
    """More states than slices of them would fill the card with."""
    x, cu = ref.inputs([(7 * i) % 19 for i in range(n)], 1, 1, dk, dv, F32, seed=n)
    check(x, cu, F32)


def test_backward_one_long_sequence_among_short_ones():
    """Lengths so far apart that the chunks' gradients take several launches."""
    x, cu = ref.inputs([3] * 150 + [700, 0] + [2] * 100 + [65], 1, 16, 64, 64, torch.bfloat16, seed=10)
    check(x, cu, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_all_empty(dtype):
    x, cu = ref.inputs([0, 0], 1, 2, 64, 64, DT[dtype], seed=3)
    do, dsf = upstream(x, cu, DT[dtype], 1)
    g = run(x, cu, do, dsf)
    assert torch.equal(g["d_initial_state"], dsf) and g["dq"].numel() == 0
    assert not run(x, cu, do, None)["d_initial_state"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["reset", "same_key", "strong_decay", "no_write"])
def test_backward_gates(dtype, what):
    x, cu = ref.inputs([130, 40], 1, 2, 128, 128, DT[dtype], seed=21)
    if what == "reset":
        x["la"][40] = -float("inf")
        x["la"][90] = -1e30
        # the oracle's 0 * inf: a forgotten state passes no gradient, which its product says too
    elif what == "same_key":
        x["la"].fill_(-0.01)
        x["k"][:] = x["k"][:1]
    elif what == "strong_decay":
        x["la"].fill_(-20.0)
    else:
        x["be"].zero_()
    check(x, cu, DT[dtype])


@pytest.mark.parametrize("amp", [1e-7, 1e4])
def test_backward_gradient_scale(amp):
    """Gradients come at any scale (means over many tokens): the results scale with them."""
    x, cu = ref.inputs([140], 1, 2, 128, 128, torch.bfloat16, seed=4)
    check(x, cu, torch.bfloat16, amp=amp)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_strided_inputs_and_given_workspace(dtype):
    x, cu = ref.inputs([100, 29], 2, 4, 64, 128, DT[dtype], seed=2)
    do, dsf = upstream(x, cu, DT[dtype], 3)
    T = cu[-1]
    w = torch.full((T, 2 * 2 * 64 + 4 * 128 + 64), float("nan"), dtype=DT[dtype], device="cuda")
    w[:, :128], w[:, 128:256], w[:, 256:768] = x["q"].reshape(T, -1), x["k"].reshape(T, -1), x["v"].reshape(T, -1)
    y = dict(x, q=w[:, :128].view(T, 2, 64), k=w[:, 128:256].view(T, 2, 64), v=w[:, 256:768].view(T, 4, 128))
    a = run(x, cu, do, dsf)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    for got in (run(y, cu, do, dsf), run(x, cu, do, dsf, workspace=ws), run(x, cu, do, dsf, workspace=ws)):
        for n in NAMES:
            assert torch.equal(a[n], got[n]), n
    with pytest.raises(kda.KdaError, match="workspace_bytes"):
        run(x, cu, do, dsf, workspace=ws[:4096])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_captured_beside_an_eager_graph(dtype):
    """Captured and replayed with new inputs while an autograd graph of the same leaves lives."""
    x, cu = ref.inputs([90, 40], 1, 2, 64, 64, DT[dtype], seed=7)
    do, dsf = upstream(x, cu, DT[dtype], 3)
    leaf = x["v"].clone().float().requires_grad_()
    alive = (leaf * 2).sum()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(x, cu, do, dsf)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(x, cu, do, dsf)
    for i in range(4):
        x["v"].copy_(torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(i)).to(DT[dtype]))
        g.replay()
        want = run(x, cu, do, dsf)
        torch.cuda.synchronize()
        for n in NAMES:
            assert torch.equal(got[n], want[n]), n
    alive.backward()
    assert (leaf.grad == 2).all()


def test_backward_against_differences():
    """Central differences of the 32-bit forward along random directions of every input."""
    x, cu = ref.inputs([37, 18], 1, 2, 64, 64, F32, seed=12)
    do, dsf = upstream(x, cu, F32, 5)
    got = run(x, cu, do, dsf)
    pairs = dict(q="dq", k="dk", v="dv", la="dlog_alpha", be="dbeta", s0="d_initial_state")

    def loss(y):
        o, s = kda.gdn_chunk_prefill(y["q"], y["k"], y["v"], y["la"], y["be"], cu_seqlens=cu, initial_state=y["s0"])
        return (o.double() * do.double()).sum().item() + (s.double() * dsf.double()).sum().item()

    for n, gn in pairs.items():
        # towards the gradient itself: the derivative is its norm, the largest there is
        d = got[gn] / got[gn].double().norm().float()
        h = 1e-2
        num = (loss(dict(x, **{n: x[n] + h * d})) - loss(dict(x, **{n: x[n] - h * d}))) / (2 * h)
        want = (got[gn].double() * d.double()).sum().item()
        # truncation h^2 times a third derivative of the loss's own size, and the forward's
        # rounding 2^-24 of terms of size ||do|| ||o|| over 2h: both below 1e-3 of the norm here
        assert abs(num - want) <= 2e-3 * abs(want), (n, num, want)
