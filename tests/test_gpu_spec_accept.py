"""GPU tests of draft verification against the plain 64-bit form: equal, not near."""
import pytest
import torch

import gdn_reference as ref
import kda_inputs as ki
import linear_attention_sequence_chunked_amd as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def case(N, K, V, dtype, seed, near=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    z = 2 * r(N, K + 1, V)
    p = torch.softmax(z, -1).to(DT[dtype])
    q = torch.softmax(z[:, :K] + near * r(N, K, V), -1).to(DT[dtype])
    x = torch.multinomial(q.float().reshape(-1, V).clamp_min(1e-9), 1, generator=g).view(N, K).int() if K else torch.zeros(N, 0).int()
    u = torch.rand(N, K + 1, generator=g)
    return [t.cuda() for t in (p, q, x, u)]


def check(p, q, x, u, counts=None):
    a, t = kda.spec_accept(p, q, x, u, num_drafts=counts)
    ra, rt = ref.accept(p, q, x, u, counts)
    assert a.cpu().numpy().tolist() == ra.tolist()
    assert t.cpu().numpy().tolist() == rt.tolist()
    return a, t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,V", [(1, 1, 1), (1, 0, 5), (3, 1, 2), (5, 4, 63), (4, 4, 257), (2, 64, 300), (1, 3, 2049),
                                   (3, 8, 32001), (40, 3, 4999), (2, 2, 151669)])
def test_accept_sizes(dtype, N, K, V):
    check(*case(N, K, V, dtype, seed=N + K + V))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [7, 8, 9, 15, 511, 4095, 4096, 4100, 8193, 16385, 32767, 32768, 32769])
def test_accept_vocabularies_around_one_workgroups(V, dtype):
    """Rows of one round and several, up to the registers of one workgroup and past them."""
    check(*case(7, 3, V, dtype, seed=V))


@pytest.mark.parametrize("V", [9, 4099, 32768, 40000])
def test_accept_draws_at_the_ends(V):
    """The draw's border below the first entry and above the last, rows with a single entry."""
    p, q, x, u = case(12, 1, V, "f32", seed=V + 1)
    u[:, 0] = 0.999
    q[:, 0] = 0.0
    q.scatter_(2, x[:, :, None].long(), 1e6)  # the draft is rejected, its own entry weighs nothing
    u[:4, 1], u[4:8, 1], u[8:, 1] = 0.0, 1.0 - 2.0 ** -24, 0.5
    for n in range(8, 12):
        p[n] = 0.0
        p[n, 0, [0, V - 1, V // 2, (V - 1) // 64 * 64][n - 8]] = 0.25
    check(p, q, x, u)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accept_ragged_counts(dtype):
    p, q, x, u = case(12, 5, 1003, dtype, seed=2)
    counts = torch.tensor([0, 1, 2, 3, 4, 5, 0, -2, 9, 5, 1, 2], dtype=torch.int32, device="cuda")
    u[:, :5] *= 0.3  # most drafts are kept
    a, t = check(p, q, x, u, counts)
    assert (a <= counts.clamp(0, 5)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accept_certain_drafts(dtype):
    p, _, x, u = case(16, 4, 777, dtype, seed=3)
    x[::2] = p[::2, :4].float().argmax(-1).int()
    u[:, :4] *= 0.02
    a, t = check(p, None, x, u)
    for n, j in enumerate(a.tolist()):
        assert j == 4 or t[n, j] != x[n, j], "the rejected token is never drawn"


def test_accept_borders():
    """Products at the border, zero rows, tokens outside, uniforms at their ends."""
    V = 8
    p = torch.zeros(9, 2, V)
    q = torch.full((9, 1, V), 1 / V)
    x = torch.zeros(9, 1).int()
    u = torch.full((9, 2), 0.5)
    p[0, 0, 0] = 1 / 16          # u q = p: not below, rejected; nothing is left of p - q: draw from p
    p[1, 0, 0] = 1 / 8           # u q < p: kept; row 1 has no weight: -1
    p[2, 0] = 1 / V
    x[2] = V                     # outside: rejected
    p[3, 0] = 1 / V
    x[3] = -1
    p[4, 0, 3:5] = 0.5
    u[4, 1] = 0.0                # the first entry with weight
    p[5, 0, 3:5] = 0.5
    u[5, 1] = 1.0                # no sum exceeds the total: the last entry with weight
    p[6, 0] = float("nan")       # weighs nothing, keeps nothing
    p[7, 0, 5] = -1.0
    p[7, 0, 6] = 0.25
    q[8] = 0.0                   # 0 < p keeps
    p[8, 0, 0] = 1e-30
    p[8, 1, 7] = 1e-30
    a, t = check(p.cuda(), q.cuda(), x.cuda(), u.cuda())
    assert t[0].tolist() == [0, -1] and t[1].tolist() == [0, -1] and t[4, 0] == 3 and t[5, 0] == 4
    assert t[6].tolist() == [-1, -1] and t[7, 0] == 6 and t[8].tolist() == [0, 7]


def test_accept_same_distribution_keeps_everything():
    p, _, x, u = case(8, 6, 500, "f32", seed=5)
    q = p[:, :6].contiguous()
    a, t = check(p, q, x, u)
    assert (a == 6).all() and torch.equal(t[:, :6], x) and (t[:, 6] >= 0).all()


def test_accept_offsets_past_32_bits():
    """A row that begins behind element 2^31."""
    N, V = 1100, 1000003
    p = torch.zeros(N, 2, V, dtype=torch.bfloat16, device="cuda")
    x = torch.full((N, 1), 5, dtype=torch.int32, device="cuda")
    p[:, 0, 5] = 1.0
    p[:, 1, V - 2] = 0.5
    p[N - 1, 1, V - 2] = 0.0
    p[N - 1, 1, V - 1] = 0.5
    a, t = kda.spec_accept(p, None, x, torch.full((N, 2), 0.5, device="cuda"))
    assert (a == 1).all() and (t[:, 0] == 5).all() and (t[:-1, 1] == V - 2).all() and t[-1, 1] == V - 1


def test_accept_captured_and_replayed():
    p, q, x, u = case(6, 4, 5003, "f32", seed=7)
    acc, tok = torch.empty(6, dtype=torch.int32, device="cuda"), torch.empty(6, 5, dtype=torch.int32, device="cuda")
    kda.spec_accept(p, q, x, u)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.spec_accept(p, q, x, u, accepted=acc, tokens=tok)
    for i in range(4):
        u.copy_(torch.rand(6, 5, generator=torch.Generator().manual_seed(i)))
        g.replay()
        a, t = check(p, q, x, u)
        assert torch.equal(a, acc) and torch.equal(t, tok)


def test_accept_feeds_the_commits():
    """Verify, accept, commit as a serving step uses them, for both recurrences: the committed
    states are those of decoding the kept drafts one by one."""
    N, K, H, V = 6, 4, 2, 911
    p, q, x, u = case(N, K, V, "f32", seed=11)
    u[:, :K] *= 0.7
    d = ki.make_decode_inputs(K, N, H, 128, 128, "bf16", seed=3, device="cuda")
    d = {n: t.transpose(0, 1).contiguous() for n, t in d.items()}
    S = ki.make_state(N, H, 128, 128, 0.3, seed=4, device="cuda")
    kda.spec_verify(*(d[n] for n in ("q", "k", "v", "log_alpha", "beta", "gate")), S)
    acc, tok = kda.spec_accept(p, q, x, u)
    want = S.clone()
    kda.spec_commit(d["k"], d["v"], d["log_alpha"], d["beta"], S, acc)
    la, be = d["log_alpha"][..., 0].float().contiguous(), d["beta"].float()
    G = ki.make_state(N, H, 128, 128, 0.3, seed=5, device="cuda")
    gwant = G.clone()
    kda.gdn_recurrent(d["q"], d["k"], d["v"], la, be, G, steps=acc, output=False)
    kept = acc.tolist()
    assert 0 < sum(kept) < N * K
    for n in range(N):
        for j in range(kept[n]):
            one = [d[m][n:n + 1, j].contiguous() for m in ("q", "k", "v", "log_alpha", "beta", "gate")]
            kda.decode_step(*one, want[n:n + 1])
            kda.gdn_recurrent(*one[:3], la[n:n + 1, j].contiguous(), be[n:n + 1, j].contiguous(), gwant[n:n + 1])
    assert torch.equal(S, want) and torch.equal(G, gwant)
