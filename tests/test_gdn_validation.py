"""Refusals of the gated delta rule's and of draft verification's entry points: made on the
host before any HIP call, so these run without a GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

from linear_attention_sequence_chunked_amd import _lib, gdn

A = 1 << 24  # fake, aligned "device" addresses; never dereferenced by these calls
STEP = 1 << 20
Q, K, V, LA, BE, S0, SF, OUT, ST, IDX, WS = (A + i * STEP for i in range(11))
INV, UNS = _lib.KDA_ERR_INVALID_ARGUMENT, _lib.KDA_ERR_UNSUPPORTED


def params(dtype=0, hk=2, hv=4, dk=64, dv=64, scale=1.0, qs=0, ks=0, vs=0):
    return _lib.GdnParams(dtype, hk, hv, dk, dv, scale, qs, ks, vs)


def status(st):
    return st, _lib.load().kda_last_error().decode()


def prefill(p=None, q=Q, k=K, v=V, la=LA, be=BE, cu=(0, 3, 5), n=2, s0=None, sf=None, out=OUT):
    p = params() if p is None else p
    c = None if cu is None else (ctypes.c_int32 * len(cu))(*cu)
    return status(_lib.load().kda_gdn_chunk_prefill(ctypes.byref(p) if p else None, q, k, v, la, be, c, n, s0, sf, out, None))


def recurrent(p=None, q=Q, k=K, v=V, la=LA, be=BE, n=2, t=1, steps=None, idx=None, slots=2, state=ST, upd=1, out=OUT):
    p = params() if p is None else p
    return status(_lib.load().kda_gdn_recurrent(ctypes.byref(p) if p else None, q, k, v, la, be, n, t, steps, idx, slots, state, upd, out, None))


def accept(dtype=1, n=2, k=3, vocab=100, p=Q, q=K, x=V, u=LA, counts=None, acc=S0, tok=SF, ws=WS, nb=1 << 16):
    return status(_lib.load().kda_spec_accept(dtype, n, k, vocab, p, q, x, u, counts, acc, tok, ws, nb, None))


BAD_PARAMS = [
    (False, INV, "params is NULL"), (params(dtype=2), INV, "dtype"), (params(hk=0), INV, "num_k_heads"),
    (params(hk=3), INV, "multiple of num_k_heads"), (params(hv=0), INV, "multiple"), (params(dk=96), UNS, "dk=96"),
    (params(dv=256), UNS, "dv=256"), (params(scale=float("nan")), INV, "scale"), (params(qs=120), INV, "q_stride"),
    (params(ks=132), INV, "k_stride"), (params(vs=255), INV, "v_stride"), (params(vs=1 << 32), UNS, "v_stride"),
    (params(qs=-128), INV, "q_stride"),
]


@pytest.mark.parametrize("p,st,msg", BAD_PARAMS)
def test_params_rejected(p, st, msg):
    for call in (prefill, recurrent):
        got, err = call(p=p)
        assert got == st and msg in err, err


@pytest.mark.parametrize("kw,st,msg", [
    (dict(n=0), INV, "num_seqs"), (dict(cu=None), INV, "cu_seqlens_host is NULL"), (dict(cu=(1, 3, 5)), INV, "must be 0"),
    (dict(cu=(0, 5, 3)), INV, "decreases"), (dict(q=None), INV, "q is NULL"), (dict(k=K + 8), INV, "k is not 16-byte"),
    (dict(v=None), INV, "v is NULL"), (dict(la=LA + 2), INV, "log_alpha"), (dict(be=None), INV, "beta is NULL"),
    (dict(out=None), INV, "out is NULL"), (dict(out=K), INV, "out overlaps k"), (dict(out=LA), INV, "out overlaps log_alpha"),
    (dict(s0=S0 + 4), INV, "initial_state is not"), (dict(s0=S0, sf=S0 + 256), INV, "final_state overlaps initial_state"),
    (dict(sf=OUT), INV, "final_state overlaps out"), (dict(sf=V), INV, "final_state overlaps v"), (dict(s0=OUT), INV, "out overlaps initial_state"),
    (dict(p=params(qs=65536), out=Q + 4 * 65536 * 2), INV, "out overlaps q"),
])
def test_prefill_rejects(kw, st, msg):
    got, err = prefill(**kw)
    assert got == st and msg in err, err


@pytest.mark.parametrize("kw,st,msg", [
    (dict(n=-1), INV, "num_seqs"), (dict(t=0), INV, "num_tokens"), (dict(t=17), INV, "num_tokens"), (dict(slots=-1), INV, "num_slots"),
    (dict(slots=1), INV, "without state_indices"), (dict(out=None, upd=0), INV, "out is NULL and update_state"),
    (dict(steps=IDX, upd=0), INV, "steps given"), (dict(state=None), INV, "state is NULL"), (dict(state=ST + 8), INV, "state is not"),
    (dict(out=ST), INV, "out overlaps state"), (dict(state=Q), INV, "state overlaps q"), (dict(out=Q), INV, "out overlaps q"),
    (dict(steps=IDX + 1), INV, "steps is not"), (dict(idx=IDX + 2), INV, "state_indices is not"), (dict(idx=ST), INV, "state overlaps state_indices"),
    (dict(n=1 << 30, slots=2, idx=IDX, q=1 << 40, k=1 << 42, v=1 << 44, la=1 << 46, be=1 << 47, out=1 << 48, state=1 << 20), UNS, "exceed one launch"),
])
def test_recurrent_rejects(kw, st, msg):
    got, err = recurrent(**kw)
    assert got == st and msg in err, err


def test_recurrent_of_no_sequences_is_nothing():
    assert recurrent(n=0)[0] == _lib.KDA_OK


@pytest.mark.parametrize("kw,st,msg", [
    (dict(dtype=3), INV, "dtype"), (dict(n=-1), INV, "num_seqs"), (dict(k=-1), INV, "num_draft"), (dict(k=65), INV, "num_draft"),
    (dict(vocab=0), INV, "vocab"), (dict(vocab=1 << 31), INV, "vocab"), (dict(p=None), INV, "target_probs is NULL"),
    (dict(q=K + 2), INV, "draft_probs is not"), (dict(x=None), INV, "draft_tokens is NULL"), (dict(u=None), INV, "uniforms is NULL"),
    (dict(acc=None), INV, "accepted is NULL"), (dict(tok=None), INV, "tokens is NULL"), (dict(ws=None), INV, "workspace is NULL"),
    (dict(nb=8), INV, "workspace_bytes 8"), (dict(acc=Q), INV, "accepted overlaps target_probs"), (dict(tok=S0), INV, "tokens overlaps accepted"),
    (dict(ws=SF), INV, "workspace overlaps tokens"), (dict(counts=S0), INV, "accepted overlaps num_drafts"),
])
def test_accept_rejects(kw, st, msg):
    got, err = accept(**kw)
    assert got == st and msg in err, err


def test_accept_workspace_sizes():
    lib = _lib.load()
    assert lib.kda_spec_accept_workspace(0, 10) == 0
    assert lib.kda_spec_accept_workspace(1, 1) == 16
    assert lib.kda_spec_accept_workspace(-1, 10) == -1 and lib.kda_spec_accept_workspace(1, 0) == -1
    assert lib.kda_spec_accept_workspace(1, 1 << 20) == 16 * 256  # at most 256 pieces
    assert accept(n=0)[0] == _lib.KDA_OK


def test_launches_beyond_the_grid_are_refused():
    """2^24 states of one launch: more threads than a grid counts."""
    p = params(hk=1, hv=1 << 16, dv=128)
    st, msg = prefill(p, cu=[0] * 257, n=256, q=None, k=None, v=None, la=None, be=None, out=None)
    assert st == UNS and "workgroups exceed one launch" in msg
    far = dict(q=1 << 54, k=1 << 55, v=1 << 56, la=1 << 57, be=1 << 58, out=1 << 59)
    st, msg = recurrent(p, n=1 << 12, slots=0, idx=1 << 53, state=None, upd=0, **far)
    assert st == UNS and "workgroups exceed one launch" in msg
    st, msg = accept(n=1 << 23, k=0, vocab=8, p=1 << 54, q=None, x=None, u=1 << 55, acc=1 << 56, tok=1 << 57, ws=1 << 58, nb=1 << 40)
    assert st == UNS and "workgroups exceed one launch" in msg


# ------------------------------------------------------------------------------ the binding

@pytest.fixture
def on_cpu(monkeypatch):
    """CPU tensors taken for GPU ones: a call that passes the checks would reach the library."""
    class Reached(Exception):
        pass

    def load():
        raise Reached
    monkeypatch.setattr(gdn, "_head_dims", lambda q, v: (q.shape[-2], v.shape[-2], q.shape[-1], v.shape[-1]))
    monkeypatch.setattr("linear_attention_sequence_chunked_amd.ops._on_gpu", lambda t: True)
    monkeypatch.setattr(gdn._lib, "load", load)
    return Reached


def tensors(T=6, hk=2, hv=4, dk=64, dv=64, dt=torch.bfloat16):
    z = lambda *s: torch.zeros(s, dtype=dt)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    return dict(q=z(T, hk, dk), k=z(T, hk, dk), v=z(T, hv, dv), log_alpha=f(T, hv), beta=f(T, hv))


def test_binding_prefill_refusals(on_cpu):
    ok = tensors()
    with pytest.raises(on_cpu):
        gdn.gdn_chunk_prefill(**ok, cu_seqlens=[0, 2, 6])
    for change, cu in [(dict(k=ok["k"][:5]), [0, 6]), (dict(q=ok["q"].float()), [0, 6]), (dict(log_alpha=ok["log_alpha"].bfloat16()), [0, 6]),
                       (dict(beta=ok["beta"][:, :3]), [0, 6]), (dict(), None), (dict(), [0, 5]), (dict(), [0, 4, 3, 6]), (dict(), [6]),
                       (dict(v=ok["v"].transpose(1, 2)), [0, 6]), (dict(initial_state=torch.zeros(2, 4, 64, 64)), [0, 6]),
                       (dict(out=torch.zeros(6, 4, 64)), [0, 6]), (dict(final_state=torch.zeros(1, 4, 64, 64).double()), [0, 6]),
                       (dict(k=torch.zeros(6, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), [0, 6])]:
        with pytest.raises(ValueError):
            gdn.gdn_chunk_prefill(**dict(ok, **change), cu_seqlens=cu)


def test_binding_token_strides(on_cpu):
    w = torch.zeros(6, 512, dtype=torch.bfloat16)
    dev = w.device
    assert gdn._tokens("q", w[:, :128].view(6, 2, 64), 2, 64, w.dtype, dev) == 512
    assert gdn._tokens("q", w[:1, :128].view(1, 2, 64), 2, 64, w.dtype, dev) == 128
    assert gdn._tokens("q", w.view(2, 3, 512)[..., :128].view(2, 3, 2, 64), 2, 64, w.dtype, dev) == 512
    assert gdn._tokens("q", w.view(6, 1, 512)[..., :128].view(6, 1, 2, 64), 2, 64, w.dtype, dev) == 512
    with pytest.raises(ValueError):  # rows of different sequences are not one stride apart
        gdn._tokens("q", w.view(2, 3, 512)[:, :2, :128].view(2, 2, 2, 64), 2, 64, w.dtype, dev)


def test_binding_refuses_overlapping_tokens(on_cpu):
    """A token stride of 0 (an expanded tensor) must not reach the library, where 0 means dense."""
    one = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for t in (one.expand(6, 2, 64), one[None].expand(3, 2, 2, 64), one[None].expand(6, 1, 2, 64), torch.zeros(512, dtype=torch.bfloat16).as_strided((6, 2, 64), (64, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            gdn._tokens("q", t, 2, 64, t.dtype, t.device)
    x = tensors()
    for name in ("q", "k", "v"):
        with pytest.raises(ValueError, match="overlap"):
            gdn.gdn_chunk_prefill(**dict(x, **{name: x[name][:1].expand_as(x[name])}), cu_seqlens=[0, 6])
        with pytest.raises(ValueError, match="overlap"):
            gdn.gdn_recurrent(**dict(x, **{name: x[name][:1].expand_as(x[name])}), state=torch.zeros(6, 4, 64, 64))


def test_binding_recurrent_refusals(on_cpu):
    x = tensors()
    st = torch.zeros(8, 4, 64, 64)
    i32 = torch.zeros(6, dtype=torch.int32)
    with pytest.raises(on_cpu):
        gdn.gdn_recurrent(**x, state=st, state_indices=i32, steps=i32)
    for kw in (dict(state=st[:, :3]), dict(state=st.half()), dict(steps=i32.long()), dict(state_indices=i32[:5]), dict(state=st[0]),
               dict(out=torch.zeros(6, 4, 64), output=False), dict(out=torch.zeros(6, 4, 64))):
        with pytest.raises(ValueError):
            gdn.gdn_recurrent(**dict(dict(x, state=st), **kw))


def test_binding_refuses_cpu_tensors():
    x = tensors()
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_chunk_prefill(**x, cu_seqlens=[0, 6])
    with pytest.raises(ValueError, match="GPU"):
        gdn.gdn_recurrent(**x, state=torch.zeros(6, 4, 64, 64))
    with pytest.raises(ValueError, match="GPU"):
        gdn.spec_accept(torch.zeros(1, 2, 4), None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))


# ------------------------------------------------------------------------------ sanitizers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_sequence_chunked_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(not os.path.exists(os.path.join(ROCM, "lib", "libamdhip64.so")), reason="needs the HIP runtime")
def test_host_paths_under_sanitizers(tmp_path):
    """The entry points' host code under ASan and UBSan, launches stubbed out."""
    exe = str(tmp_path / "gdn_driver")
    here = os.path.join(ROOT, "tests", "sanitize")
    cmd = ["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{CSRC}",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1", os.path.join(CSRC, "gdn_api.cpp"),
           os.path.join(CSRC, "gdn_plan.cpp"), os.path.join(here, "gdn_driver.cpp"), f"-L{ROCM}/lib", "-lamdhip64",
           f"-Wl,-rpath,{ROCM}/lib", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and "0 unexpected results" in r.stdout, r.stdout + r.stderr
