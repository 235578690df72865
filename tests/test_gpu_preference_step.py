"""A run as preference training uses the operators together: answers from decode(), the step with the loss in the
middle, the clipped gradients, and the answers of the model after a change to its adapters."""
import numpy as np
import pytest

from layer_streamed_nf4_b200 import synth

pytestmark = pytest.mark.gpu

CFG = synth.StackConfig("tiny", 3, 256, 128, 512, 96, 16, 32.0, "nf4", vocab=0)


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from layer_streamed_nf4_b200 import lsnf4
    return lsnf4


def _batch(T, vocab, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    tgt = rng.integers(0, vocab, T).astype(np.int32)
    start = np.array([0, T // 4, T // 2, T // 2 + 9, T - 3], np.int32)
    for i in range(4):
        tgt[start[i]:start[i] + 4] = -100
    return torch.from_numpy(tgt).cuda(), torch.from_numpy(start).cuda()


@pytest.mark.parametrize("mode,ahead", [("resident", False), ("streamed", True), ("streamed", False)])
def test_preference_step(lib, mode, ahead):
    """Loss, rewards and the last layer's output gradient against fp64 from the stack's own outputs.  The logits are
    bf16 and their GEMM is held to 2e-2 of their RMS elsewhere, so each differs from fp64 by eps = 2^-8 |l| + 2e-2 rms;
    a token's log-probability by 2 eps, a sequence's by n times that; the gradient's factors by exp(2 eps) - 1 and the
    change of the loss's slope (at most beta^2 / 4 times the ratio's error, relative to its value), both GEMMs' and
    the roundings' relative errors of 2^-8 and 5e-3 added."""
    import torch
    from layer_streamed_nf4_b200.stack import Preference, Stack
    st = Stack(CFG, mode=mode, n_slots=2, dequant_ahead=ahead, keep_outputs=True)
    V, beta = 640, 0.5
    tgt, start = _batch(CFG.tokens, V)
    pr = Preference(st, V, tgt, start, beta)
    down = 6
    old = st.dY[st.L - 1, down].clone()
    max_norm = 1e-3
    st.step(preference=pr, max_norm=max_norm)
    torch.cuda.synchronize()
    st.check_status()
    head = pr.head.double()
    out = {}
    for name, h in (("ref", st.y_ref[st.L - 1, down]), ("own", st.y[st.L - 1, down])):
        out[name] = (h.double() @ head.T).cpu().numpy()
    eps = {k: 2.0 ** -8 * np.abs(v).max() + 2e-2 * np.sqrt(np.mean(v * v)) for k, v in out.items()}
    t, s = tgt.cpu().numpy(), start.cpu().numpy()
    logp, n = {}, np.zeros(4)
    for k, l in out.items():
        lse = np.log(np.exp(l).sum(1))
        logp[k] = np.zeros(4)
        for i in range(4):
            rows = [r for r in range(s[i], s[i + 1]) if t[r] >= 0]
            n[i] = len(rows)
            logp[k][i] = sum(l[r, t[r]] - lse[r] for r in rows)
    got_own, got_ref = pr.logp.cpu().numpy(), pr.ref_logp.cpu().numpy()
    assert (np.abs(got_own - logp["own"]) <= 2 * n * eps["own"]).all()
    assert (np.abs(got_ref - logp["ref"]) <= 2 * n * eps["ref"]).all()
    # the loss from the log-probabilities as computed: fp32 roundings only
    ratio = got_own - got_ref
    z = beta * (ratio[0::2] - ratio[1::2])
    loss = np.log1p(np.exp(-z))
    assert np.allclose(pr.loss.cpu().numpy(), loss, rtol=2.0 ** -20) and np.isclose(float(pr.mean_loss), loss.mean(), rtol=2.0 ** -20)
    d = -beta / (1 + np.exp(z)) / 2
    c = np.stack([d, -d], 1).reshape(-1)
    l, p = out["own"], np.exp(out["own"] - np.log(np.exp(out["own"]).sum(1))[:, None])
    g = np.zeros_like(l)
    for i in range(4):
        for r in range(s[i], s[i + 1]):
            if t[r] >= 0:
                g[r] = -c[i] * p[r]
                g[r, t[r]] += c[i]
    want = g @ head.cpu().numpy()
    got = st.dY[st.L - 1, down].double().cpu().numpy()
    rel = np.expm1(2 * eps["own"]) + 2 * 2.0 ** -8 + 5e-3
    assert np.linalg.norm(got - want) <= rel * np.linalg.norm(want) + 1e-12
    assert (got[s[4]:] == 0).all() and not torch.equal(old, st.dY[st.L - 1, down])
    # clipped: the norm of what the buffer holds now, and what it was before
    total = float(st._clip[4])
    now = float(st.grads.double().square().sum().sqrt())
    assert total > max_norm and abs(now - max_norm) <= max_norm * 2.0 ** -20
    # the same step without clipping gives the same gradients up to the factor
    clipped = st.grads.clone()
    pr2 = Preference(st, V, tgt, start, beta, head=pr.head)
    st.step(preference=pr2)
    torch.cuda.synchronize()
    assert torch.equal(pr2.loss, pr.loss)
    f = np.float32(max_norm / float(st.grads.double().square().sum().sqrt()))
    assert float((st.grads * float(f) - clipped).abs().max()) <= float(clipped.abs().max()) * 2.0 ** -21
    st.close()


def test_adapters_off_means_no_preference(lib):
    """With B = 0 the model is its reference: every ratio is 0, every loss log 2, and the gradients push apart."""
    import torch
    from layer_streamed_nf4_b200.stack import Preference, Stack
    st = Stack(CFG, mode="streamed", n_slots=3)
    for k in st.B:
        st.B[k].zero_()
    tgt, start = _batch(CFG.tokens, 640, 1)
    pr = Preference(st, 640, tgt, start, 0.1)
    st.step(preference=pr)
    torch.cuda.synchronize()
    assert torch.equal(pr.logp, pr.ref_logp) and bool((pr.reward == 0).all())
    assert np.allclose(pr.loss.cpu().numpy(), np.log(2.0), rtol=2.0 ** -22)
    assert float(st.grads.abs().max()) > 0
    st.close()


@pytest.mark.parametrize("mode,S", [("resident", 2), ("streamed", 2), ("streamed", 1)])
def test_decode_agrees_with_the_forward(lib, mode, S):
    """decode() and forward() on the same tokens.  Per element: forward rounds each weight to bf16 (2^-8 of |w x|
    summed), s u to bf16 (2^-8 of |s u B| summed), each output once more (2^-8 |y| on either side); decode rounds the
    levels to fp16 (2^-11) and the sums' order differs (fp32, below 2^-12 of the sums together)."""
    import torch
    from layer_streamed_nf4_b200.stack import Stack
    st = Stack(CFG, mode=mode, n_slots=S)
    few = st.with_tokens(5, mode=mode, n_slots=S)
    for adapter in (True, False):
        few.forward(adapter=adapter)
        torch.cuda.synchronize()
        d = few.y if adapter else few.y_ref
        want = {k: v.clone() for k, v in d.items()}
        for v in d.values():
            v.fill_(float("nan"))
        few.decode(adapter=adapter)
        torch.cuda.synchronize()
        for k, v in d.items():
            a, b = v.double(), want[k].double()
            l, pi = (st.L - 1, k[1])                    # without kept outputs, the last layer's are left
            p, x = few.proj[pi], few.x[l, pi].double().abs()
            W = torch.empty(p.N, p.K, dtype=torch.bfloat16, device="cuda")
            addr = few._acquire(l)
            lib.nf4_dequant(few._nf4_view(addr, l, p), W, few.stream)
            few._release(l)
            sums = x @ W.double().abs().T
            lora = few.scale * (x @ few.A[l, pi].double().abs().T) @ few.B[l, pi].double().abs().T if adapter else 0.0
            assert bool(((a - b).abs() <= (2.0 ** -8 + 2.0 ** -10) * (sums + lora) + 2.0 ** -7 * (b.abs() + 2.0 ** -8 * sums)).all()), k
    few.close()
    st.close()


def test_the_three_together(lib):
    """Answer, train a step on preferences with clipping, move the adapters along the gradient, answer again: the loss
    is finite, the gradients' norm is the bound, and the answers change only through the adapters."""
    import torch
    from layer_streamed_nf4_b200.stack import Preference, Stack
    st = Stack(CFG, mode="streamed", n_slots=2)
    few = st.with_tokens(1, mode="no_h2d")
    few.A, few.B = st.A, st.B                       # the adapters being trained
    few._calls = {}
    few.decode()
    few.decode(adapter=False)
    torch.cuda.synchronize()
    before, base = [few.y[0, i].clone() for i in range(7)], [few.y_ref[0, i].clone() for i in range(7)]
    tgt, start = _batch(CFG.tokens, 640, 2)
    pr = Preference(st, 640, tgt, start, 0.5)
    st.step(preference=pr, max_norm=0.25)
    for k in st.B:
        st.A[k] -= st.dA[k].to(torch.bfloat16)
        st.B[k] -= st.dB[k].to(torch.bfloat16)
    few.decode()
    few.decode(adapter=False)
    torch.cuda.synchronize()
    assert bool(pr.mean_loss.isfinite().all()) and float(st._clip[4]) > 0
    assert all(torch.equal(few.y_ref[0, i], base[i]) for i in range(7))
    # (the down projection's share of the bounded norm need not reach a step of bf16: any projection's may)
    assert any(not torch.equal(few.y[0, i], before[i]) for i in range(7))
    few.close()
    st.close()


@pytest.mark.parametrize("where", ["decode", "head"])
def test_a_kernel_that_gave_up_is_noticed(lib, where):
    """check_status() reads the workspaces of decode() and of the loss's head too: a status word as a kernel sets it
    is raised once."""
    import torch
    from layer_streamed_nf4_b200.stack import Preference, Stack
    st = Stack(CFG, tokens=16, mode="resident")
    tgt, start = _batch(16, 640, 4)
    pr = Preference(st, 640, tgt, start.clamp(max=16), 0.1)
    st.decode()
    st.check_status()
    (st._decode_ws if where == "decode" else pr._hws)[:4].view(torch.int32).fill_(1)
    with pytest.raises(lib.LsnError):
        st.check_status()
    st.check_status()
    st.close()


def test_answers_come_from_the_trained_adapters(lib):
    """A stack made by with_tokens answers with the adapters of the stack it came from, changed in place before it was
    made or after: with B = 0 the answers are the reference's, with another B they differ from the first ones."""
    import dataclasses
    import torch
    from layer_streamed_nf4_b200.stack import Stack
    st = Stack(dataclasses.replace(CFG, vocab=320), mode="streamed", n_slots=2)
    early = st.with_tokens(3, mode="resident")
    early.decode()
    torch.cuda.synchronize()
    first = [early.y[0, i].clone() for i in range(7)]
    for k in st.B:
        st.B[k] *= -2
    late = st.with_tokens(3, mode="resident")
    for few in (early, late):
        few.decode()
        torch.cuda.synchronize()
        assert any(not torch.equal(few.y[0, i], first[i]) for i in range(7))
    assert all(torch.equal(early.y[0, i], late.y[0, i]) for i in range(7))
    for k in st.B:
        st.B[k].zero_()
    for few in (early, late):
        few.decode()
        few.decode(adapter=False)
        torch.cuda.synchronize()
        assert all(torch.equal(few.y[0, i], few.y_ref[0, i]) for i in range(7))
    assert late.embedding is st.embedding and late.grads.data_ptr() != st.grads.data_ptr()
    shared = st.with_inputs(mode="streamed")
    assert all(shared.A[k] is st.A[k] and shared.B[k] is st.B[k] for k in st.A)
    for s in (early, late, shared, st):
        s.close()
