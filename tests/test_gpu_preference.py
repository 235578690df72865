"""Sequence log-probabilities and the preference loss against a plain fp64 computation.

Tolerances come from the roundings of the computation.  exp(x - m) by ex2.approx: 2^-22, its argument's roundings
2 |x - m| 2^-24, the fp32 sum of V terms no deeper than V / 256 + 64 additions: `tol_s` relative in the sum, so absolute
in lse and in each token's log-probability; n tokens add up to n tol_s.  The loss moves by at most its slope times that.
dlogits: |c| p times the relative error of p (tol_s, the lse's own rounding, ex2), the error of c, and half a step of
the output type (bf16 2^-8, fp32 2^-24)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from layer_streamed_nf4_b200 import lsnf4
    return lsnf4


class Batch:
    def __init__(self, lib, lens, V, pad=0, dtype="bf16", tail=0, lead=0, average=False, seed=0, std=2.0, prompt=0.3, offset=0):
        import torch
        rng = np.random.default_rng(seed)
        self.lib, self.V, self.ld, self.average = lib, V, V + pad, average
        self.start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32) + lead
        self.T = int(self.start[-1]) + tail
        self.n = len(lens)
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        buf = torch.from_numpy(rng.normal(0, std, self.T * self.ld + offset).astype(np.float32)).cuda().to(self.dt)
        self.logits = buf[offset:].view(self.T, self.ld)
        self.targets = rng.integers(0, V, self.T).astype(np.int32)
        for i, n in enumerate(lens):
            k = int(n * prompt)
            self.targets[self.start[i]:self.start[i] + k] = rng.choice([-100, -1, V, 2 ** 30], k)
        self.ref = rng.normal(0, 1, self.n) - 6.0 * (1 if average else np.maximum(np.array(lens, float) * (1 - prompt), 0))
        self.upload()

    def upload(self):
        import torch
        lib, T, n = self.lib, self.T, self.n
        self.tgt, self.st = torch.from_numpy(self.targets).cuda(), torch.from_numpy(self.start).cuda()
        self.refd = torch.from_numpy(self.ref).cuda()
        self.sl = lib.seq_logits(self.logits, T, self.V, self.ld, lib.LSN_DT_BF16 if self.dt == torch.bfloat16 else lib.LSN_DT_F32, self.tgt, n, self.st, self.average)
        nan = float("nan")
        self.lse = torch.full((T + 1,), nan, device="cuda")
        self.logp = torch.full((n,), nan, device="cuda", dtype=torch.float64)
        self.count = torch.full((n,), -7, device="cuda", dtype=torch.int32)
        self.reward, self.dlogp = torch.full((n,), nan, device="cuda"), torch.full((n,), nan, device="cuda")
        self.loss, self.mean = torch.full((max(1, n // 2),), nan, device="cuda"), torch.full((1,), nan, device="cuda")
        self.nws = lib.seq_logp_ws_bytes(self.sl)
        self.ws = torch.zeros(self.nws, dtype=torch.uint8, device="cuda")

    def ref64(self):
        """lse, logp, count, scored rows, each row's sequence and probabilities in fp64."""
        x = self.logits[:, :self.V].double().cpu().numpy()
        with np.errstate(invalid="ignore", divide="ignore"):
            m = x.max(1, initial=-np.inf)
            self.m = m
            lse = m + np.log(np.exp(x - m[:, None]).sum(1))
        on = np.zeros(self.T, bool)
        logp, count = np.zeros(self.n), np.zeros(self.n, int)
        seq = np.zeros(self.T, int)
        with np.errstate(invalid="ignore"):
            for i in range(self.n):
                for t in range(self.start[i], self.start[i + 1]):
                    seq[t] = i
                    if 0 <= self.targets[t] < self.V:
                        on[t] = True
                        logp[i] += x[t, self.targets[t]] - lse[t]
                        count[i] += 1
        if self.average:
            logp = logp / np.maximum(count, 1)
        return x, lse, logp, count, on, seq

    def tol_s(self, x):
        f = x[np.isfinite(x)]
        spread = float(f.max() - f.min()) if f.size else 0.0
        return 2.0 ** -22 + 2.0 ** -24 * (2 * min(spread, 100.0) * 1.45 + self.V / 256 + 64)

    def check_fwd(self, rows=None):
        x, lse, logp, count, on, _ = self.ref64()
        ts = self.tol_s(x)
        got = self.lse.cpu().numpy()[:self.T].astype(float)
        want = np.where(on, lse, 0.0)
        ok = np.abs(got - want) <= ts + np.abs(want) * 2.0 ** -24
        assert ok.all(), (np.flatnonzero(~ok)[:5], got[~ok][:5], want[~ok][:5])
        assert np.array_equal(self.count.cpu().numpy(), count)
        n = 1 if self.average else np.maximum(count, 1)
        assert (np.abs(self.logp.cpu().numpy() - logp) <= n * ts + 1e-12 * np.abs(logp)).all()
        assert bool(self.lse[self.T].isnan()), "wrote behind the last row"


def loss64(kind, beta, e, h):
    z = beta * h
    if kind == 0:
        sp = lambda v: np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))
        sg = lambda v: 1 / (1 + np.exp(-v))
        with np.errstate(over="ignore"):
            return (1 - e) * sp(-z) + e * sp(z), beta * (e * sg(z) - (1 - e) * sg(-z)), beta * beta / 4
    if kind == 1:
        return np.maximum(0, 1 - z), np.where(1 - z > 0, -beta, 0.0), 0.0
    return (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta), 2.0


def check_loss(b, kind, beta, e=0.0, scale=1.0, ref=True):
    """Loss, rewards, mean and dlogp; returns dlogp in fp64 and its tolerance."""
    x, lse, logp, count, on, _ = b.ref64()
    ts = b.tol_s(x)
    a = logp - (b.ref if ref else 0.0)
    err = (1 if b.average else np.maximum(count, 1)) * ts + 1e-12 * np.abs(logp)
    h, dh = a[0::2] - a[1::2], err[0::2] + err[1::2]
    loss, d, curv = loss64(kind, beta, e, h)
    tol = np.abs(d) * dh + curv * dh ** 2 + np.abs(loss) * 2.0 ** -23 + 1e-30
    if kind == 1:
        assert (np.abs(1 - beta * h) > beta * dh).all(), "a pair at the hinge's corner"
    assert (np.abs(b.loss.cpu().numpy() - loss) <= tol).all(), (b.loss.cpu().numpy(), loss)
    assert (np.abs(b.reward.cpu().numpy() - beta * a) <= beta * err + np.abs(beta * a) * 2.0 ** -23).all()
    P = len(h)
    assert abs(float(b.mean) - loss.mean()) <= tol.mean() + abs(loss.mean()) * 2.0 ** -23 + 1e-30
    dl = np.stack([d, -d], 1).reshape(-1) * scale / P
    told = np.repeat(curv * dh, 2) * abs(scale) / P + np.abs(dl) * 2.0 ** -23
    assert (np.abs(b.dlogp.cpu().numpy() - dl) <= told).all()
    return dl, told


def check_grad(b, dl, told, got, logits=None):
    import torch
    x, lse, _, count, on, seq = b.ref64() if logits is None else logits
    ts = b.tol_s(x)
    n = np.maximum(count, 1) if b.average else np.ones(b.n)
    c, dc = np.where(on, (dl / n)[seq], 0.0), np.where(on, (told / n)[seq], 0.0)
    with np.errstate(invalid="ignore", over="ignore"):
        arg = np.where(on[:, None], x - lse[:, None], -np.inf)
        p = np.exp(arg)
        hot = np.zeros_like(p)
        hot[np.flatnonzero(on), b.targets[on]] = 1.0
        want = np.where(on[:, None], c[:, None] * (hot - p), 0.0)
        rel = ts + np.abs(np.where(on, lse, 0))[:, None] * 2.0 ** -24 + 2.0 ** -22 + 2 * np.minimum(np.abs(arg), 200) * 1.45 * 2.0 ** -24
    half = 2.0 ** -8 if b.dt == torch.bfloat16 else 2.0 ** -24
    tol = np.abs(c)[:, None] * p * rel + dc[:, None] * np.abs(hot - p) + (np.abs(c)[:, None] * (hot + p)) * 2.0 ** -23 + np.abs(want) * half + 1e-37
    g = got.double().cpu().numpy()[:b.T, :b.V]
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], g[bad][:4], want[bad][:4])


SHAPES = [((3, 1), 17, 0, 0), ((5, 9, 0, 4), 1000, 0, 2), ((40, 33), 8192, 8, 0), ((1, 2), 32003, 5, 3), ((7, 300, 120, 2, 1, 1), 999, 1, 0),
          ((70, 61), 50000, 0, 1), ((2, 2), 151936, 0, 0)]


@pytest.mark.parametrize("lens,V,pad,tail", SHAPES)
@pytest.mark.parametrize("dtype,average,offset", [("bf16", False, 0), ("fp32", True, 0), ("bf16", True, 3), ("fp32", False, 1)])
def test_logp(lib, lens, V, pad, tail, dtype, average, offset):
    import torch
    b = Batch(lib, lens, V, pad, dtype, tail, average=average, offset=offset, seed=V)
    lib.seq_logp_fwd(b.sl, b.lse, b.logp, b.count, b.ws, b.nws)
    torch.cuda.synchronize()
    b.check_fwd()


@pytest.mark.parametrize("lens,V,pad,tail", SHAPES)
@pytest.mark.parametrize("dtype,average,kind,e,ld_extra,offset", [("bf16", False, 0, 0.0, 0, 0), ("fp32", False, 0, 0.1, 3, 0), ("bf16", True, 2, 0.0, 1, 5),
                                                                  ("fp32", True, 1, 0.0, 0, 2)])
def test_loss_and_gradients(lib, lens, V, pad, tail, dtype, average, kind, e, ld_extra, offset):
    """Forward and backward apart, then in one call: the same bits; columns behind V and the row behind T untouched."""
    import torch
    b = Batch(lib, lens, V, pad, dtype, tail, average=average, offset=offset, seed=V + kind, lead=1 if V < 5000 else 0)
    beta = 0.7 if average else 0.1
    p = lib.preference(kind, beta, e, grad_scale=0.5)
    lib.preference_loss_fwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, b.ws, b.nws)
    ld_d = V + pad + ld_extra
    d1 = torch.full((b.T + 1, ld_d), 3.0, dtype=b.dt, device="cuda")
    lib.seq_logp_bwd(b.sl, b.lse, b.dlogp, b.count, d1, ld_d)
    torch.cuda.synchronize()
    b.check_fwd()
    dl, told = check_loss(b, kind, beta, e, 0.5)
    check_grad(b, dl, told, d1)
    assert bool((d1[:, V:] == 3.0).all()) and bool((d1[b.T:] == 3.0).all())
    keep = [t.clone() for t in (b.lse[:b.T], b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp)]
    b.upload()
    d2 = torch.full((b.T + 1, ld_d), 3.0, dtype=b.dt, device="cuda")
    lib.preference_loss_fwd_bwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d2, ld_d, b.ws, b.nws)
    torch.cuda.synchronize()
    assert torch.equal(d1, d2)
    assert all(torch.equal(x, y) for x, y in zip(keep, (b.lse[:b.T], b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp)))


@pytest.mark.parametrize("dtype,V,pad,offset", [("bf16", 4097, 0, 0), ("fp32", 1003, 2, 1), ("bf16", 30000, 16, 0)])
def test_in_place_gradients(lib, dtype, V, pad, offset):
    import torch
    b = Batch(lib, (20, 11, 6, 30), V, pad, dtype, 2, seed=5, offset=offset)
    before = b.ref64()
    behind = b.logits[:, V:].clone()
    p = lib.preference(lib.LSN_PREF_SIGMOID, 0.2)
    lib.preference_loss_fwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, b.ws, b.nws)
    torch.cuda.synchronize()
    dl, told = check_loss(b, 0, 0.2)
    lib.preference_loss_fwd_bwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, b.logits, b.ld, b.ws, b.nws)
    torch.cuda.synchronize()
    check_grad(b, dl, told, b.logits, logits=before)
    assert torch.equal(b.logits[:, V:], behind)


def test_tensors_that_are_columns_of_wider_ones(lib):
    import torch
    b = Batch(lib, (9, 14, 3, 2), 501, 11, seed=6)
    p = lib.preference(lib.LSN_PREF_SIGMOID, 0.3)
    want, wide = (torch.full((b.T, n), 7.0, dtype=b.dt, device="cuda") for n in (b.V, b.V + 20))
    a = b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp
    lib.preference_loss_fwd_bwd(b.sl, *a, want, b.V, b.ws, b.nws)
    sl = lib.seq_logits(b.logits[:, :b.V], b.T, b.V, b.ld, lib.LSN_DT_BF16, b.tgt, b.n, b.st)
    lib.preference_loss_fwd_bwd(sl, *a, wide[:, 8:8 + b.V], b.V + 20, b.ws, b.nws)
    assert torch.equal(wide[:, 8:8 + b.V], want) and bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + b.V:] == 7).all())
    lib.seq_logp_bwd(sl, b.lse, b.dlogp, b.count, wide[:, 3:3 + b.V], b.V + 20)
    assert torch.equal(wide[:, 3:3 + b.V], want)
    with pytest.raises(lib.LsnError, match="strides"):
        lib.seq_logp_bwd(sl, b.lse, b.dlogp, b.count, torch.zeros(b.V, b.T, dtype=b.dt, device="cuda").t(), b.T)


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_without_a_reference_and_optional_outputs(lib, kind):
    import torch
    b = Batch(lib, (9, 14, 3, 2), 501, seed=kind)
    p = lib.preference(kind, 0.3)
    lib.preference_loss_fwd(b.sl, None, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, b.ws, b.nws)
    torch.cuda.synchronize()
    check_loss(b, kind, 0.3, ref=False)
    keep = b.loss.clone(), b.dlogp.clone()
    b.upload()
    lib.preference_loss_fwd(b.sl, None, p, b.lse, b.logp, None, None, b.loss, None, b.dlogp, b.ws, b.nws)
    torch.cuda.synchronize()
    assert torch.equal(b.loss, keep[0]) and torch.equal(b.dlogp, keep[1])


def test_gradient_of_any_function_of_the_log_probabilities(lib):
    import torch
    b = Batch(lib, (9, 14, 3), 777, dtype="fp32", seed=8, average=True)
    lib.seq_logp_fwd(b.sl, b.lse, b.logp, b.count, b.ws, b.nws)
    dl = np.array([0.5, -2.0, 0.0])
    d = torch.empty(b.T, b.V, device="cuda")
    lib.seq_logp_bwd(b.sl, b.lse, torch.tensor(dl, dtype=torch.float32, device="cuda"), b.count, d, b.V)
    torch.cuda.synchronize()
    check_grad(b, dl, np.abs(dl) * 2.0 ** -23, d)


def test_gradient_against_differences(lib):
    """Central differences of the mean loss itself.  Each of the 2 x 2 sequence sums is off by n tol_s, the loss by
    slope times that, over 2 delta; the third derivative of the loss along one logit is below 1 here."""
    import torch
    b = Batch(lib, (4, 6, 5, 3), 37, dtype="fp32", seed=3, std=1.0)
    p = lib.preference(lib.LSN_PREF_SIGMOID, 0.5, 0.1)
    args = (b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp)
    d = torch.empty(b.T, b.V, device="cuda")
    lib.preference_loss_fwd_bwd(b.sl, *args, d, b.V, b.ws, b.nws)
    torch.cuda.synchronize()
    x, _, _, count, on, _ = b.ref64()
    base, delta = b.logits.clone(), 2.0 ** -4
    noise = 0.5 * 2 * count.max() * b.tol_s(x) + 2.0 ** -23
    rng = np.random.default_rng(1)
    for t in range(b.T):
        for v in {int(b.targets[t]) if on[t] else 0, int(rng.integers(0, b.V))}:
            val = []
            for sgn in (1, -1):
                b.logits.copy_(base)
                b.logits[t, v] += sgn * delta
                lib.preference_loss_fwd(b.sl, *args, b.ws, b.nws)
                val.append(float(b.mean))
            num = (val[0] - val[1]) / (2 * delta)
            assert abs(num - float(d[t, v])) <= delta ** 2 / 6 + noise / delta, (t, v, num, float(d[t, v]))


def test_masked_vocabulary_and_the_lowest_value(lib):
    """Tokens masked with -infinity or the type's lowest value take no probability; a row with nothing else but the
    lowest value is uniform over it."""
    import torch
    for dtype in ("bf16", "fp32"):
        b = Batch(lib, (6, 8), 700, dtype=dtype, seed=2, prompt=0.0)
        low = torch.finfo(b.dt).min
        b.logits[:, 100:300] = float("-inf")
        b.logits[:, 400:500] = low
        b.logits[3] = low
        b.targets[:] = np.random.default_rng(0).integers(0, 100, b.T)
        b.upload()
        d = torch.empty(b.T, b.V, dtype=b.dt, device="cuda")
        p = lib.preference(lib.LSN_PREF_SIGMOID, 0.1)
        lib.preference_loss_fwd_bwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
        torch.cuda.synchronize()
        x = b.logits.double().cpu().numpy()
        on = [t for t in range(b.T) if t != 3]
        lse = np.log(np.exp(x[on]).sum(1))
        assert np.abs(b.lse.cpu().numpy()[on] - lse).max() <= 2.0 ** -18
        got = d.float().cpu().numpy()
        assert np.isfinite(got).all()
        assert (got[on][:, 100:300] == 0).all() and (got[on][:, 400:500] == 0).all()
        # uniform over 700 of the lowest value (log 700 is far below half a step of its exponent): logp = -log 700
        tok = x[on, b.targets[on]] - lse
        want = tok[:5].sum() - np.log(700.0)
        assert abs(float(b.logp[0]) - want) <= 6 * 2.0 ** -18


def test_non_finite_rows_stay_in_their_pair(lib):
    import torch
    for bad in ("nan", "inf", "-inf row"):
        b = Batch(lib, (6, 8, 5, 7, 4, 4), 700, seed=2, prompt=0.2)
        t = int(b.start[2]) + 4
        if bad == "-inf row":
            b.logits[t] = float("-inf")
        else:
            b.logits[t, 77] = float(bad)
        d = torch.empty(b.T, b.V, dtype=b.dt, device="cuda")
        p = lib.preference(lib.LSN_PREF_SIGMOID, 0.1)
        lib.preference_loss_fwd_bwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
        torch.cuda.synchronize()
        loss = b.loss.cpu().numpy()
        assert np.isnan(loss[1]) and np.isfinite(loss[[0, 2]]).all(), bad
        g = d.float().cpu().numpy()
        s = b.start
        scored = (b.targets >= 0) & (b.targets < b.V)
        mine = np.zeros(b.T, bool)
        mine[s[2]:s[4]] = True
        assert np.isnan(g[mine & scored]).all(), bad
        assert np.isfinite(g[~mine]).all() and (g[~scored] == 0).all(), bad


def test_an_impossible_target(lib):
    """A scored token of probability zero: the sequence's log-probability is -infinity, its gradients stay finite."""
    import torch
    for kind, want in ((0, [np.inf, 0.0]), (1, [np.inf, 0.0])):
        b = Batch(lib, (6, 8, 5, 7), 300, dtype="fp32", seed=2, prompt=0.0)
        b.logits[2, b.targets[2]] = float("-inf")                          # chosen of pair 0
        t = int(b.start[3]) + 1
        b.logits[t, b.targets[t]] = float("-inf")                          # rejected of pair 1
        d = torch.empty(b.T, b.V, device="cuda")
        lib.preference_loss_fwd_bwd(b.sl, b.refd, lib.preference(kind, 0.1), b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
        torch.cuda.synchronize()
        assert b.loss.cpu().tolist() == want
        assert np.isfinite(d.cpu().numpy()).all()
        assert np.allclose(b.dlogp.cpu().numpy(), [-0.05, 0.05, 0, 0])


def test_sequences_with_nothing_scored(lib):
    import torch
    b = Batch(lib, (5, 0, 4, 6), 200, dtype="fp32", seed=2, prompt=0.0, average=True)
    b.targets[b.start[2]:b.start[3]] = -100
    b.upload()
    d = torch.full((b.T, b.V), 9.0, device="cuda")
    lib.preference_loss_fwd_bwd(b.sl, b.refd, lib.preference(0, 0.4), b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
    torch.cuda.synchronize()
    b.check_fwd()
    check_grad(b, *check_loss(b, 0, 0.4), d)
    assert float(b.logp[1]) == 0.0 and float(b.logp[2]) == 0.0 and bool((d[b.start[2]:b.start[3]] == 0).all())


def test_no_rows_at_all(lib):
    import torch
    b = Batch(lib, (0, 0), 64, seed=1)
    b.sl = lib.seq_logits(None, 0, 64, 64, lib.LSN_DT_BF16, None, 2, b.st)
    lib.preference_loss_fwd_bwd(b.sl, None, lib.preference(0, 0.4), None, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, None, 64, b.ws, b.nws)
    torch.cuda.synchronize()
    assert b.logp.cpu().tolist() == [0.0, 0.0] and abs(float(b.mean) - np.log(2)) < 1e-6


def test_many_pairs_and_reruns_give_the_same_bits(lib):
    import torch
    rng = np.random.default_rng(4)
    b = Batch(lib, tuple(rng.integers(0, 6, 600)), 257, seed=9)
    p = lib.preference(lib.LSN_PREF_SIGMOID, 0.1)
    d = torch.empty(b.T, b.V, dtype=b.dt, device="cuda")
    first = None
    for _ in range(4):
        lib.preference_loss_fwd_bwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
        torch.cuda.synchronize()
        now = [t.clone() for t in (b.lse[:b.T], b.logp, b.loss, b.mean, b.dlogp, d)]
        assert first is None or all(torch.equal(x, y) for x, y in zip(first, now))
        first = now
    b.check_fwd()
    check_grad(b, *check_loss(b, 0, 0.1), d)


def test_captured_and_replayed_with_other_sequences(lib):
    import torch
    b = Batch(lib, (20, 30, 25, 5), 2000, seed=3)
    p = lib.preference(lib.LSN_PREF_SIGMOID, 0.1)
    d = torch.empty(b.T, b.V, dtype=b.dt, device="cuda")
    call = lambda st: lib.preference_loss_fwd_bwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws, st)  # noqa: E731
    call(None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call(st)
    for cut in ((0, 10, 40, 60, 75), (3, 3, 50, 51, 80), (0, 0, 0, 0, 80)):
        b.start = np.array(cut, np.int32)
        b.st.copy_(torch.from_numpy(b.start))
        b.logits.normal_(0, 2)
        g.replay()
        torch.cuda.synchronize()
        b.check_fwd()
        check_grad(b, *check_loss(b, 0, 0.1), d)


@pytest.mark.parametrize("pdl", [0, 1])
def test_dependent_launch_option(lib, pdl):
    import torch
    from tests.helpers import lib_option
    with lib_option(lib, lib.LSN_OPT_PDL, pdl):
        b = Batch(lib, (20, 30), 5000, seed=3)
        d = torch.empty(b.T, b.V, dtype=b.dt, device="cuda")
        for _ in range(3):
            lib.preference_loss_fwd_bwd(b.sl, b.refd, lib.preference(0, 0.1), b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
        torch.cuda.synchronize()
        b.check_fwd()
        check_grad(b, *check_loss(b, 0, 0.1), d)


def test_offsets_beyond_32_bits(lib):
    """A batch of over 2^32 logits: its last rows against their own 64-bit values."""
    import torch
    V, T = 151936, 28400                                             # 4.3e9 logits, 8.6 GB, in place
    logits = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    logits[-64:].normal_(0, 2)
    tail = logits[-64:].clone()
    tgt = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    st = torch.tensor([0, T - 64, T], dtype=torch.int32, device="cuda")
    sl = lib.seq_logits(logits, T, V, V, lib.LSN_DT_BF16, tgt, 2, st)
    lse, logp = torch.empty(T, device="cuda"), torch.empty(2, dtype=torch.float64, device="cuda")
    n = lib.seq_logp_ws_bytes(sl)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    lib.seq_logp_fwd(sl, lse, logp, None, ws, n)
    dlogp = torch.tensor([1.0, 2.0], device="cuda")
    lib.seq_logp_bwd(sl, lse, dlogp, None, logits, V)
    torch.cuda.synchronize()
    x = tail.double()
    ref = torch.logsumexp(x, 1)
    assert float((lse[-64:] - ref).abs().max()) <= 2.0 ** -22 + 2.0 ** -24 * (V / 256 + 64 + 60)
    assert float((lse[:-64] - np.log(V)).abs().max()) <= 2.0 ** -22 + 2.0 ** -24 * (V / 256 + 64 + 60)
    want = -2.0 * torch.softmax(x, 1)
    want[torch.arange(64, device="cuda"), tgt[-64:].long()] += 2.0
    assert float((logits[-64:].double() - want).abs().max()) <= 2.0 * 2.0 ** -8
    assert float((logits[0].float() + 1.0 / V).abs().median()) <= 2.0 ** -8 / V


@pytest.mark.parametrize("dtype,T,V", [("bf16", 1200, 12000), ("fp32", 300, 8190)])
@pytest.mark.parametrize("first,later", [(-3.3e38, -2e38), (1.5e38, 3e38), (0.5, 2e38), (-1e5, -7e4), (6e4, 7e4), (-7e4, -6e4)])
def test_a_maximum_that_grows_along_the_row(lib, dtype, T, V, first, later):
    """One piece of a row, two rounds of each thread: the first 4 x 256 words hold one value, the rest a larger one,
    over which the row is uniform."""
    import torch
    b = Batch(lib, (9, 7), V, dtype=dtype, tail=T - 16, seed=1, prompt=0.0)
    n = 1024 * (8 if dtype == "bf16" else 4)
    b.logits[:16, :n] = first
    b.logits[:16, n:V] = later
    b.targets[:16] = np.random.default_rng(0).integers(n, V, 16)
    b.targets[16:] = -100
    b.upload()
    lib.seq_logp_fwd(b.sl, b.lse, b.logp, b.count, b.ws, b.nws)
    torch.cuda.synchronize()
    ts = b.tol_s(np.zeros(1))
    want, m = -np.log(V - n), float(b.logits[0, V - 1])
    assert (np.abs(b.logp.cpu().numpy() - want * np.array([9, 7])) <= np.array([9, 7]) * ts).all(), (b.logp, want)
    assert (np.abs(b.lse[:16].double().cpu().numpy() - (m - want)) <= ts + abs(m) * 2.0 ** -24).all()


def check_scored_rows(lib, b, beta=0.1):
    """The whole loss with its gradient against fp64 on the scored rows, with the tolerances of the checks above."""
    import torch
    d = torch.full((b.T, b.V), 9.0, dtype=b.dt, device="cuda")
    p = lib.preference(lib.LSN_PREF_SIGMOID, beta)
    lib.preference_loss_fwd_bwd(b.sl, b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
    torch.cuda.synchronize()
    rows = np.flatnonzero((b.targets >= 0) & (b.targets < b.V) & (np.arange(b.T) >= b.start[0]) & (np.arange(b.T) < b.start[-1]))
    x = b.logits[torch.from_numpy(rows).cuda(), :b.V].double()
    tgt = torch.from_numpy(b.targets[rows]).long().cuda()
    lse = torch.logsumexp(x, 1)
    near = x[x > x.amax(1, keepdim=True) - 200]
    ts = b.tol_s(np.array([float(near.min()), float(near.max())]))
    assert bool(((b.lse[torch.from_numpy(rows).cuda()].double() - lse).abs() <= ts + lse.abs() * 2.0 ** -24).all())
    tok = (x.gather(1, tgt[:, None])[:, 0] - lse).cpu().numpy()
    seq = np.searchsorted(b.start, rows, side="right") - 1
    logp, n = np.bincount(seq, tok, b.n), np.bincount(seq, minlength=b.n)
    assert (np.abs(b.logp.cpu().numpy() - logp) <= n * ts + 1e-12 * np.abs(logp)).all()
    a, err = logp - b.ref, n * ts + 1e-12 * np.abs(logp)
    h, dh = a[0::2] - a[1::2], err[0::2] + err[1::2]
    loss, dl, curv = loss64(0, beta, 0.0, h)
    assert (np.abs(b.loss.cpu().numpy() - loss) <= np.abs(dl) * dh + curv * dh ** 2 + np.abs(loss) * 2.0 ** -23 + 1e-30).all()
    c = np.stack([dl, -dl], 1).reshape(-1) / len(h)
    dc = np.repeat(curv * dh, 2) / len(h) + np.abs(c) * 2.0 ** -23
    C, dC = (torch.from_numpy(v[seq]).cuda()[:, None] for v in (np.abs(c), dc))
    arg = x - lse[:, None]
    prob, hot = arg.exp(), torch.zeros_like(x).scatter_(1, tgt[:, None], 1.0)
    want = torch.from_numpy(c[seq]).cuda()[:, None] * (hot - prob)
    rel = ts + lse.abs()[:, None] * 2.0 ** -24 + 2.0 ** -22 + 2 * arg.abs().clamp_max(200) * 1.45 * 2.0 ** -24
    half = 2.0 ** -8 if b.dt == torch.bfloat16 else 2.0 ** -24
    tol = C * prob * rel + dC * (hot - prob).abs() + C * (hot + prob) * 2.0 ** -23 + want.abs() * half + 1e-37
    bad = ~((d[torch.from_numpy(rows).cuda()].double() - want).abs() <= tol)
    assert not bool(bad.any()), int(bad.sum())
    off = torch.ones(b.T, dtype=torch.bool, device="cuda")
    off[torch.from_numpy(rows).cuda()] = False
    assert bool((d[off] == 0).all())


MASKS = [(-1e4,), (-66000.0, -65000.0), (-1e5,), (-1e9,), (-2e9,), (-3e9,), (-1e10,), (-1e20,), (-1e30,), (-3e37,), (-1e10, -1e30),
         (float("-inf"), -1e12, -3.3e38)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("masks", MASKS, ids=str)
@pytest.mark.parametrize("where", ["words", "all but a few", "halves"])
@pytest.mark.parametrize("lens,V,tail", [((6, 8, 5, 3), 700, 0), ((6, 8), 32003, 2), ((6, 8), 12000, 1190)])
def test_finite_masks_of_any_size(lib, lens, V, tail, where, masks, dtype):
    """Tokens masked with a finite number take no probability, whatever its size, and leave the other tokens theirs:
    single aligned words, whole rows but a few tokens, the first half of a row; rows of one word a thread and of
    several."""
    b = Batch(lib, lens, V, dtype=dtype, tail=tail, seed=3, prompt=0.2)
    rng = np.random.default_rng(1)
    word = 16 // b.logits.element_size()
    for t in range(int(b.start[-1])):
        m = masks[t % len(masks)] if t % 3 else masks[0]
        keep = np.unique(np.append(rng.integers(0, V, 5), b.targets[t] if 0 <= b.targets[t] < V else 0))
        old = b.logits[t, keep].clone()
        if where == "words":
            for w in rng.integers(0, V // word, 6):
                b.logits[t, w * word:(w + 1) * word] = m
        elif where == "halves":
            b.logits[t, :V // 2] = m
        else:
            b.logits[t] = m
            if len(masks) > 1:
                b.logits[t, V // 3:2 * V // 3] = masks[(t + 1) % len(masks)]
        b.logits[t, keep] = old
    check_scored_rows(lib, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("top", [7e4, 3e9, 1e10, 1e30])
def test_one_large_logit(lib, top, dtype):
    """A token far above the others has probability one."""
    import torch
    b = Batch(lib, (6, 8), 700, dtype=dtype, seed=4, prompt=0.0)
    at = np.random.default_rng(2).integers(0, 700, b.T)
    b.logits[torch.arange(b.T, device="cuda"), torch.from_numpy(at).cuda()] = top
    b.targets[:] = at
    b.upload()
    d = torch.empty(b.T, b.V, dtype=b.dt, device="cuda")
    lib.preference_loss_fwd_bwd(b.sl, None, lib.preference(0, 0.1), b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp, d, b.V, b.ws, b.nws)
    torch.cuda.synchronize()
    assert bool((b.lse[:b.T] == b.logits[0, at[0]].float()).all()) and bool((b.logp == 0).all()) and bool((d == 0).all())


def test_fp32_probabilities_to_the_last_bits(lib):
    """With lse = 0 and a factor of 1 the gradient is [v = y] - exp(l): expf's 2 ulp, 2^-22, however small it is."""
    import torch
    V, T = 1003, 7
    logits = -torch.rand(T, V, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 80.0
    tgt, st = torch.full((T,), 5, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    sl = lib.seq_logits(logits, T, V, V, lib.LSN_DT_F32, tgt, 1, st)
    d = torch.empty(T, V, device="cuda")
    lib.seq_logp_bwd(sl, torch.zeros(T, device="cuda"), torch.ones(1, device="cuda"), None, d, V)
    torch.cuda.synchronize()
    p = logits.double().exp()
    rel = (d.double() + p).abs() / p
    rel[:, 5] = 0
    assert float(rel.max()) <= 2.0 ** -22
    assert float((d[:, 5].double() - (1 - p[:, 5])).abs().max()) <= 2.0 ** -22


@pytest.mark.parametrize("e", [0.0, 0.125])
def test_the_loss_of_exact_ratios(lib, e):
    """No rows: every log-probability is 0 and the ratios are the reference's, exactly.  Loss and gradients are the
    fp64 values rounded once to fp32 (2^-24), where the loss is large as where it all but vanishes."""
    import torch
    h = np.concatenate([np.linspace(-170, 170, 171), [0.0, 1e-9, -1e-9, 1500.0, -1500.0]])
    P, beta = len(h), 0.5
    ref = np.zeros(2 * P)
    ref[1::2] = h                                                # h = (0 - 0) - (0 - ref of the rejected)
    st = torch.zeros(2 * P + 1, dtype=torch.int32, device="cuda")
    sl = lib.seq_logits(None, 0, 64, 64, lib.LSN_DT_F32, None, 2 * P, st)
    f32 = lambda n: torch.full((n,), float("nan"), device="cuda")  # noqa: E731
    loss, dlogp, mean, reward, logp = f32(P), f32(2 * P), f32(1), f32(2 * P), torch.empty(2 * P, dtype=torch.float64, device="cuda")
    n = lib.seq_logp_ws_bytes(sl)
    lib.preference_loss_fwd(sl, torch.from_numpy(ref).cuda(), lib.preference(0, beta, e), None, logp, None, reward, loss, mean, dlogp,
                            torch.zeros(n, dtype=torch.uint8, device="cuda"), n)
    torch.cuda.synchronize()
    z = beta * h
    t = np.exp(-np.abs(z))
    up, down = np.maximum(-z, 0) + np.log1p(t), np.maximum(z, 0) + np.log1p(t)
    sig = lambda v: np.where(v >= 0, 1 / (1 + t), t / (1 + t))  # noqa: E731
    want = (1 - e) * up + e * down
    dw = beta * (e * sig(z) - (1 - e) * sig(-z)) / P
    half = 2.0 ** -24 * 1.001
    assert (np.abs(loss.double().cpu().numpy() - want) <= half * want + 2.0 ** -150).all()
    # with smoothing the two terms cancel in part: what fp64 leaves of either
    assert (np.abs(dlogp.double().cpu().numpy()[0::2] - dw) <= half * np.abs(dw) + 2.0 ** -50 * beta / P * (e > 0) + 2.0 ** -150).all()
    assert torch.equal(dlogp[0::2], -dlogp[1::2])
    assert abs(float(mean) - want.mean()) <= 2.0 ** -23 * want.mean()


@pytest.mark.parametrize("dtype,T,V", [("bf16", 300, 151936), ("fp32", 300, 151936), ("fp32", 500, 60000), ("bf16", 1200, 9000)])
def test_errors_do_not_add_up_over_tokens(lib, dtype, T, V):
    """The error of a long sequence's log-probability, by token: each exponential is 5.2e-8 low on average at most
    (ex2.approx's mean over its arguments) and 1.3e-8 high for each unit below its thread's maximum (fp32's log2 e);
    what scales and joins the sums errs evenly, and all that is random averages out over hundreds of tokens."""
    import torch
    b = Batch(lib, (T - 40, 40), V, dtype=dtype, seed=12, prompt=0.0)
    lib.seq_logp_fwd(b.sl, b.lse, b.logp, b.count, b.ws, b.nws)
    torch.cuda.synchronize()
    want = 0.0
    for t in range(0, T - 40, 100):
        x = b.logits[t:min(t + 100, T - 40), :V].double()
        want += float((x.gather(1, b.tgt[t:t + len(x), None].long())[:, 0] - torch.logsumexp(x, 1)).sum())
    assert abs(float(b.logp[0]) - want) <= (T - 40) * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,pad,offset", [(700, 0, 0), (32003, 5, 3)])
@pytest.mark.parametrize("level", [5000.0, -7e4, -1e9, -1e30, "lowest", 1e10])
def test_gradients_of_rows_far_from_zero(lib, level, V, pad, offset, dtype):
    """Rows of which a mask leaves nothing (all one number), of two numbers, and ordinary ones lifted by 5000: their
    probabilities do not depend on the level.  Apart, in one call and in place: the same bits."""
    import torch
    b = Batch(lib, (6, 8), V, pad, dtype, 2, seed=5, prompt=0.2, offset=offset)
    top = torch.finfo(b.dt).min if level == "lowest" else level
    for t in range(0, b.T - 2, 3):
        b.logits[t, :V] = top
        if t % 2 and level != "lowest":
            b.logits[t, :V // 3] = top * (1 if top < 0 else -1) * 2
    if level == 5000.0:
        b.logits[1:b.T - 2:3, :V] += level
    x = b.logits[:, :V].double()
    p = lib.preference(lib.LSN_PREF_SIGMOID, 0.1)
    d1, d2 = (torch.full((b.T, V + 3), 9.0, dtype=b.dt, device="cuda") for _ in range(2))
    a = b.refd, p, b.lse, b.logp, b.count, b.reward, b.loss, b.mean, b.dlogp
    lib.preference_loss_fwd_bwd(b.sl, *a, d1, V + 3, b.ws, b.nws)
    lib.seq_logp_bwd(b.sl, b.lse, b.dlogp, b.count, d2, V + 3)
    lib.preference_loss_fwd_bwd(b.sl, *a, b.logits, b.ld, b.ws, b.nws)
    torch.cuda.synchronize()
    assert torch.equal(d1, d2) and torch.equal(d1[:, :V], b.logits[:, :V]) and bool((d1[:, V:] == 9).all())
    m = x.amax(1, keepdim=True)
    prob = (x - m).exp()
    prob /= prob.sum(1, keepdim=True)
    on = torch.from_numpy((b.targets >= 0) & (b.targets < V) & (np.arange(b.T) < b.start[-1])).cuda()
    hot = torch.zeros_like(x).scatter_(1, b.tgt.long().clamp(0, V - 1)[:, None], 1.0)
    seq = np.clip(np.searchsorted(b.start, np.arange(b.T), side="right") - 1, 0, b.n - 1)
    c = (b.dlogp.double()[torch.from_numpy(seq).cuda()] * on)[:, None]
    want = c * (hot - prob)
    # the lse of a row below 4096 is off by 2^-13 at most; the argument's roundings, ex2, sums and the output's step
    near = (m[:, 0].abs() < 4096)[:, None] * (m.abs() + 20.0) * 2.0 ** -24
    rel = near + b.tol_s(np.zeros(1)) + 2.0 ** -22 + 2 * (x - m).abs().clamp_max(200) * 1.45 * 2.0 ** -24
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = c.abs() * prob * rel + c.abs() * (hot + prob) * 2.0 ** -23 + want.abs() * half + 1e-37
    bad = ~((d1[:, :V].double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:3])
