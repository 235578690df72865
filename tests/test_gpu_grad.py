"""The global gradient norm and clipping against fp64.  norm: the squares' fp32 sums of four carry 4 roundings
(2^-22 relative), the rest is fp64, the result is rounded once to fp32.  Clipped values: the factor's rounding, the
product's (2^-24 each) and the type's half step."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from layer_streamed_nf4_b200 import lsnf4
    return lsnf4


def make(sizes, types, seed=0, std=1.0, shift=0):
    """Tensors of the sizes, each starting `shift` elements into an allocation of its own."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = torch.float32 if types[i % len(types)] == "fp32" else torch.bfloat16
        out.append((torch.randn(n + shift + 9, generator=g, device="cuda") * std).to(dt)[shift:shift + n])
    return out


def run(lib, src, max_norm=None, dst=None, ws=None, stream=None):
    import torch
    dt = {torch.float32: lib.LSN_DT_F32, torch.bfloat16: lib.LSN_DT_BF16}
    arr = lib.grad_array([lib.grad_tensor(s, s.numel(), dt[s.dtype], None if dst is None else dst[i]) for i, s in enumerate(src)])
    n = lib.grad_ws_bytes(arr)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if ws is None else ws
    norm = torch.full((2,), -1.0, device="cuda")
    if max_norm is None:
        lib.grad_norm(arr, norm, ws, n, stream)
    else:
        lib.grad_clip(arr, max_norm, norm, ws, n, stream)
    torch.cuda.synchronize()
    assert float(norm[1]) == -1.0
    return float(norm[0]), ws


def norm64(src):
    return float(np.sqrt(sum(float(s.double().square().sum()) for s in src)))


def check(src0, got, total, max_norm):
    import torch
    f = min(1.0, max_norm / total)
    for s, g in zip(src0, got):
        want = s.double() * f
        half = 2.0 ** -8 if s.dtype == torch.bfloat16 else 2.0 ** -24
        tol = want.abs() * (0.0 if f == 1.0 else half + 2.0 ** -21) + (0.0 if f == 1.0 else 1e-40)
        assert bool(((g.double() - want).abs() <= tol).all())


SIZES = [[1], [0, 5, 0], [3, 4, 5, 4095, 4096, 4097, 8191, 8193], [100000, 7, 262144], list(range(1, 300)), [17] * 1100 + [5000] * 3, [], [0, 0],
         [2500001]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("types", [("fp32",), ("bf16",), ("fp32", "bf16")])
@pytest.mark.parametrize("shift,ratio", [(0, 0.3), (3, 0.5), (1, 2.0)])
def test_norm_and_clip(lib, sizes, types, shift, ratio):
    import torch
    src = make(sizes, types, seed=len(sizes), shift=shift)
    before = [s.clone() for s in src]
    total = norm64(src)
    got, ws = run(lib, src)
    assert abs(got - total) <= total * 2.0 ** -21
    assert all(torch.equal(a, b) for a, b in zip(src, before))
    max_norm = ratio * total if total > 0 else 1.0
    # apart, at another alignment than the source's
    dst = [torch.full((s.numel() + 12,), 5.0, dtype=s.dtype, device="cuda") for s in src]
    view = [d[4:4 + s.numel()] for d, s in zip(dst, src)]
    got2, _ = run(lib, src, max_norm, view, ws)
    assert got2 == got
    if total > 0:
        check(before, view, total, max_norm)
    for d, s in zip(dst, src):
        assert bool((d[:4] == 5).all()) and bool((d[4 + s.numel():] == 5).all())
    assert all(torch.equal(a, b) for a, b in zip(src, before))
    # in place
    got3, _ = run(lib, src, max_norm, None, ws)
    assert got3 == got
    assert all(torch.equal(a, b) for a, b in zip(src, view))


def test_tensors_of_one_buffer(lib):
    """Tensors that lie end to end, in order, with gaps, out of order, and of two types side by side."""
    import torch
    flat = torch.randn(300000, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    half = flat[200000:].to(torch.bfloat16)
    cuts = [(0, 7), (7, 0), (7, 50001), (50008, 3), (60000, 12345), (72345, 1), (150000, 20000), (100000, 4096), (104096, 1)]
    src = [flat[a:a + n] for a, n in cuts] + [half[:33], half[33:5000], half[5000:5001]]
    total = norm64(src)
    out, outh = torch.zeros_like(flat), torch.zeros_like(half)
    dst = [out[a:a + n] for a, n in cuts] + [outh[:33], outh[33:5000], outh[5000:5001]]
    before = [s.clone() for s in src]
    got, ws = run(lib, src, total / 3, dst)
    assert abs(got - total) <= total * 2.0 ** -21
    check(before, dst, total, total / 3)
    covered = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
    for a, n in cuts:
        covered[a:a + n] = True
    assert bool((out[~covered] == 0).all()) and bool((outh[5001:] == 0).all())
    apart = [torch.empty(n + 4, device="cuda")[4:] for _, n in cuts] + [torch.empty_like(d) for d in dst[-3:]]
    run(lib, src, total / 3, apart, ws)                     # sources end to end, destinations not
    assert all(torch.equal(x, y) for x, y in zip(apart, dst))


def test_more_tensors_than_a_launch_takes(lib):
    src = make([5] * 2500 + [70000], ("fp32", "bf16"), seed=3)
    before = [s.clone() for s in src]
    total = norm64(src)
    got, _ = run(lib, src, total / 2)
    assert abs(got - total) <= total * 2.0 ** -21
    check(before, src, total, total / 2)


def test_values_beyond_the_square_root_of_the_range(lib):
    """Squares that overflow or vanish in fp32."""
    for std in (1e25, 1e-25, 1e-38):
        src = make([5000, 33], ("fp32",), std=std)
        total = norm64(src)
        got, _ = run(lib, src)
        assert abs(got - total) <= total * 2.0 ** -21
        before = [s.clone() for s in src]
        run(lib, src, total / 8)
        check(before, src, total, total / 8)


def test_one_large_value_among_zeros(lib):
    import torch
    src = [torch.zeros(100003, device="cuda"), torch.zeros(5001, dtype=torch.bfloat16, device="cuda")]
    src[0][77777] = -3.0
    src[1][5000] = 4.0
    got, _ = run(lib, src, 2.5)
    assert got == 5.0 and float(src[0][77777]) == -1.5 and float(src[1][5000]) == 2.0
    assert float(src[0].abs().sum()) == 1.5


@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_non_finite_norms_are_reported_and_change_nothing(lib, bad):
    import torch
    src = make([300, 5000], ("fp32", "bf16"))
    src[1][4999] = float(bad)
    before = [s.clone() for s in src]
    got, ws = run(lib, src, 0.1)
    assert np.isnan(got) if bad == "nan" else got == float("inf")
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(src, before))
    src[1][4999] = 1.0                                              # the workspace is fit for the next call
    total = norm64(src)
    got, _ = run(lib, src, 0.1, None, ws)
    assert abs(got - total) <= total * 2.0 ** -21


def test_zero_gradients(lib):
    import torch
    src = [torch.zeros(1000, device="cuda")]
    got, _ = run(lib, src, 1.0)
    assert got == 0.0 and bool((src[0] == 0).all())


def test_reruns_give_the_same_bits(lib):
    import torch
    src = make([123457] * 20, ("fp32", "bf16"))
    dst = [torch.empty_like(s) for s in src]
    ws, first = None, None
    for _ in range(5):
        got, ws = run(lib, src, 10.0, dst, ws)
        now = (got, [d.clone() for d in dst])
        assert first is None or (first[0] == got and all(torch.equal(a, b) for a, b in zip(first[1], now[1])))
        first = now


def test_captured_and_replayed(lib):
    import torch
    src = make([70000, 33, 1025], ("fp32", "bf16", "fp32"))
    arr = lib.grad_array([lib.grad_tensor(s, s.numel(), lib.LSN_DT_F32 if s.dtype == torch.float32 else lib.LSN_DT_BF16) for s in src])
    n = lib.grad_ws_bytes(arr)
    ws, norm = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        lib.grad_clip(arr, 5.0, norm, ws, n, st)
    for k in range(3):
        for i, s in enumerate(src):
            s.copy_(torch.randn(s.numel(), device="cuda", generator=torch.Generator(device="cuda").manual_seed(10 * k + i)) * (0.01 if k == 1 else 1.0))
        before = [s.clone() for s in src]
        total = norm64(src)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert abs(float(norm) - total) <= total * 2.0 ** -21
        check(before, src, total, 5.0)


def test_offsets_beyond_32_bits(lib):
    import torch
    n = (1 << 32) + 4099
    src = [torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
    src[0][-1], src[0][3] = 3.0, 4.0
    got, _ = run(lib, src, 2.5)
    assert got == 5.0 and float(src[0][-1]) == 1.5 and float(src[0][3]) == 2.0


@pytest.mark.parametrize("std", [1e37, 3e37])
def test_a_norm_beyond_fp32_is_infinite(lib, std):
    """Finite gradients whose norm fp32 does not hold: reported as infinite, and nothing is scaled."""
    import torch
    src = make([5000, 33], ("fp32",), std=std)
    src[0].clamp_(-3e38, 3e38)
    assert bool(src[0].isfinite().all()) and norm64(src) > 3.5e38
    before = [s.clone() for s in src]
    dst = [torch.full_like(s, 5.0) for s in src]
    got, _ = run(lib, src, 1.0, dst)
    assert got == float("inf") and all(torch.equal(a, b) for a, b in zip(dst, before))
    got, _ = run(lib, src, 1.0)
    assert got == float("inf") and all(torch.equal(a, b) for a, b in zip(src, before))


@pytest.mark.parametrize("types", [("fp32",), ("fp32", "bf16")])
@pytest.mark.parametrize("max_norm", [1e-3, 1e-7])
def test_a_factor_below_the_normal_range(lib, max_norm, types):
    """A norm of 1e38 brought down to a small one: the factor, below 2^-126, keeps its 24 bits."""
    import torch
    src = make([5000, 333], types, std=1e36)
    before = [s.clone() for s in src]
    total = norm64(src)
    dst = [torch.empty_like(s) for s in src]
    run(lib, src, max_norm, dst)
    check(before, dst, total, max_norm)
    run(lib, src, max_norm)
    check(before, src, total, max_norm)


def test_a_factor_next_to_the_power_of_two(lib):
    """A factor that is 2^-100 but for a part in 2^30: scaled in place like any other."""
    import torch
    src = [torch.full((1,), 2.0 ** 127, device="cuda"), torch.full((4096,), 2.0 ** 100, device="cuda")]
    total = norm64(src)
    max_norm = float(np.nextafter(np.float32(total * 2.0 ** -100), np.float32(0)))
    before = [s.clone() for s in src]
    run(lib, src, max_norm)
    check(before, src, total, max_norm)
