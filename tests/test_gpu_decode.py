"""Few-token NF4 linears (lora_linear_decode, lora_layer_decode) against a plain fp64 computation from the packed
format.

Tolerance, per output element, from the roundings the header names: the bf16 output, |y| 2^-8; the levels in fp16,
2^-11 of sum |w x|; fp32 sums of K terms in 64-blocks, per warp, per CTA and joined, fewer than 4 + 64 + K/64 additions
deep, each 2^-24 of sum |w x| (the adapter's likewise over K and r terms)."""
import numpy as np
import pytest

from layer_streamed_nf4_b200 import synth
from tests.helpers import DeviceNF4, bits_to_device_bf16

pytestmark = pytest.mark.gpu

# Calls of few rounds take one launch, larger ones two (see the kernels): each test below that is about the arithmetic
# runs on shapes of both kinds.  LONG's first projection alone makes a call a large one.
LONG = [(4352, 64, 0), (4352, 192, 0), (256, 320, 1), (4224, 64, 2), (4160, 128, 3), (64, 64, 4), (1088, 64, 5)]
LAYER = [(256, 256, 0), (256, 64, 0), (256, 64, 0), (256, 256, 1), (256, 704, 2), (256, 704, 2), (704, 256, 3)]


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from layer_streamed_nf4_b200 import lsnf4
    return lsnf4


def _levels(lib):
    return np.array(lib.nf4_codebook(), np.float32).astype(np.float64)


def dequant64(lib, dw):
    """level times absmax in fp64, from the arrays as stored."""
    packed, q, s2, off = dw.arrays()
    codes = np.stack([packed >> 4, packed & 15], 1).reshape(-1, 64)
    table = np.array(lib.dq_codebook(), np.float32)
    amax = (table[q] * np.repeat(s2, 256)[:q.size]).astype(np.float32) + off
    return (_levels(lib)[codes] * amax[:, None].astype(np.float64)).reshape(dw.rows, dw.cols)


class Proj:
    def __init__(self, lib, K, N, T, r, seed, adapter=True, x=None):
        import torch
        c = synth.linear_case(T, K, N, r, 16.0, seed=seed)
        self.K, self.N, self.T, self.r, self.scale = K, N, T, r, 1.75
        self.dw = DeviceNF4(N, K).quantize(c.W)
        self.x = x if x is not None else bits_to_device_bf16(c.x)
        self.A = bits_to_device_bf16(c.A) if adapter else None
        self.B = bits_to_device_bf16(c.B) if adapter else None
        self.y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")   # one row behind the last
        self.base = lib.base_nf4(self.dw.w)
        self.W64 = dequant64(lib, self.dw)

    def desc(self, lib):
        return lib.lora_proj(self.base, self.x, self.A, self.B, y=self.y)

    def ref(self):
        x = self.x.double().cpu().numpy()
        with np.errstate(invalid="ignore", over="ignore"):
            y = x @ self.W64.T
            s = np.abs(x) @ np.abs(self.W64).T
            if self.A is not None:
                A, B = self.A.double().cpu().numpy(), self.B.double().cpu().numpy()
                y = y + self.scale * (x @ A.T) @ B.T
                sl = self.scale * (np.abs(x) @ np.abs(A).T) @ np.abs(B).T
            else:
                sl = 0.0
        depth = 4 + 64 + self.K // 64 + 160
        return y, np.abs(y) * 2.0 ** -8 + s * (2.0 ** -11 + depth * 2.0 ** -24) + sl * (depth + self.r) * 2.0 ** -23 + 1e-37

    def check(self, rows=None):
        y, tol = self.ref()
        got = self.y[:self.T].double().cpu().numpy()
        rows = slice(None) if rows is None else rows
        bad = ~(np.abs(got - y)[rows] <= tol[rows])
        assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - y)[rows] / tol[rows])))
        assert bool((self.y[self.T:] == 7.0).all()), "wrote behind the last token"


def _ws(lib, projs, T, r, fill=0xFF):
    import torch
    n = lib.decode_ws_bytes(projs, T, r)
    assert n > 0
    ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
    ws[:256] = 0                                       # the status word; the rest needs no value
    return ws, n


def run_single(lib, p, ws=None, stream=None):
    ws, n = ws or _ws(lib, [p.desc(lib)], p.T, p.r)
    lib.lora_linear_decode(p.base, p.x, p.T, p.A, p.B, p.r, p.scale, p.y, ws, n, stream)
    return ws, n


@pytest.mark.parametrize("K,N", [(64, 64), (128, 192), (448, 64), (64, 1984), (1088, 320), (2048, 256), (4864, 896)])
@pytest.mark.parametrize("T,r", [(1, 8), (2, 64), (7, 24), (8, 16), (9, 16), (16, 40)])
def test_single_linear(lib, K, N, T, r):
    import torch
    p = Proj(lib, K, N, T, r, seed=K + N + T)
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("K,N", [(4160, 64), (4224, 320), (4352, 576), (6464, 192), (8192, 64), (2112, 2048), (64, 19456)])
@pytest.mark.parametrize("T,r", [(1, 8), (2, 64), (3, 24), (8, 16), (9, 16), (16, 40)])
def test_single_linear_of_the_large_kind(lib, K, N, T, r):
    """Rows of 65, 66, 68, 101, 128, 33 and 1 blocks: stages that end inside a row, groups of 256 constants that end
    inside a stage, rows of codes that start at every alignment."""
    import torch
    p = Proj(lib, K, N, T, r, seed=K + N + T)
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("K,N", [(576, 448), (4224, 448)])
@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count_with_the_adapter_off(lib, T, K, N):
    import torch
    p = Proj(lib, K, N, T, 16, seed=T, adapter=False)
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("name,K,N,T", [("8b q", 4096, 4096, 1), ("8b down", 14336, 4096, 3), ("8b k", 4096, 1024, 16),
                                        ("72b down", 29568, 8192, 8), ("0.5b gate", 896, 4864, 1)])
def test_full_size(lib, name, K, N, T):
    import torch
    p = Proj(lib, K, N, T, 16, seed=11)
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


def _layer(lib, shapes, T, r, adapter, seed=5):
    xs, projs = {}, []
    for i, (K, N, xi) in enumerate(shapes):
        on = adapter if isinstance(adapter, bool) else adapter[i]
        p = Proj(lib, K, N, T, r, seed=seed + i, adapter=on, x=xs.get(xi))
        xs.setdefault(xi, p.x)
        projs.append(p)
    return projs


def run_layer(lib, projs, ws=None, stream=None):
    arr = lib.proj_array([p.desc(lib) for p in projs])
    T, r = projs[0].T, projs[0].r
    ws, n = ws or _ws(lib, arr, T, r)
    lib.lora_layer_decode(arr, T, r, projs[0].scale, ws, n, stream)
    return ws, n


@pytest.mark.parametrize("T,r,adapter", [(1, 16, True), (1, 16, False), (5, 8, True), (13, 64, True),
                                         (4, 16, (True, False, True, False, False, True, True))])
@pytest.mark.parametrize("shapes", [LAYER, LONG], ids=["small", "large"])
def test_layer(lib, shapes, T, r, adapter):
    import torch
    projs = _layer(lib, shapes, T, r, adapter)
    run_layer(lib, projs)
    torch.cuda.synchronize()
    for p in projs:
        p.check()


def test_sixteen_projections_of_one_input(lib):
    import torch
    projs = _layer(lib, [(192, 64 * (1 + i % 5), 0) for i in range(16)], 3, 8, True)
    run_layer(lib, projs)
    torch.cuda.synchronize()
    for p in projs:
        p.check()


def test_layer_of_the_8b_shapes(lib):
    import torch
    h, kv, m = 4096, 1024, 14336
    projs = _layer(lib, [(h, h, 0), (h, kv, 0), (h, kv, 0), (h, h, 1), (h, m, 2), (h, m, 2), (m, h, 3)], 1, 16, True)
    ws = run_layer(lib, projs)
    torch.cuda.synchronize()
    first = [p.y.clone() for p in projs]
    for p in projs:
        p.check()
    for _ in range(3):                                 # the same workspace again: the same bits
        for p in projs:
            p.y[:p.T] = 0
        run_layer(lib, projs, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(p.y, f) for p, f in zip(projs, first))


def test_agrees_with_the_training_forward(lib):
    """lora_linear_fwd on the same inputs: its weights (2^-8 of each product), its LoRA operand and output are
    rounded to bf16, so the two lie within the sum of both tolerances."""
    import torch
    p = Proj(lib, 512, 512, 5, 8, seed=3)
    n = lib.lora_ws_bytes(5, 512, 512, 8, lib.LSN_BASE_NF4)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    y = torch.empty(5, 512, dtype=torch.bfloat16, device="cuda")
    lib.lora_linear_fwd(p.base, p.x, 5, p.A, p.B, 8, p.scale, y, ws, n)
    run_single(lib, p)
    torch.cuda.synchronize()
    _, tol = p.ref()
    x = p.x.double().abs().cpu().numpy()
    s = x @ np.abs(p.W64).T
    sl = p.scale * (x @ p.A.double().abs().cpu().numpy().T) @ p.B.double().abs().cpu().numpy().T
    diff = np.abs(y.double().cpu().numpy() - p.y[:5].double().cpu().numpy())
    assert (diff <= 2 * tol + (s + sl) * 2.0 ** -8).all()


@pytest.mark.parametrize("K", [320, 4160])
@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-5, 1e4, 1e30])
def test_inputs_of_any_magnitude(lib, std, K):
    import torch
    p = Proj(lib, K, 128, 3, 8, seed=2)
    p.x.copy_((p.x.float() * std).to(torch.bfloat16))
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("K", [256, 4224])
def test_outliers_beside_small_values(lib, K):
    """One value 2^20 times the others in a block: the small ones still count in full (2^-28 of the largest)."""
    import torch
    p = Proj(lib, K, 64, 2, 8, seed=4, adapter=False)
    p.x[:, 17] *= 2.0 ** 20
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()
    big = p.y.clone()
    p.x[:, 17] = 0
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()
    assert not torch.equal(big, p.y)


@pytest.mark.parametrize("K", [320, 4160])
def test_non_finite_and_zero_inputs_stay_in_their_token(lib, K):
    import torch
    p = Proj(lib, K, 128, 6, 8, seed=9)
    p.x[1, 70] = float("inf")
    p.x[3, 5] = float("nan")
    p.x[4] = 0
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check(rows=[0, 2, 4, 5])
    y, _ = p.ref()
    got = p.y[:6].float().cpu().numpy()
    assert not np.isfinite(got[1]).any() and np.isnan(got[3]).all()
    # through the adapter (u holds infinities of both signs) every output of the token is NaN, here as by the formula
    assert np.isnan(y[1]).all() and np.isnan(got[1]).all()
    assert (got[4] == 0).all()


@pytest.mark.parametrize("K,T", [(320, 3), (4160, 3), (4160, 2)])
def test_infinity_without_an_adapter_keeps_its_sign(lib, K, T):
    """Infinity times a weight is infinite with the weight's sign, times a zero weight NaN."""
    import torch
    p = Proj(lib, K, 128, T, 8, seed=9, adapter=False)
    p.x[1, 70] = float("inf")
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check(rows=[0, 2] if T > 2 else [0])
    y, _ = p.ref()
    got = p.y[1].float().cpu().numpy()
    assert np.isinf(y[1]).any() and np.array_equal(np.isnan(got), np.isnan(y[1]))
    assert np.array_equal(got[np.isinf(y[1])], y[1][np.isinf(y[1])])


@pytest.mark.parametrize("K", [256, 4224])
def test_zero_blocks_and_zero_offset_weights(lib, K):
    import torch
    p = Proj(lib, K, 64, 2, 8, seed=1)
    W = synth.normal_f32((64, K), 0.02, 1, 2)
    W[3] = 0
    W[:, 64:128] = 0
    p.dw.quantize(W)
    p.W64 = dequant64(lib, p.dw)
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("K", [128, 4352])
def test_second_level_codes_of_255_stand_for_zero(lib, K):
    """The table's entry 255 is 0 like entry 127 (the codec never writes it; a weight from elsewhere may hold it)."""
    import torch
    p = Proj(lib, K, 64, 3, 8, seed=8, adapter=False)
    o, n = p.dw.layout, 64 * K // 64
    q = p.dw.blob[o[1]:o[1] + n]
    q[::3] = 255
    p.W64 = dequant64(lib, p.dw)
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


def test_zero_tokens(lib):
    import torch
    p = Proj(lib, 128, 64, 1, 8, seed=1)
    lib.lora_linear_decode(p.base, None, 0, p.A, p.B, 8, 1.0, None, None, 0)
    torch.cuda.synchronize()
    assert bool((p.y == 7.0).all())


@pytest.mark.parametrize("K", [448, 4352])
def test_constants_apart_and_unaligned(lib, K):
    """The four arrays of a weight lie apart, the byte codes of the absmax at an odd address."""
    import torch
    p = Proj(lib, K, 192, 3, 8, seed=8)
    packed, q, s2, off = p.dw.arrays()
    qb = torch.zeros(q.size + 1, dtype=torch.uint8, device="cuda")
    qb[1:] = torch.from_numpy(q)
    keep = [torch.from_numpy(packed).cuda(), qb, torch.from_numpy(s2).cuda(), torch.tensor([off], device="cuda")]
    p.base = lib.base_nf4(lib.make_nf4_weight(192, K, keep[0], qb.data_ptr() + 1, keep[2], keep[3]))
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("shapes", [LAYER, LONG], ids=["small", "large"])
def test_captured_and_replayed_on_another_stream(lib, shapes):
    import torch
    projs = _layer(lib, shapes, 2, 16, True)
    ws = run_layer(lib, projs)                          # first use outside the capture
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        run_layer(lib, projs, ws, st)
        run_layer(lib, projs, ws, st)                   # two calls in a row share the workspace
    new = {}
    for i, p in enumerate(projs):                       # new inputs for the replay
        if id(p.x) not in new:
            new[id(p.x)] = True
            p.x.copy_(synth.device_normal(tuple(p.x.shape), 1.0, 77, i, device="cuda", dtype=torch.bfloat16))
        p.y[:2] = 0
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for p in projs:
        p.check()


def test_two_streams_with_a_workspace_each(lib):
    import torch
    a, b = Proj(lib, 4096, 1024, 1, 16, seed=1), Proj(lib, 4096, 1024, 9, 16, seed=2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = _ws(lib, [a.desc(lib)], 1, 16), _ws(lib, [b.desc(lib)], 9, 16)
    torch.cuda.synchronize()
    for _ in range(20):
        run_single(lib, a, wa, sa)
        run_single(lib, b, wb, sb)
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("T,H", [(4, 512), (2, 4352), (9, 2112)])
def test_chained_calls_read_what_the_call_before_wrote(lib, T, H):
    """The output of one call is the next one's input, with no other work between them on the stream."""
    import torch
    a, b = Proj(lib, H, H, T, 16, seed=21), Proj(lib, H, H, T, 16, seed=22)
    ws = _ws(lib, [a.desc(lib)], T, 16)
    torch.cuda.synchronize()
    b.x = a.y[:T]
    for _ in range(10):
        run_single(lib, a, ws)
        run_single(lib, b, ws)
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("K", [1024, 4160])
@pytest.mark.parametrize("pdl", [0, 1])
def test_dependent_launch_option(lib, pdl, K):
    import torch
    from tests.helpers import lib_option
    with lib_option(lib, lib.LSN_OPT_PDL, pdl):
        p = Proj(lib, K, 512, 2, 16, seed=6)
        run_single(lib, p)
        torch.cuda.synchronize()
        p.check()


@pytest.mark.parametrize("K,kernels", [(256, 1), (4160, 2)])
def test_timing_counts_the_calls(lib, K, kernels):
    import torch
    p = Proj(lib, K, 256, 1, 8, seed=1)
    lib.timing_enable(True)
    run_single(lib, p)
    torch.cuda.synchronize()
    t = lib.timing_read()
    lib.timing_enable(False)
    assert t["decode"]["launches"] == 1 and t["decode"]["kernels"] == kernels and t["decode"]["ms"] > 0


@pytest.mark.parametrize("T", [1, 16])
def test_offsets_beyond_32_bits(lib, T):
    """Rows of 2^27 + 128 weights: 16 tokens of them are over 2^32 bytes, laid out and read.  x is zero but for the
    first and the last block, so that these alone make the outputs."""
    import torch
    K, N = (1 << 27) + 128, 64
    nb = K // 64
    g = torch.Generator(device="cuda").manual_seed(3)
    packed = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    q = torch.randint(100, 156, (N, nb), dtype=torch.uint8, device="cuda", generator=g)
    s2 = torch.rand((N * nb + 255) // 256, device="cuda", generator=g) * 0.01
    off = torch.full((1,), 0.05, device="cuda")
    base = lib.base_nf4(lib.make_nf4_weight(N, K, packed, q, s2, off))
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[:, :64].normal_(generator=g)
    x[:, -64:].normal_(generator=g)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    d = lib.lora_proj(base, x, None, None, y=y)
    ws, n = _ws(lib, [d], T, 8)
    lib.lora_linear_decode(base, x, T, None, None, 8, 1.0, y, ws, n)
    torch.cuda.synchronize()
    lib.ws_status(ws)
    lv = torch.from_numpy(_levels(lib)).cuda()
    want, tol = 0.0, 0.0
    for b in (0, nb - 1):
        c = packed[:, 32 * b:32 * b + 32].long()
        blk = torch.arange(N, device="cuda") * nb + b
        am = (q[:, b].double() - 127) / 127 * s2[blk // 256].double() + 0.05
        W = torch.stack([lv[c // 16], lv[c % 16]], 2).view(N, 64) * am[:, None]
        want = want + x[:, 64 * b:64 * b + 64].double() @ W.T
        tol = tol + x[:, 64 * b:64 * b + 64].double().abs() @ W.abs().T
    tol = tol * (2.0 ** -11 + 300 * 2.0 ** -24) + want.abs() * 2.0 ** -8
    assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("K", [256, 4224])
@pytest.mark.parametrize("up", [28, 33, 38])
def test_values_far_below_the_largest_of_their_block(lib, K, up):
    """One value 2^up times the others in a block, against weights of zero: the others count exactly down to 2^-31 of
    the largest, and are off by at most 2^-39 of it each below that."""
    import torch
    p = Proj(lib, K, 64, 3, 8, seed=4, adapter=False)
    W = synth.normal_f32((64, K), 0.02, 1, 2)
    W[:, 17] = 0
    p.dw.quantize(W)
    p.W64 = dequant64(lib, p.dw)
    assert (p.W64[:, 17] == 0).all()
    p.x[:, 17] = 2.0 ** up * 4
    run_single(lib, p)
    torch.cuda.synchronize()
    x = p.x.double().cpu().numpy()
    x[:, 17] = 0
    y, s = x @ p.W64.T, np.abs(x) @ np.abs(p.W64).T
    lost = np.where(np.abs(x[:, :64]) < 2.0 ** (up + 2 - 31), 2.0 ** (up + 2 - 39), 0.0) @ np.abs(p.W64[:, :64]).T
    tol = np.abs(y) * 2.0 ** -8 + s * (2.0 ** -11 + (228 + K // 64) * 2.0 ** -24) + lost * (1 + 2.0 ** -7) + 1e-37
    got = p.y[:3].double().cpu().numpy()
    assert (np.abs(got - y) <= tol).all(), float(np.max(np.abs(got - y) / tol))


@pytest.mark.parametrize("K", [256, 4224])
@pytest.mark.parametrize("T", [1, 2, 5, 11])
def test_a_block_of_the_largest_inputs(lib, T, K):
    """A block of values of 1e38: its sum with the levels alone leaves fp32's range, with the absmax it does not."""
    import torch
    p = Proj(lib, K, 64, T, 8, seed=40, adapter=False)
    p.x[:, 64:128] = torch.where(p.x[:, 64:128] > 0, 1e38, -1e38)
    run_single(lib, p)
    torch.cuda.synchronize()
    p.check()
