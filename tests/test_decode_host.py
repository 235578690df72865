"""Argument checks of the few-token NF4 linears, on the host alone: every refusal comes before anything is enqueued."""
import pytest

P = 1 << 20   # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from layer_streamed_nf4_b200 import build
    build.build()
    from layer_streamed_nf4_b200 import lsnf4
    return lsnf4


def _base(lib, N=128, K=256, **kw):
    a = dict(packed=P, absmax_q=P, absmax_s2=P, offset=P) | kw
    return lib.base_nf4(lib.make_nf4_weight(N, K, *a.values()))


def _call(lib, base=None, x=P, T=1, A=P, B=P, r=8, y=P, ws=P, n=1 << 40):
    lib.lora_linear_decode(_base(lib) if base is None else base, x, T, A, B, r, 1.0, y, ws, n, stream=0)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=17), dict(r=0), dict(r=4), dict(r=12), dict(r=72), dict(x=None), dict(x=P + 2), dict(y=None),
                                dict(y=P + 8), dict(A=None), dict(B=None), dict(A=P + 4), dict(ws=None), dict(ws=P + 4), dict(n=64)])
def test_bad_arguments(lib, kw):
    with pytest.raises(lib.LsnError) as e:
        _call(lib, **kw)
    assert e.value.status == lib.LSN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(N=96), dict(K=100), dict(N=0), dict(packed=None), dict(packed=P + 8), dict(offset=P + 2), dict(absmax_s2=None)])
def test_bad_weights(lib, kw):
    with pytest.raises(lib.LsnError) as e:
        _call(lib, base=_base(lib, **kw))
    assert e.value.status == lib.LSN_ERR_INVALID_ARG


def test_bf16_bases_are_not_supported(lib):
    with pytest.raises(lib.LsnError) as e:
        _call(lib, base=lib.base_bf16(P, 128, 256))
    assert e.value.status == lib.LSN_ERR_UNSUPPORTED


def test_layer_calls_check_every_projection(lib):
    good = lib.lora_proj(_base(lib), P, P, P, y=P)
    bad = lib.lora_proj(_base(lib), P, P, None, y=P)
    with pytest.raises(lib.LsnError) as e:
        lib.lora_layer_decode([good, bad], 1, 8, 1.0, P, 1 << 40, stream=0)
    assert e.value.status == lib.LSN_ERR_INVALID_ARG and "projection 1" in str(e.value)
    with pytest.raises(lib.LsnError):
        lib.lora_layer_decode([good] * 17, 1, 8, 1.0, P, 1 << 40, stream=0)


def test_no_tokens_is_a_no_op(lib):
    _call(lib, x=None, T=0, y=None, ws=None, n=0)


def test_workspace_sizes(lib):
    d = lambda K, N: lib.lora_proj(_base(lib, N=N, K=K), P, P, P, y=P)  # noqa: E731
    one = lib.decode_ws_bytes([d(4096, 4096)], 1, 16)
    assert one >= 4096 * 2 + 16 * 4
    assert lib.decode_ws_bytes([d(4096, 4096)], 16, 16) >= 16 * 4096 * 2
    assert lib.decode_ws_bytes([d(4096, 4096)] * 3, 1, 16) >= one + 2 * (4096 * 2 + 16 * 4)
    assert lib.decode_ws_bytes([d(4096, 4096)], 17, 16) == 0 and lib.decode_ws_bytes([d(4096, 4096)], 1, 12) == 0
