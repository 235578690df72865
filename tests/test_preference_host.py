"""Argument checks of the sequence log-probabilities, the preference loss and the gradient norm, on the host alone:
every refusal comes before anything is enqueued."""
import ctypes
import os
import subprocess

import pytest

P = 1 << 20   # an aligned address that is never read
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from layer_streamed_nf4_b200 import build
    build.build()
    from layer_streamed_nf4_b200 import lsnf4
    return lsnf4


def _in(lib, **kw):
    a = dict(logits=P, T=8, V=100, ld=104, dtype=lib.LSN_DT_BF16, targets=P, n_seq=4, seq_start=P, average=False) | kw
    return lib.seq_logits(**a)


FAR = 1 << 30


def _fwd(lib, sl, lse=P, logp=P, count=None, ws=P, n=1 << 30):
    lib.seq_logp_fwd(sl, lse, logp, count, ws, n, stream=0)


def _bwd(lib, sl, lse=P, dlogp=P, count=None, dlogits=FAR, ld_d=100):
    lib.seq_logp_bwd(sl, lse, dlogp, count, dlogits, ld_d, stream=0)


def _loss(lib, sl, p=None, ref=P, lse=P, logp=P, count=P, reward=P, loss=P, mean=P, dlogp=P, ws=P, n=1 << 30):
    lib.preference_loss_fwd(sl, ref, p or lib.preference(lib.LSN_PREF_SIGMOID, 0.1), lse, logp, count, reward, loss, mean, dlogp, ws, n, stream=0)


def _refused(lib, f, *a, **kw):
    with pytest.raises(lib.LsnError) as e:
        f(lib, *a, **kw)
    assert e.value.status == lib.LSN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(T=-1), dict(V=0), dict(ld=99), dict(dtype=2), dict(n_seq=-1), dict(n_seq=0), dict(logits=None), dict(targets=None),
                                dict(seq_start=None), dict(logits=P + 1), dict(targets=P + 2), dict(seq_start=P + 1), dict(T=1 << 31)])
def test_bad_logits(lib, kw):
    sl = _in(lib, **kw)
    for f in (_fwd, _bwd, _loss):
        _refused(lib, f, sl)


def test_bad_dtype_alignment(lib):
    _refused(lib, _fwd, _in(lib, dtype=lib.LSN_DT_F32, logits=P + 2))


@pytest.mark.parametrize("kw", [dict(lse=None), dict(logp=None), dict(logp=P + 4), dict(ws=None), dict(ws=P + 8), dict(n=16)])
def test_bad_forward(lib, kw):
    _refused(lib, _fwd, _in(lib), **kw)


@pytest.mark.parametrize("kw", [dict(lse=None), dict(dlogp=None), dict(dlogits=None), dict(dlogits=FAR + 1), dict(ld_d=99), dict(dlogits=P + 16),
                                dict(dlogits=P)])     # overlapping the logits in part, or in place with another stride
def test_bad_backward(lib, kw):
    _refused(lib, _bwd, _in(lib), **kw)


def test_averages_need_the_counts(lib):
    _refused(lib, _bwd, _in(lib, average=True))


@pytest.mark.parametrize("kw", [dict(loss=None), dict(dlogp=None), dict(lse=None), dict(logp=None), dict(ref=P + 4), dict(reward=P + 2), dict(mean=P + 1)])
def test_bad_loss_tensors(lib, kw):
    _refused(lib, _loss, _in(lib), **kw)


@pytest.mark.parametrize("a", [(7, 0.1), (0, 0.0), (0, -1.0), (0, float("inf")), (0, float("nan")), (0, 0.1, 0.6), (0, 0.1, -0.1), (1, 0.1, 0.1), (2, 0.1, 0.1),
                               (0, 0.1, float("nan")), (0, 0.1, 0.0, float("inf"))])
def test_bad_losses(lib, a):
    _refused(lib, _loss, _in(lib), p=lib.preference(*a))


def test_sequences_come_in_pairs(lib):
    _refused(lib, _loss, _in(lib, n_seq=3))


def test_no_rows_backward_is_a_no_op(lib):
    _bwd(lib, _in(lib, T=0, logits=None, targets=None), lse=None, dlogits=None)


def test_workspace_sizes(lib):
    assert lib.seq_logp_ws_bytes(_in(lib)) >= 8 * 8
    assert lib.seq_logp_ws_bytes(_in(lib, T=5000)) >= 5000 * 8
    assert lib.seq_logp_ws_bytes(_in(lib, T=-1)) == 0 and lib.seq_logp_ws_bytes(_in(lib, V=0)) == 0
    assert lib.grad_ws_bytes([]) > 0 and lib.grad_ws_bytes([0] * 5000) > lib.grad_ws_bytes([0])


def _clip(lib, t, max_norm=1.0, norm=P, ws=P, n=1 << 30):
    lib.grad_clip(t, max_norm, norm, ws, n, stream=0)


def _g(lib, src=P, numel=64, dtype=None, dst=None):
    return lib.grad_tensor(src, numel, lib.LSN_DT_F32 if dtype is None else dtype, dst)


@pytest.mark.parametrize("kw", [dict(src=None), dict(src=P + 2), dict(numel=-1), dict(dtype=5), dict(dst=P + 4), dict(dst=P + 2), dict(dst=P + 128),
                                dict(src=P + 128, dst=P)])
def test_bad_gradients(lib, kw):
    _refused(lib, _clip, [_g(lib), _g(lib, **kw)])


@pytest.mark.parametrize("kw", [dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=float("inf")), dict(max_norm=float("nan")), dict(norm=None),
                                dict(norm=P + 2), dict(ws=None), dict(ws=P + 4), dict(n=100)])
def test_bad_clip_arguments(lib, kw):
    _refused(lib, _clip, [_g(lib)], **kw)


def test_struct_layouts_match_the_header(lib, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "lsnf4.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu %zu %zu %zu\\n", sizeof(lsn_seq_logits), offsetof(lsn_seq_logits, targets),\n'
                   "offsetof(lsn_seq_logits, seq_start), offsetof(lsn_seq_logits, average), sizeof(lsn_preference), sizeof(lsn_grad),\n"
                   "offsetof(lsn_grad, dtype), sizeof(lsn_kernel_timing)); return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    S = lib.SeqLogits
    assert got == [ctypes.sizeof(S), S.targets.offset, S.seq_start.offset, S.average.offset, ctypes.sizeof(lib.Preference), ctypes.sizeof(lib.Grad),
                   lib.Grad.dtype.offset, ctypes.sizeof(lib.KernelTiming)]
