"""Host logic of the stack's few-token forward and of the preference step, on CPU: the pool's slots over decode()
sweeps, and the refusals of decode() and Preference."""
import pytest
import torch

from layer_streamed_nf4_b200 import lsnf4
from layer_streamed_nf4_b200.stack import Preference
from tests.test_stack_window_cpu import _cpu_stack


@pytest.mark.parametrize("ahead", [True, False])
@pytest.mark.parametrize("L,S", [(1, 1), (2, 2), (5, 1), (5, 2), (8, 5), (6, 6), (4, 7)])
def test_decode_sweeps_the_layers_in_order(monkeypatch, L, S, ahead):
    """A few-token forward acquires each layer once, in order, releases it, and reads the layers that the last sweep
    did not leave resident; between training steps the pool stays consistent."""
    st, pool = _cpu_stack(monkeypatch, L, S, ahead)
    for k in range(3):
        a0, c0 = len(pool.acquired), pool.copies
        st.decode(adapter=k % 2 == 0)
        assert pool.acquired[a0:] == list(range(L)) and sum(pool.refs) == 0
        assert pool.copies - c0 <= L
    st.step(reference=True)
    st.decode()
    assert sum(pool.refs) == 0


def test_decode_refusals(monkeypatch):
    st, _ = _cpu_stack(monkeypatch, 2, 2, False)
    st.T = lsnf4.LSN_DECODE_MAX_T + 1
    with pytest.raises(AssertionError):
        st.decode()
    st.T, st.nf4 = 4, False
    with pytest.raises(AssertionError):
        st.decode()


@pytest.mark.parametrize("bad", ["vocab", "targets type", "targets size", "start type", "odd sequences", "one sequence", "api", "shared dY"])
def test_preference_refusals(monkeypatch, bad):
    st, _ = _cpu_stack(monkeypatch, 2, 2, False)
    a = dict(vocab=128, targets=torch.zeros(st.T, dtype=torch.int32), seq_start=torch.tensor([0, 2, 4], dtype=torch.int32), beta=0.1)
    if bad == "vocab":
        a["vocab"] = 100
    if bad == "targets type":
        a["targets"] = a["targets"].long()
    if bad == "targets size":
        a["targets"] = a["targets"][:-1]
    if bad == "start type":
        a["seq_start"] = a["seq_start"].long()
    if bad == "odd sequences":
        a["seq_start"] = torch.tensor([0, 1, 2, 4], dtype=torch.int32)
    if bad == "one sequence":
        a["seq_start"] = torch.tensor([0, 4], dtype=torch.int32)
    if bad == "api":
        st.api = "proj"
    if bad == "shared dY":
        st._distinct = False
    with pytest.raises(ValueError):
        Preference(st, **a)


class _FakeStatus:
    """ws_status on host memory: a non-zero first word is cleared and raised."""

    def __init__(self):
        self.read = []

    def __call__(self, ws, stream=None):
        self.read.append(ws.data_ptr())
        word = ws[:4].view(torch.int32)
        if int(word):
            word.zero_()
            raise lsnf4.LsnError(lsnf4.LSN_ERR_TIMEOUT, "fake status", "gave up")


@pytest.mark.parametrize("where", ["decode", "head", "sweeps", "head of a second loss"])
def test_check_status_reads_every_workspace(monkeypatch, where):
    st, _ = _cpu_stack(monkeypatch, 2, 2, False)
    status = _FakeStatus()
    monkeypatch.setattr(lsnf4, "ws_status", status)
    st.ws = [torch.zeros(256, dtype=torch.uint8)]
    st.check_status()                                   # before any decode() or loss
    st._decode_ws = torch.zeros(256, dtype=torch.uint8)
    losses = []
    for _ in range(2):
        pr = Preference.__new__(Preference)
        pr.stack, pr._hws = st, torch.zeros(256, dtype=torch.uint8)
        pr._register()
        losses.append(pr)
    st.check_status()
    bad = {"decode": st._decode_ws, "head": losses[0]._hws, "sweeps": st.ws[0], "head of a second loss": losses[1]._hws}[where]
    bad[2] = 1
    with pytest.raises(lsnf4.LsnError):
        st.check_status()
    st.check_status()
    assert not st._copy()._preferences and st._copy()._decode_ws is None
    losses.clear()                                      # a loss that is gone is not asked any more
    del pr, bad
    status.read.clear()
    st.check_status()
    assert len(status.read) == 2
