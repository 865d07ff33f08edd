"""The rotation's arguments at the edge of what the library's types hold."""
import copy
import ctypes
import pickle

import pytest
import torch

from sliding_window_global_b200 import Rotary, SwaError, load_library, rotary_frequencies
from sliding_window_global_b200.rotary import RotaryArgs, RotaryBackwardArgs
from tests.test_rotary import _args

INVALID = 1


@pytest.mark.parametrize("cls,entry", [(RotaryArgs, "swa_rotary_forward"), (RotaryBackwardArgs, "swa_rotary_backward")])
def test_positions_that_pass_int32_are_refused(cls, entry):
    """start, start + 1, ... must not wrap to negative positions."""
    call = getattr(load_library(), entry)
    for start, n in ((2 ** 31 - 1, 2), (2 ** 31 - 5, 6), (1, 2 ** 31 - 65)):
        assert call(ctypes.byref(_args(cls, start=start, seq_len=n)), None) == INVALID


@pytest.mark.gpu
def test_the_last_positions():
    """start up to the last int32, and a start that is not used beside positions."""
    g = torch.Generator().manual_seed(67)
    r = Rotary(64)
    x = torch.randn((1, 2, 9, 64), generator=g).cuda()
    pos = (2 ** 31 - 9 + torch.arange(9)).to(torch.int32)[None].cuda()
    want, _ = r.forward(x, positions=pos)
    assert torch.equal(r.forward(x, start=2 ** 31 - 9)[0], want)
    assert torch.equal(r.forward(x, positions=pos, start=2 ** 31 - 1)[0], want)
    assert torch.equal(r.backward(x, start=2 ** 31 - 9)[0], r.backward(x, positions=pos, start=2 ** 31 - 1)[0])
    for call in (r.forward, r.backward):
        with pytest.raises(SwaError) as e:
            call(x, start=2 ** 31 - 8)
        assert e.value.status == INVALID


@pytest.mark.parametrize("cls,entry", [(RotaryArgs, "swa_rotary_forward"), (RotaryBackwardArgs, "swa_rotary_backward")])
@pytest.mark.parametrize("empty", [dict(batch=0), dict(seq_len=0)])
def test_a_call_without_rows_has_no_status_of_others(cls, entry, empty):
    """Nothing is launched, so nothing that the CUDA runtime remembers is reported (here: that
    there is no device)."""
    assert getattr(load_library(), entry)(ctypes.byref(_args(cls, start=2 ** 31 - 1, **empty)), None) == 0


@pytest.mark.parametrize("amplitude", [1e-50, -1e-46, 1e39, -1e300])
def test_amplitudes_that_fp32_does_not_hold_are_refused(amplitude):
    """Rounded to 0 an amplitude would stand for the default, 1."""
    with pytest.raises(ValueError):
        Rotary(64, amplitude=amplitude)
    assert Rotary(64, amplitude=1e-40).amplitude == 1e-40


def test_a_rotation_can_be_copied_and_pickled():
    """As a module that holds one is."""
    freq, amp = rotary_frequencies(48, scaling="yarn", factor=8.0)
    r = Rotary(64, rotary_dim=48, interleaved=False, frequencies=freq, amplitude=amp)
    for other in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert isinstance(other, Rotary) and other is not r
        assert (other.head_dim, other.rotary_dim, other.interleaved, other.amplitude) == (64, 48, False, amp)
        at, size = other.fields[2], 24
        assert list((ctypes.c_double * size).from_address(at)) == freq.tolist()
    assert copy.deepcopy(Rotary(128, rotary_dim=0)).rotary_dim == 0
