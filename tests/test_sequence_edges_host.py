"""Refusals of the sequence-layer entries at extreme sizes and arguments, without a GPU (placeholder addresses; nothing is
dereferenced)."""

import os
import subprocess
import sys

import pytest

import newton_evaluation_nonlinear_amd as pn
from test_sequence_host import GIB, TOK, _attention_block, _no_error_left, _rotary_block, _step_block  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("sizes, backward", [(dict(B=1 << 24, H=1, HK=1, T=1, dk=1, dv=1), True),
                                             (dict(B=1 << 12, H=1 << 12, HK=1, T=1, dk=8, dv=130), False),
                                             (dict(B=1 << 12, H=1 << 10, HK=1, T=1, dk=200, dv=8), True)])
def test_launches_past_2_32_threads_are_refused_first(sizes, backward):
    """What no launch can hold is an error of the arguments, found before any work is queued."""
    lib = pn.lib()
    far = TOK(4, 8, 8, 8), TOK(5, 8, 8, 8), TOK(6, 8, 8, 8)
    block = _attention_block(dtype=1, q=far[0], k=far[1], v=far[2], **sizes)
    f = lib.pn_linear_attention_backward if backward else lib.pn_linear_attention
    assert f(block) == pn.EUNSUPPORTED and pn.last_error() != ""
    assert lib.pn_linear_attention_workspace_bytes(block, int(backward)) == 0 and pn.last_error() != ""


def test_steps_past_2_32_threads_are_refused():
    f = pn.lib().pn_linear_attention_step
    assert f(_step_block(B=1 << 24, H=1, HK=1, dk=1, dv=1, n_slots=1 << 24)) == pn.EUNSUPPORTED
    assert f(_step_block(B=1 << 12, H=1 << 12, HK=1, dk=1, dv=1, n_slots=1 << 12)) == pn.EUNSUPPORTED


@pytest.mark.parametrize("at", [4, 5, 6, 7, 8, 9, 10, 12, 14, 15])
def test_norm_gradients_refuse_a_workspace_over_other_arrays(at):
    kw = dict(qw=12 * GIB, kw=12 * GIB + 4096, dqw=14 * GIB, dkw=15 * GIB)
    n = pn.lib().pn_qk_norm_rotary_workspace_bytes(_rotary_block(**kw))
    assert pn.lib().pn_qk_norm_rotary_backward(_rotary_block(**kw, ws=at * GIB, wsn=n)) == pn.EINVAL
    assert "overlaps" in pn.last_error()


@pytest.mark.parametrize("kw", [dict(pos=12 * GIB, pos64=2), dict(pos=12 * GIB + 4, pos64=1), dict(pos=12 * GIB, pst=-1),
                                dict(pos=12 * GIB, psb=1 << 41), dict(pos=6 * GIB)])
def test_positions_are_checked_without_a_rotation_too(kw):
    for name in ("pn_rotary", "pn_qk_norm_rotary", "pn_qk_norm_rotary_backward"):
        assert getattr(pn.lib(), name)(_rotary_block(R=0, **kw)) == pn.EINVAL, name


def test_import_needs_no_cuda_build_of_torch():
    """The package loads, and its helpers of plain numbers work, on a torch that lacks the device bindings."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "import newton_evaluation_nonlinear_amd as pn\n"
            "assert pn.rotary_frequencies(4)[0] == 1.0 and pn.param_count(pn.CELL_DIAG_TANH, 5, 1) == 5\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
