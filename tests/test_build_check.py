"""The build's check of the compiler's assembly: registers saved before the mask of lanes is restored."""

import pytest

from newton_evaluation_nonlinear_amd import _build

JOIN = """_Z6kernelv:
; %bb.0:
	s_and_saveexec_b64 s[0:1], vcc
	s_cbranch_execz .LBB0_2
; %bb.1:
	ds_write_b32 v3, v2
.LBB0_2:                                ; %join
{before}	s_or_b64 exec, exec, s[0:1]
{after}	s_endpgm
"""
SAVE = "\tscratch_store_dwordx2 off, v[190:191], off offset:528 ; 8-byte Folded Spill\n"


@pytest.mark.parametrize("before, after, found", [("", "", []), ("", SAVE, []), (SAVE, "", ["_Z6kernelv"]),
                                                  ("\tv_lshlrev_b32_e32 v34, 3, v0\n" + SAVE, SAVE, ["_Z6kernelv"])])
def test_registers_saved_under_a_narrowed_mask(before, after, found):
    assert _build.lost_lanes(JOIN.format(before=before, after=after).splitlines(True)) == found


def test_a_build_with_lost_lanes_is_refused(tmp_path):
    (tmp_path / "a-hip-amdgcn-amd-amdhsa-gfx950.s").write_text(JOIN.format(before="", after=SAVE))
    _build.check_lanes(str(tmp_path))
    (tmp_path / "b-hip-amdgcn-amd-amdhsa-gfx950.s").write_text(JOIN.format(before=SAVE, after=""))
    with pytest.raises(RuntimeError, match="_Z6kernelv"):
        _build.check_lanes(str(tmp_path))
