"""The look through the device assembly that every build makes."""
from rank_lm_head_amd.build import lost_lanes

# lanes whose mask is off skip to .LBB0_2, which gives them back with s_or_b64
BODY = """_Z6kernelv:
; %bb.0:
	v_and_b32_e32 v122, 63, v0
	s_and_saveexec_b64 s[4:5], vcc
	s_cbranch_execz .LBB0_2
; %bb.1:
	v_mov_b32_e32 v8, v122
	ds_write_b32 v10, v11
.LBB0_2:                                ; =>This Loop Header: Depth=1
{}	s_or_b64 exec, exec, s[4:5]
	v_mov_b32_e32 v9, v122
	s_endpgm
"""


def test_lanes_back_first():
    for scalar in ("", "\ts_mov_b64 s[72:73], s[30:31]\n", "\tv_writelane_b32 v127, s0, 3\n\ts_waitcnt lgkmcnt(0)\n",
                   "                                        ; implicit-def: $vgpr46\n", "\tv_readlane_b32 s4, v127, 0\n"):
        assert lost_lanes(BODY.format(scalar)) == []


def test_a_copy_or_a_spill_before_the_lanes_are_back():
    for text in ("v_mov_b32_e32 v8, v122", "v_mov_b64_e32 v[8:9], v[122:123]", "scratch_store_dword off, v1, off offset:4",
                 "v_accvgpr_write_b32 a3, v1", "scratch_load_dword v1, off, off"):
        for before in ("", "\ts_mov_b64 s[72:73], s[30:31]\n"):
            found = lost_lanes(BODY.format(f"{before}\t{text}    ; 4-byte Folded Spill\n"))
            assert len(found) == 1 and "_Z6kernelv" in found[0] and text in found[0]


def test_other_blocks_may_begin_with_vector_instructions():
    """Blocks that only scalar branches lead to, and those whose lanes are narrowed further before they come back."""
    scalar = BODY.replace("s_cbranch_execz", "s_cbranch_vccz")
    assert lost_lanes(scalar.format("\tv_mov_b32_e32 v8, v122\n")) == []
    nested = BODY.format("\ts_and_saveexec_b64 s[6:7], vcc\n\tv_mov_b32_e32 v8, v122\n\ts_or_b64 exec, exec, s[6:7]\n")
    assert lost_lanes(nested) == []


def test_else_blocks():
    found = lost_lanes(BODY.format("\tv_mov_b32_e32 v8, v122\n").replace("s_or_b64 exec, exec, s[4:5]",
                                                                         "s_or_saveexec_b64 s[4:5], s[4:5]"))
    assert len(found) == 1
