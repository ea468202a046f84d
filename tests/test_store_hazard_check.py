"""The build's scan for stores whose data the next instruction overwrites (selective_state_space_33_amd/build.py,
store_hazards) on small assembly texts."""
import pytest

from selective_state_space_33_amd.build import store_hazards

WIDE = "\tbuffer_store_dwordx4 v[42:45], v137, s[28:31], s18 offen\n"


@pytest.mark.parametrize("store,write", [
    (WIDE, "\tv_accvgpr_read_b32 v42, a12\n"),
    (WIDE, "\tv_mul_f32_e32 v45, v1, v2\n"),
    (WIDE, "\tv_pk_mul_f16 v[44:47], v[0:3], v[0:3]\n"),
    ("\tglobal_store_dwordx4 v[0:1], v[4:7], off\n", "\tv_mov_b32_e32 v5, 0\n"),
    ("\tbuffer_store_dwordx3 v[4:6], v1, s[0:3], 0 offen\n", "\t; a comment\n.LBB0_1:\n\tv_mov_b32_e32 v6, 0\n"),
])
def test_overwritten_data_is_found(store, write):
    assert len(store_hazards(store + write)) == 1


@pytest.mark.parametrize("store,behind", [
    (WIDE, "\ts_nop 0\n\tv_accvgpr_read_b32 v42, a12\n"),             # an instruction between
    (WIDE, "\tv_mul_f32_e32 v46, v42, v43\n"),                         # reads them
    (WIDE, "\tv_cmp_gt_f32_e32 vcc, v42, v43\n"),
    (WIDE, "\tv_mov_b32_e32 v137, 0\n"),                               # the address
    ("\tbuffer_store_dwordx2 v[42:43], v137, s[28:31], s18 offen\n", "\tv_mov_b32_e32 v42, 0\n"),   # 8 bytes
    ("\tglobal_store_dwordx4 v[4:5], v[0:3], off\n", "\tv_mov_b32_e32 v5, 0\n"),
])
def test_others_are_not(store, behind):
    assert store_hazards(store + behind) == []
