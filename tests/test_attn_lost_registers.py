"""The scan for lost registers (test_layer_host.py) on assembly in which the compiler lost some: an excerpt of the attention's
one-launch form for bf16 and 64 channels, as clang 22 of ROCm 7.2 compiled an earlier state of its loop without the empty asm
statement that its values pass through now."""
from test_layer_host import lost_registers

NAME = "_ZN4qlin12_GLOBAL__N_111attn_kernelILi0ELi64ELi8ELb1EEEvNS0_8AttnArgsE:\n"

# v77, v71 and v74 are the second dwords of three tokens' values (s[4:5] .. s[8:9]: live tokens); v71 becomes the
# maximum, v77 and v74 what is left of two p; the byte permutations read all three as values.
LOST = """
	v_mfma_f32_16x16x32_bf16 v[42:45], v[10:13], v[2:5], v[86:89]
	v_cndmask_b32_e64 v76, 0, v76, s[4:5]
	v_cndmask_b32_e64 v70, 0, v70, s[6:7]
	v_cndmask_b32_e64 v75, 0, v75, s[8:9]
	v_cndmask_b32_e64 v77, 0, v77, s[4:5]
	v_cndmask_b32_e64 v71, 0, v71, s[6:7]
	v_cndmask_b32_e64 v74, 0, v74, s[8:9]
	v_perm_b32 v90, v70, v76, s57
	v_cndmask_b32_e32 v71, 0, v55, vcc
	v_sub_f32_e32 v43, v88, v71
	v_exp_f32_e32 v43, v43
	v_sub_f32_e32 v42, v87, v71
	v_exp_f32_e32 v42, v42
	v_cvt_pk_bf16_f32 v45, v43, s0
	v_lshlrev_b32_e32 v45, 16, v45
	v_sub_f32_e32 v77, v43, v45
	v_cvt_pk_bf16_f32 v44, v42, s0
	v_lshlrev_b32_e32 v44, 16, v44
	v_sub_f32_e32 v74, v42, v44
	v_perm_b32 v91, v72, v74, s57
	v_mfma_f32_16x16x32_bf16 v[18:21], v[90:93], v[86:89], v[18:21]
	v_cvt_pk_bf16_f32 v94, v74, v77
	v_mfma_f32_16x16x32_bf16 v[18:21], v[90:93], v[94:97], v[18:21]
	v_perm_b32 v70, v71, v77, s58
	v_mfma_f32_16x16x32_bf16 v[38:41], v[70:73], v[86:89], v[38:41]
	s_endpgm
"""


def test_the_scan_finds_what_the_compiler_lost():
    found = {line for _, line in lost_registers(NAME + LOST)}
    assert found == {"v_perm_b32 v91, v72, v74, s57", "v_perm_b32 v70, v71, v77, s58"}


def test_the_scan_passes_the_same_code_with_registers_of_their_own():
    own = LOST
    for was, now in (("v_sub_f32_e32 v77, v43, v45", "v_sub_f32_e32 v98, v43, v45"), ("v_sub_f32_e32 v74, v42, v44", "v_sub_f32_e32 v99, v42, v44"),
                     ("v_cvt_pk_bf16_f32 v94, v74, v77", "v_cvt_pk_bf16_f32 v94, v99, v98")):
        assert was in own
        own = own.replace(was, now)
    assert not lost_registers(NAME + own)
