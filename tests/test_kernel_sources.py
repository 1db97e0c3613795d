"""Rules of the kernels' sources that no run can show broken: the GPU may order things kindly for years."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_integer_gemm_gb300", "csrc")


def code_of(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["pack_fp4.cu", "moe.cu", "gemm_fp4_kernel.cuh", "gemm_fp4.cuh"])
def test_kernels_set_up_early_make_no_read_only_loads(name):
    # a read-only load, or one through a const restrict pointer, promises that nobody writes the memory during the
    # kernel's life; that of a kernel launched ahead of the end of the one before it begins while that one writes
    code = code_of(name)
    assert "griddepcontrol.wait" in code or "overlap" in code or name == "gemm_fp4.cuh"
    for word in ("__ldg", "__ldcg", "__ldcs", "__restrict__", "ld.global.nc"):
        assert word not in code, word


def test_hand_overs_between_the_ctas_of_a_4_bit_product():
    # mbar_arrive_peer does not release at cluster scope: it may only hand over tensor memory that was read, never
    # shared memory that threads wrote (a pair's scales) or read (the partials of a split k)
    code = code_of("gemm_fp4_kernel.cuh")
    targets = re.findall(r"mbar_arrive_peer\(([^;]*)\);", code)
    assert targets and all(t.startswith("empty_leader") for t in targets), targets
    assert re.search(r"(mbar_arrive_remote|bulk_copy_to_cta)\([^;]*smem_u32\(&red_empty", code)
    # ... and what waits for them acquires at cluster scope
    assert re.search(r"PAIR \? mbar_try_wait_cluster\(c, pc\)", code) and "wait_bounded_cluster(c, pc, wd)" in code
    assert re.search(r"fp4_warp_wait3<PAIR>\([^;]*&sf_full\[", code)
    waits = re.findall(r"(\w+)\(&red_(?:empty|full)\[bar\], rph", code)
    assert len(waits) == 2 and set(waits) == {"fp4_warp_wait_cluster"}


def test_hand_overs_between_the_ctas_of_a_pair():
    # the same in the integer GEMMs' kernel: where the operand comes from TMA its relay may arrive without cluster
    # scope, where threads wrote it (packed weights) it sends a notice that the MMA threads acquire at cluster scope
    code = code_of("gemm_ss_kernel.cuh")
    peers = [m.start() for m in re.finditer(r"mbar_arrive_peer\(", code)]
    assert len(peers) == 2
    relay = [p for p in peers if code[p:].startswith("mbar_arrive_peer(pfull_remote")]
    assert len(relay) == 1 and re.search(r"if constexpr \(kNotice\)\s+bulk_copy_to_cta\([^;]*;\s+else\s+$",
                                         code[:relay[0]])
    assert re.search(r"kNotice\) \{\s+mbar_arrive_expect_tx\(&pfull\[s\], 16\);[^}]*wait_bounded_cluster\(&pfull\[s\]", code)
    assert "kNotice = kPair && Cfg::kPackedP" in code


def test_row_sums_of_the_preparation_pass_are_not_read_through_read_only_loads():
    # that pass and the GEMM overlap, as above (the operands' bytes themselves come by TMA)
    code = code_of("gemm_ss_kernel.cuh")
    assert "prm.sumP" in code and "prm.sumQ" in code
    for word in ("__ldg", "__restrict__", "ld.global.nc"):
        assert word not in code, word


def test_a_split_k_that_gave_up_waits_for_the_partials_on_their_way():
    # a CTA may not leave while another one's st.async may still land in its shared memory: every way out of the
    # epilogue's loop by an expired wait ends in a bounded wait for what the other CTAs send
    code = code_of("gemm_fp4_kernel.cuh")
    epilogue = code[code.index("const uint32_t empty_leader"):code.index("griddepcontrol.launch_dependents")]
    assert "st_async_v4" in epilogue and not re.search(r"wait\w*\([^;]*\)\) break;", epilogue)
    assert epilogue.count("if (!ok) break;") == 3
    drain = epilogue[epilogue.index("if (cs > 1 && !ok)"):]
    assert "&red_full[" in drain and re.search(r"while \(!mbar_try_wait\([^;]*globaltimer_ns\(\) - t0 < prm.limit_ns", drain)


def test_pack_has_no_limit_that_no_call_reaches():
    # K is at most IGEMM_FP4_MAX_K, so the k axis always fits in a grid's second dimension
    code = code_of("pack_fp4.cu")
    assert "65535) return" not in code and re.search(r"static_assert\(IGEMM_FP4_MAX_K[^;]*65535", code)
