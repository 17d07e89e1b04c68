"""The build's checks of the generated code around matrix instructions that the
compiler does not see into: on small listings, and on the built library."""
import re

from moe_ragged_bf16_amd import build

HEAD = "0000000000001000 <kernel>:\n"
MFMA = "v_mfma_scale_f32_16x16x128_f8f6f4 v[40:43], v[8:15], v[16:23], v[40:43], v30, v31 op_sel_hi:[0,0,0]"


def listing(*lines):
    """A function of 8-byte instructions; "->n" marks a branch to line n."""
    out = []
    for i, line in enumerate(lines):
        text, _, target = line.partition("->")
        comment = "// %012X: 00000000" % (0x1000 + 8 * i)
        if target:
            n = int(target)
            comment += " <kernel+0x%x>" % (8 * n) if n else " <kernel>"
        out.append("\t%s  %s" % (text.strip(), comment))
    return HEAD + "\n".join(out) + "\n"


NOPS = ["s_nop 10"]                                       # 11 wait states


def test_results_are_left_alone_until_they_are_there():
    bad = lambda *lines: build.mfma_result_hazards(listing(MFMA, *lines))
    assert bad("v_mov_b32_e32 v1, v41")
    assert bad(*NOPS, "v_cvt_pk_bf16_f32 v5, v42, s0")
    assert not bad(*NOPS, "s_mov_b32 s0, s1", "v_cvt_pk_bf16_f32 v5, v42, s0")
    assert not bad("s_nop 15", "ds_write_b128 v2, v[40:43]")
    assert bad("s_nop 7", "ds_write_b128 v2, v[40:43]") and bad("v_mov_b32_e32 v43, 0")
    assert not bad("v_mov_b32_e32 v44, v8")
    # accumulating onto it is what the hardware waits for; taking it as a factor, or writing a part, is not
    assert not bad(MFMA)
    assert not bad(MFMA.replace("v[40:43]", "v[60:63]", 1))
    assert bad(MFMA.replace("v[8:15]", "v[36:43]")) and bad(MFMA.replace("v[40:43]", "v[42:45]"))
    accumulators = MFMA.replace("v[40:43]", "a[0:3]")
    assert build.mfma_result_hazards(listing(accumulators, "v_accvgpr_read_b32 v1, a3"))
    assert not build.mfma_result_hazards(listing(accumulators, "v_accvgpr_read_b32 v1, a4"))


def test_hazards_along_branches():
    """A taken branch leads from the product to the read, or from the write to the product."""
    loop = listing("v_mov_b32_e32 v1, v41", *["s_mov_b32 s0, s1"] * 14, MFMA, "s_cbranch_scc1 0 -> 0", "s_nop 15", "s_endpgm")
    assert build.mfma_result_hazards(loop)
    once = listing("v_mov_b32_e32 v1, v41", *["s_mov_b32 s0, s1"] * 14, MFMA, "s_nop 15", "s_endpgm")
    assert not build.mfma_result_hazards(once)
    over = listing(MFMA, "s_branch 0 -> 4", "v_mov_b32_e32 v1, v41", "s_endpgm", "s_endpgm")
    assert not build.mfma_result_hazards(over)
    source = listing(MFMA, "s_nop 15", "v_mov_b32_e32 v30, v1", "s_cbranch_scc1 0 -> 0", "s_endpgm")
    assert build.mfma_source_hazards(source)
    settled = listing(MFMA, "s_nop 15", "v_mov_b32_e32 v30, v1", "s_nop 1", "s_cbranch_scc1 0 -> 0", "s_endpgm")
    assert not build.mfma_source_hazards(settled)


def test_the_built_code():
    build.check_mfma_results(build.LIB_PATH)
    build.check_mfma_sources(build.LIB_PATH)


def test_results_of_the_asm_products_wait_by_rule():
    """Between the last product and the first conversion of a result in the kernels
    whose products are asm statements stands a wait of 16 states, on every path."""
    asm = build.device_assembly(build.LIB_PATH)
    for kernel in ("fp8_mid_kernel", "fp8_gemm_kernel"):
        body = re.search(r"[0-9a-f]+ <\w*%s\w*>:\n(.*?)(?=\n\n|\Z)" % kernel, asm, re.S)
        f = build._functions(body.group(0))[0]
        products = [i for i, ins in enumerate(f) if ins.mfma]
        assert products
        results = set().union(*(f[i].operands[0] for i in products))
        seen, todo = set(), [j for i in products for j in f[i].next]
        reached = 0
        while todo:                                       # everything behind a product without such a wait between
            j = todo.pop()
            if j in seen:
                continue
            seen.add(j)
            ins = f[j]
            if ins.text == "s_nop 15":
                reached += 1
                continue
            if not ins.mfma and ins.name.startswith(("v_cvt_pk_bf16", "v_accvgpr_read", "ds_write", "buffer_store")):
                assert not results & set().union(*ins.operands), (kernel, ins.text)
            todo += ins.next
        assert reached
