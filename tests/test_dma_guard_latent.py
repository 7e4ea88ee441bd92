"""The LDS DMA issue order of the latent attention kernels, by the checks of
test_dma_guard_asm on the gfx950 code of every form of them (no GPU needed)."""

import subprocess

import pytest

from fp8_block_scaled_nt_amd import build as B
from tests.test_dma_guard_asm import m0_writes_outside_guards, unguarded_successors

FORMS = [f"latent_attn_kernel<{L}, {f8}, {nt}>(LatentAttnParams)" for L in (256, 512) for f8 in ("false", "true") for nt in (1, 2, 4)]
FORMS += [f"latent_expanded_kernel<{d}, {mt}>(LatentExpandedParams)" for d in (64, 128) for mt in (1, 2)]
FORMS += [f"latent_expanded_kernel<{d}, {mt}, true>(LatentExpandedParams)" for d in (64, 128) for mt in (1, 2)]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    at = tmp_path_factory.mktemp("asm")
    (at / "forms.hip").write_text('#include "latent_kernel.h"\nnamespace dg {\n' +
                                  "".join(f"template __global__ void {f};\n" for f in FORMS) + "}\n")
    flags = [f for f in B.HIPCC_FLAGS if f not in ("-shared", "-fPIC", "-Wall")]
    r = subprocess.run([hipcc] + flags + ["-Wno-inline-asm", "--cuda-device-only", "-S", "-I", B.CSRC, str(at / "forms.hip"),
                                          "-o", str(at / "forms.s")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = (at / "forms.s").read_text()
    # the checks look at kernels of one name
    for name in ("18latent_attn_kernel", "22latent_expanded_kernel"):
        assert "_ZN2dg" + name in text
        text = text.replace("_ZN2dg" + name, "_ZN2dg18gemm_fp8_nt_kernel")
    return text.split("\n")


def test_every_lds_dma_is_followed_by_a_guard(asm):
    found, dmas = unguarded_successors(asm)
    assert dmas > 300
    assert not found, found[:10]


def test_every_m0_write_is_inside_a_guard(asm):
    found, total = m0_writes_outside_guards(asm)
    assert total > 300
    assert not found, found[:10]


def test_main_loops_do_not_spill(asm):
    # a reload would wait for every DMA in flight
    block, spills, products = [], [], 0
    for line in asm + [".LBB"]:
        if line.startswith((".LBB", "_Z")):
            if any("v_mfma" in x for x in block):
                products += 1
                spills += [x for x in block if "scratch_" in x]
            block = []
        block.append(line)
    assert products > len(FORMS) and not spills, spills
