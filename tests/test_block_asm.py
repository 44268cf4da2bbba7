"""CPU checks of the compiled gfx950 code (no GPU needed): the strips through which
waves store, and the E4M3 products."""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tile_partitioned_dense_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"


def compiled(source, define, out):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC, f"-D{define}", "-S",
           "--cuda-device-only", os.path.join(CSRC, source), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True)
    return out.read_text()


def check_strips(asm, barriers):
    kernels = re.findall(r"^_Z\S+:.*?s_endpgm", asm, flags=re.S | re.M)
    assert kernels
    for k in kernels:
        events = re.findall(r"ds_write_b128|ds_write_b64|; wave barrier|s_barrier|global_store", k)
        assert events.count("; wave barrier") >= barriers and events.count("global_store")
        stored = False
        for e in events:
            write = e.startswith("ds_write")
            assert not (write and stored), "a strip is written where the last one may still be read"
            stored = e == "global_store" or (stored and write)


@pytest.mark.parametrize("source,define", [
    ("kernels_block.hip", "TG_BLOCK_CONFIG=5"),    # E4M3, 32 x 128: two strips a wave
    ("kernels_train.hip", "TG_TRAIN_KERNEL=9"),    # stores of the gated block and of the loss
    ("kernels_train.hip", "TG_TRAIN_KERNEL=52"),
    ("kernels_train.hip", "TG_TRAIN_KERNEL=107"),
    ("kernels_mx.hip", "TG_MX_CONFIG=6"),
])
def test_strips_are_kept_apart(source, define, tmp_path):
    """A wave stores its results by strips that its lanes pass each other through
    LDS. Lanes with nothing to store may not run ahead and write the next strip
    before the others have read theirs: the compiler keeps them together
    only where it is told to."""
    check_strips(compiled(source, define, tmp_path / "k.s"), 4)  # before and behind each strip's reads


@pytest.fixture(scope="module", params=[0, 4], ids=["tile", "stream"])
def asm(request, tmp_path_factory):
    """Assembly of the 256 x 256 tile and of the 16 x 128 one."""
    return compiled("kernels_block.hip", f"TG_BLOCK_CONFIG={request.param}", tmp_path_factory.mktemp("asm") / "k.s")


def kernels(asm):
    """{mangled name: {resource: value}} of the kernels' metadata."""
    found = {}
    for part in asm.split(".amdgpu_metadata")[1].split("  - .agpr_count:")[1:]:
        name = re.search(r"\.name:\s+(\S+)", part).group(1)
        found[name] = {k: int(v) for k, v in re.findall(r"\.(\w+):\s+(\d+)\n", part)}
    return found


def test_experts_kernels_use_no_scratch(asm):
    """Their call has neither bias nor activation, so nothing of an epilogue may
    take registers that the sums need."""
    experts = {n: r for n, r in kernels(asm).items()
               if re.search(r"block_tile_kernel(ILi\d+E|Li\d+E)+Lb1E|block_gemm_kernel(ILi\d+E|Li\d+E)+Lb1E", n)}
    assert experts
    for name, r in experts.items():
        assert r["private_segment_fixed_size"] == 0 and r["vgpr_spill_count"] == 0, (name, r)


# M0 may be set from any scalar register; an asm block without instructions pins a value
ALLOWED = re.compile(r"^(s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)|"
                     r"buffer_load_dword(x4)? v\d+, s\[\d+:\d+\], (0|s\d+|vcc_lo|vcc_hi) offen( nt)? lds)$")


def test_inline_asm_only_sets_m0_and_loads(asm):
    """The compiler does not see what such a block writes: it may set M0
    (declared) and issue a load into LDS, with the cache hint nt, and nothing else."""
    lines = [line.split(";")[0].strip() for b in re.findall(r";;#ASMSTART\n(.*?);;#ASMEND", asm, flags=re.S)
             for line in b.splitlines()]
    lines = [line for line in lines if line]
    assert any("lds" in line for line in lines)
    for line in lines:
        assert ALLOWED.match(line), f"unexpected instruction in inline asm: {line}"
    outside = re.sub(r";;#ASMSTART\n.*?;;#ASMEND", "", asm, flags=re.S)
    assert not re.search(r"^\s*s_\w+\s+m0\b", outside, flags=re.M)
