"""What the compiler makes of the attention's inline assembly, which needs no GPU."""
import os
import re
import subprocess

from sparse_embedding_lookup_dlrm_amd import build


def test_inline_assembly_leaves_m0_as_it_was(tmp_path):
    """No block claims a register that the compiler keeps for itself, and each block that writes m0 saves it first
    and puts it back last."""
    out = tmp_path / "paged_attn.s"
    cmd = [build.hipcc(), "-x", "hip", f"--offload-arch={build.ARCH}", *build.COMMON, *build.DEVICE_FLAGS,
           "--cuda-device-only", "-S", os.path.join(build.CSRC, "paged_attn.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "-Winline-asm" not in r.stderr, r.stderr[:2000]
    blocks = [b for b in re.findall(r"#ASMSTART\n(.*?);;#ASMEND", out.read_text(), re.S) if "m0" in b]
    assert blocks
    for b in blocks:
        lines = [x.strip() for x in b.strip().splitlines()]
        saved = re.fullmatch(r"s_mov_b32 (s\d+), m0", lines[0])
        assert saved and lines[-1] == f"s_mov_b32 m0, {saved.group(1)}", b
