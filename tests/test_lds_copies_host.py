"""The copies from memory into LDS are inline assembly, in which the compiler resolves no hazards: the generated
code of a kernel with spilled scalar registers is read for the wait states of every copy."""
import re
import subprocess

from gated_delta_rule_47_amd import _build


def wait_states(lines):
    """Wait states that these instructions take at least: one each, s_nop N takes N + 1."""
    return sum(int(l.split()[1]) + 1 if l.startswith("s_nop") else 1 for l in lines)


def test_every_copy_waits_for_its_scalar_registers(tmp_path):
    out = tmp_path / "k.s"
    subprocess.run([_build.HIPCC] + _build.FLAGS + ["-S", "--cuda-device-only",
                   _build.CSRC + "/kda_decay_bwd_bf16_kd32.hip", "-o", str(out)], check=True, capture_output=True)
    text = out.read_text()
    assert "v_readlane_b32" in text                               # (spilled ones read back by vector instructions)
    copies = 0
    for block in re.findall(r";;#ASMSTART\n(.*?);;#ASMEND", text, re.S):
        lines = [l.strip() for l in block.strip().splitlines()]
        if not any(l.endswith(" lds") for l in lines):
            continue
        copies += 1
        assert lines[0].startswith("s_mov_b32 m0, ") and lines[-1].startswith("buffer_load_dwordx4 v")
        assert wait_states(lines[1:-1]) >= 1                      # m0 written, then read
        # a scalar register written by the vector instruction in front of the block, then read by the copy
        assert wait_states(lines[:-1]) >= 5, block
    assert copies > 500
    # nothing else of these kernels relies on m0
    assert not [l for l in text.splitlines() if re.search(r"\bm0\b", l) and not re.search(r"s_mov_b32 m0, |^\s*;", l)]
