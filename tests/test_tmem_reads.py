"""What the sources promise the compiler about reads of tensor memory (CPU): a load's registers hold nothing before the wait, so the
wait has to be where they come from, or arithmetic on them may be moved in front of it."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_moe_quantize_gb300", "csrc")


def test_waits_for_tensor_memory_produce_the_loaded_registers():
    waits = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"asm\s+volatile\s*\((?:[^;]|;(?=[^\"\n]*\"))*tcgen05\.wait::ld[^;]*;(?:[^;]*);", text):
            waits += 1
            assert '"+r"' in m.group(0), f"{os.path.basename(path)}: {m.group(0)[:100]}"
    assert waits > 0
