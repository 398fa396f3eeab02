"""Kernels launched with programmatic stream serialization start before the preceding kernel of the stream has
finished, so what that kernel may have written must not be read by a load that the compiler may move above the wait
(a read-only load).  Checked on the sources: in files whose kernels wait so, read-only loads name weights only."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_mamba_b200", "csrc")

# int8 codes, sign words, LoRA factors and scales: written before the call is enqueued (include/dfssm.h)
WEIGHTS = re.compile(r"""^(?:reinterpret_cast<const\s[\w\s]+\*>\()?\(?\s*
                         (?: a\.W\b | row\b | wb\b | a\.norm_w\b | L\.(?:lora_a|lora_b)(?:_scale)?\b | L\.w_scale\b )""",
                     re.X)


def read_only_loads(text):
    for m in re.finditer(r"__ldg\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1], text.count("\n", 0, m.start()) + 1


def test_read_only_loads_are_of_weights():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        if "pdl_wait()" not in text or os.path.basename(path) == "common.cuh":
            continue
        seen += 1
        for what, line in read_only_loads(text):
            assert WEIGHTS.match(what), f"{os.path.basename(path)}:{line}: __ldg({what})"
        assert "__restrict__" not in text, path
    assert seen >= 6
