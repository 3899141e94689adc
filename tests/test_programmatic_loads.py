"""Kernels that may be resident while an earlier one still writes block tables, lengths
or offsets (launched with programmatic serialisation, they wait at griddep_wait) read
those by plain loads.  A read-only load assumes data that is constant for as long as the
kernel runs, and nothing orders it behind that wait."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_263_gb300", "csrc")
# queries: no kernel that lets the next one start early writes them
CONSTANT = {("latent_decode.cu", "reinterpret_cast<const uint4 *>(src")}


def test_no_read_only_loads_behind_the_programmatic_wait():
    found, waiting = [], 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        name, text = os.path.basename(path), open(path).read()
        code = re.sub(r"//[^\n]*", "", text)
        # latent_work.cuh, shared_prefix.cuh: what those kernels include
        if "griddep_wait()" not in code and not name.endswith(".cuh"):
            continue
        waiting += 1
        for m in re.finditer(r"__ldg\(|\.global\.nc|LDG_NC", code):
            rest = code[m.end():m.end() + 120]
            if not any(name == n and rest.startswith(a) for n, a in CONSTANT):
                found.append((name, code.count("\n", 0, m.start()) + 1, rest.split("\n")[0][:40]))
        # const and __restrict__ together let the compiler choose such loads by itself
        found += [(name, "restrict") for _ in re.finditer(r"const [^;,()]*__restrict__", code)]
    assert waiting >= 8
    assert not found
