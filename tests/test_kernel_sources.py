"""Rules that the kernels' sources keep and that no run can show: a compiler that happens to do
the safe thing hides the fault."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "manifold_constrained_hyper_gb300", "csrc")


def _functions_that(what):
    """(file, name, the function's text) of the device functions whose body has `what` in it."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = open(path).read()
        for m in re.finditer(r"__device__ __forceinline__ [\w:<>&\s\*]*?(\w+)\([^;{]*\) \{\n(.*?)\n\}\n", text, re.S):
            if what in m.group(2):
                yield os.path.basename(path), m.group(1), m.group(2)


def test_a_tensor_memory_load_s_registers_go_through_its_wait():
    """tcgen05.ld leaves its destination registers undefined until tcgen05.wait::ld. A function
    that loads and does not wait may do nothing else: what it loaded goes out as the 32-bit
    registers of the load, not yet packed into or converted to anything."""
    seen = 0
    for path, name, body in _functions_that("tcgen05.ld."):
        seen += 1
        if "tcgen05.wait::ld" in body:
            continue
        load = body[body.index("asm volatile("):]
        after = load[load.index(");") + 2:].strip()
        assert not after, (path, name, after)
        assert '"=l"' not in load and '"=f"' not in load, (path, name)
    assert seen >= 4


def test_a_run_s_wait_takes_the_registers_of_its_load():
    """The block kernels' runs: the wait has the load's eight registers as operands, so that no
    use of them can stand before it."""
    waits = [b for _, n, b in _functions_that("tcgen05.wait::ld") if n == "tmem_run_wait"]
    assert len(waits) == 1
    assert len(re.findall(r'"\+r"\(l\.v\[\d\]\)', waits[0])) == 8
    assert waits[0].index("tcgen05.wait::ld") < waits[0].index("<< 32")
