"""A load from tensor memory writes its registers when it completes, and tcgen05.wait::ld has no operand that holds back
what uses them: a compiler may move such a use ahead of the wait. So the wait is written once, in a function that ties the
registers to it, and every load in the sources is followed by that function with the load's own registers (CPU check of the
source: whether a use moves is decided anew at each build)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_tree_absorb_gb300", "csrc")


def _sources():
    files = {os.path.basename(f): open(f).read() for ext in ("cu", "cuh") for f in glob.glob(os.path.join(CSRC, "*." + ext))}
    assert files
    return files


def test_the_wait_is_written_once():
    assert {f: t.count("tcgen05.wait::ld") for f, t in _sources().items() if "tcgen05.wait::ld" in re.sub(r"//.*", "", t)} == {
        "tc_ptx.cuh": 1}
    assert not [f for f, t in _sources().items() if "tmem_wait_ld" in t]


def test_every_load_is_tied_to_its_wait():
    seen = 0
    for name, text in _sources().items():
        if name == "tc_ptx.cuh":
            continue
        lines = text.splitlines()
        for i, line in enumerate(lines):
            m = re.search(r"\btmem_ld\w*\(.*,\s*(\w+)(\[\w+\])?\);", line)
            if not m:
                assert not re.search(r"\btmem_ld\w*\(", line), f"{name}:{i + 1}: a load that this check cannot read"
                continue
            seen += 1
            # up to the wait there is nothing but other loads and the wait's own loop
            for later in lines[i + 1:i + 6]:
                w = re.search(r"\bloaded\((.*)\);", later)
                if w:
                    assert m.group(1) in re.findall(r"\w+", w.group(1)), f"{name}:{i + 1}: {m.group(1)} is not tied to the wait"
                    break
                assert re.search(r"\btmem_ld\w*\(|#pragma unroll|for \(int k", later), f"{name}:{i + 1}: used before the wait"
            else:
                raise AssertionError(f"{name}:{i + 1}: no wait")
    assert seen >= 10
