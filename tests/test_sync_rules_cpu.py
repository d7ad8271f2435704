"""Rules of synchronisation that the kernels' sources keep, read from the sources:
what breaks them shows on a GPU only as a race or a hang."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir, "int8_dequant_gemm_b200", "csrc")


def sources():
    """Every kernel source without its comments, by file name."""
    out = {}
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
            out[name] = re.sub(r"//[^\n]*", "", text)
    return out


def functions(text):
    """(name, body) of each function definition whose body is in braces."""
    for m in re.finditer(r"\b(\w+)\s*\(([^(){};]|\([^()]*\))*\)\s*(const\s*)?\{", text):
        if m.group(1) in ("if", "for", "while", "switch"):
            continue
        depth, at = 1, m.end()
        while depth and at < len(text):
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[m.end():at - 1]


def test_cluster_barriers_gather_their_warp():
    """barrier.cluster in its .aligned form is undefined for a warp whose lanes
    are apart, as they are after waits that lanes leave one by one: the three
    wrappers, the only places that issue it, gather the warp first."""
    found = {}
    for name, text in sources().items():
        for fn, body in functions(text):
            if "barrier.cluster" in body:
                found.setdefault(name, set()).add(fn)
                assert body.find("__syncwarp()") >= 0, (name, fn)
                assert body.find("__syncwarp()") < body.find("barrier.cluster"), (name, fn)
    assert found == {"ptx.cuh": {"cluster_sync", "cluster_arrive", "cluster_wait"}}


def test_a_warp_agrees_that_its_loads_failed():
    """What a warp's polling loops found becomes `ok` by a vote, not lane by lane."""
    text = sources()["a8.cu"]
    assert re.findall(r"\bok = (?!true|__all_sync)[^;]*;", text) == []
