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


# GEMM kernels that read their weights before they wait for the launch before
# them: launched behind a pre-pass (or behind one of themselves), never first
BEHIND_A_PREPASS = {"xs_qgemm_kernel", "ws_qgemm_kernel", "pl_qgemm_kernel"}


def test_launches_wait_before_they_release_the_next():
    """A kernel may read what an earlier launch wrote only behind a wait for it:
    leaving launch_dependents out delays the next launch but makes nothing
    visible to it.  So every kernel waits before it lets the next start, but for
    those behind a pre-pass, and a weight written just before a call (by
    quantize_a8 or a copy) is complete when the call's GEMM reads it."""
    seen = set()
    for name, text in sources().items():
        for fn, body in functions(text):
            # cvt_x16_kernel's early release, for a launch that waits itself (below)
            body = body.replace("if (next_waits) pdl_launch_dependents();", "")
            release = body.find("pdl_launch_dependents()")
            if release < 0 or name == "ptx.cuh":
                continue
            seen.add(fn)
            wait = body.find("pdl_wait_prior_grid()")
            assert wait >= 0, (name, fn)
            if fn not in BEHIND_A_PREPASS:
                assert wait < release, (name, fn)
                assert "tma_load" not in body[:wait], (name, fn)
    assert seen > BEHIND_A_PREPASS | {"cvt_x16_kernel", "cvt_x16_group_kernel", "pl_prep_kernel",
                                      "xp_qgemm_kernel"}


def test_gemms_that_read_ahead_follow_a_prepass():
    """Host side: each function that launches one of them launches its pre-pass
    first (`run_list` launches the single ones after its chunks)."""
    text = sources()
    for name, fn, first, then in (("api.cu", "run_gemm", "launch_cvt_x16(", ("launch_xs(", "launch_ws(")),
                                  ("api.cu", "run_list", "launch_cvt_x16_group(",
                                   ("launch_xs_group(", "launch_xs(", "launch_ws(")),
                                  ("noalloc.cu", "rt_qgemm_noalloc", "launch_cvt_x16(", ("launch_xs(", "launch_ws(")),
                                  ("pl.cu", "launch_pl_batch", "launch_pl_prep(", ("launch_pl(",))):
        body = next(b for f, b in functions(text[name]) if f == fn)
        assert first in body, (name, fn)
        for call in then:
            assert body.find(first) < body.find(call), (name, fn, call)
    calls = {(name, fn) for name, t in text.items() for fn, b in functions(t)
             if re.search(r"rtq::launch_(xs|ws|xs_group)\(", b)}
    assert calls == {("api.cu", "run_gemm"), ("api.cu", "run_list"), ("noalloc.cu", "rt_qgemm_noalloc")}


def test_a_prepass_that_releases_at_once_has_a_reader_that_waits():
    text = sources()
    xs = dict(functions(text["xs.cu"]))["xs_qgemm_kernel"]
    assert 0 < xs.find("if (P.w_wait) pdl_wait_prior_grid();") < xs.find("tma_load")
    for name, fn in (("api.cu", "run_gemm"), ("noalloc.cu", "rt_qgemm_noalloc")):
        body = dict(functions(text[name]))[fn]
        assert "const bool w_wait = kern == RT_KERNEL_TC_X_RESIDENT &&" in body
        assert re.search(r"launch_cvt_x16\([^;]*\bw_wait, ctl, s\)", body)
        assert re.search(r"launch_xs\([^;]*\bctl, s, w_wait\)", body)
