"""A rule of the CUDA sources, checked by a scan (no GPU): where all lanes of a warp wait on an mbarrier and
then go on or give up, they do it together.

Each lane polls the barrier, the clock and the abort flag for itself.  When a wait runs out, or another
role of the CTA gives up, some lanes can see the phase complete and others not; a warp that
parted so would reach elect.sync, tcgen05.ld, a cluster barrier or a shuffle with some of its lanes only, for
which nothing is defined.  So a whole warp's answer is voted on: by warp_wait, or once at the end of a tile, until
which no lane leaves."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "w8a8_quantized_projections_gb300", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def voted(text, pos):
    """Whether the expression at pos is an argument of __all_sync( or __any_sync(."""
    depth = 0
    for i in range(pos - 1, -1, -1):
        if text[i] in ";{}" and depth == 0:
            return False
        depth += (text[i] == ")") - (text[i] == "(")
        if depth < 0:
            if re.search(r"__a(ll|ny)_sync$", text[max(0, i - 12):i]):
                return True
            depth = 0
    return False


def stays(text, pos):
    """Whether the wait at pos only goes into the kept flag `ok`."""
    before = re.split(r"[;{}]", text[:pos])[-1]
    if re.match(r"\s*bool ok = ", before):       # of one turn of the loop: voted on before the turn can end
        way = text[pos:text.index("return", pos)]
        return re.search(r"if \(!__all_sync\(0xFFFFFFFFu, ok\)\) $", way) is not None and not re.search(r"\b(break|continue)\b", way)
    return re.match(r"\s*ok = ok && ", before) is not None or \
        re.fullmatch(r"\s*if \(!", before) is not None and re.match(r"[^;{]*\) ok = false;", text[pos:]) is not None


def lone_exits(text):
    """What leaves a loop on the flag `ok` of a lane, which has not been voted on."""
    return re.findall(r"if \([^;{]*\bok\b[^;{]*\) (?:break|return|continue);", re.sub(r"if \(!\(ok = __all_sync\(kWarp, ok\)\)\)", "", text)) + \
        re.findall(r"(?<=;)[^;(){}]*&& ok;", text)


def unvoted(text, calls=r"mbar_wait|mbar_wait_cl|wait_pair|stay_wait"):
    return [text[m.start():m.end() + 40].split(",")[0] for m in re.finditer(r"\b(%s)\(" % calls, text)
            if not re.match(r"\s*(__device__|static)", text[text.rfind("\n", 0, m.start()) + 1:m.start()])
            and not voted(text, m.start()) and not stays(text, m.start())]


def test_the_scan_finds_what_it_looks_for():
    assert unvoted("if (!mbar_wait(&b, 0, w, 1)) break;") == ["mbar_wait(&b"]
    assert unvoted("x(); if (!__all_sync(kAll, ready || (mbar_wait(&b, 0, w, 1) && mbar_wait(&d, 1, w, 2)))) break;") == []
    assert unvoted("__all_sync(kAll, y); mbar_wait(&b, 0, w, 1);") == ["mbar_wait(&b"]
    assert unvoted("if (!warp_wait(&b, 0, w, 1)) break;") == []
    assert unvoted("ok = ok && (ready || (mbar_wait(&b, 0, w, 1) && mbar_wait(&d, 0, w, 1)));") == []
    assert unvoted("if (!stay_wait(&b, 0, w, 1)) ok = false;") == []
    assert unvoted("bool ok = mbar_wait(&b, 0, w, 1); x(); if (!__all_sync(0xFFFFFFFFu, ok)) return;") == []
    assert unvoted("bool ok = mbar_wait(&b, 0, w, 1); if (!ok) return; if (!__all_sync(0xFFFFFFFFu, ok)) return;") == ["mbar_wait(&b"]
    assert unvoted("if (!stay_wait(&b, 0, w, 1)) { ok = false; break; }") == ["stay_wait(&b"]
    assert lone_exits("if (!ok) break; if (!(ok = __all_sync(kWarp, ok))) break; for (;i < n && ok;) x();") == ["if (!ok) break;", "i < n && ok;"]


def test_warps_of_the_cache_attention_agree():
    assert unvoted(code("kv_attention.cu")) == []
    assert len(re.findall(r"\bwarp_wait\(", code("kv_attention.cu"))) >= 8


def test_warps_of_the_block_linears_agree():
    """Their lanes stay in the loop and keep their answers; the tile's end votes."""
    text = code("fp8_block.cu")
    helper = text[text.index("__device__ __forceinline__ bool stay_wait("):text.index("__device__ __forceinline__ bool elect_one(")]
    text = text.replace(helper, "")
    assert unvoted(text) == []
    assert lone_exits(text) == []
    assert text.count("ok = __all_sync(kWarp, ok)") == 2 and len(re.findall(r"elect_one\(\) && ok", text)) == 4


def test_warps_of_the_gemms_agree():
    """Converters and epilogue; copies and MMAs are issued by functions that one lane runs."""
    text = code("gemm.cu")
    converter = text[text.index("static __device__ void converter("):text.index("static __device__ void forwarder(")]
    epilogue = text[text.index("static __device__ void epilogue_tiles("):text.index("__global__")]
    assert unvoted(converter) == [] and unvoted(epilogue) == []
    assert len(re.findall(r"__all_sync|\bwarp_wait\(|\bwarp_pair\(", converter + epilogue)) >= 11
    assert re.search(r"bool warp_pair\([^{]*\{\s*return __all_sync\(0xFFFFFFFFu, wait_pair\(", text)
    for role in ("G::producer(", "G::mma_issuer(", "G::forwarder("):
        assert re.search(r"if \(lane == 0[^{]*\{[^{}]*$", text[:text.index(role)]), role


@pytest.mark.parametrize("name", ["norm.cu", "quant_act.cu"])
def test_warps_that_keep_rows_leave_together(name):
    """They go on after a wait that ran out, as far as the row's barrier, and leave on the flag of the CTA, which another
    warp may be setting while they read it: by vote, as reductions over the warp follow."""
    text = code(name)
    assert re.findall(r"if \([^;{]*abort_flag[^;{]*\) break;", text) == re.findall(r"if \(__any_sync\([^,]*, abort_flag\)\) break;", text) != []
    assert not re.search(r"(if|while) \([^;{)]*mbar_wait\(", text)


def test_the_shared_helper_votes():
    helper = code("clef_ptx.cuh").split("bool warp_wait(")[1].split("}")[0]
    assert "__all_sync(0xFFFFFFFFu, mbar_wait(" in helper
