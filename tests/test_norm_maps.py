"""A rule of the norm's sources, by a scan (no GPU): tensor maps are prefetched where they are made, under the conditions of
their first copies (a row of whole lines, a residual)."""
from test_warp_waits import code


def test_only_maps_that_are_made_are_prefetched():
    text = code("norm.cu")
    block = text[text.index("if (lines) {", text.index("norm_staged_kernel(")):]
    block = block[:block.index("}")]
    assert text.count("tma_prefetch_desc(") == block.count("tma_prefetch_desc(") == 3
    assert "if (a.r) tma_prefetch_desc(&tmr);" in block
