"""Warp barriers and collectives of the kernels name their lanes: a barrier over the lanes that
happen to be converged (the active mask) separates nothing from the others of its warp."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def kernel_sources():
    out = {}
    for path in sorted(glob.glob(os.path.join(ROOT, "block_sparse_long_09_b200", "csrc", "*.cu*"))):
        text = open(path).read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        out[os.path.basename(path)] = re.sub(r"//[^\n]*", "", text)
    return out


def test_no_barrier_over_the_active_mask():
    src = kernel_sources()
    assert "attn_chunk_tc.cu" in src
    assert [f for f, text in src.items() if re.search(r"__activemask|activemask\.b32", text)] == []


def test_walk_state_is_read_and_written_between_barriers():
    """The work list of the chunk attention is walked through shared memory: a whole warp's step has a
    barrier before its reads, one between reads and writes, and one behind them; the step of an
    elected lane has none (its warp waits elsewhere)."""
    text = kernel_sources()["attn_chunk_tc.cu"]
    body = text[text.index("bool next(const ChunkArgs &a)"):]
    body = body[:body.index("return true;")]
    marks = [m.group(0) for m in re.finditer(r"__syncwarp\([^)]*\)|= state\[0\]|state\[0\] =", body)]
    assert marks == ["__syncwarp()", "= state[0]", "__syncwarp()", "state[0] =", "__syncwarp()"]
    elected = text[text.index("if (elect_one())"):text.index("} else if (warp < 4)")]
    assert "next<true>" not in elected and elected.count("next<false>") == 2
    assert text.count("next<true>") + 2 == text.count("it.next<")
