"""The register split of the prompt attention's warp roles, read from its source: setmaxnreg has to be executed
by every warp of a warpgroup alike (four warps from a multiple of four), and the shares have to fit into what
the block was launched with, or an increase waits for good."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_one_instruction_per_warpgroup_and_no_more_than_the_launch_has():
    src = open(os.path.join(ROOT, "fp4_activation_sparse_b200", "csrc", "sharq_attn_tiles.cu")).read()
    threads = int(re.search(r"constexpr int kThreads = (\d+);", src).group(1))
    assert threads % 128 == 0
    src = re.sub(r"//[^\n]*", "", src)
    # the branch that each instruction opens: `if (warp < n) {`, `} else if (warp < n) {` or `} else {`
    found = re.findall(r"(?:if \(warp < (\d+)\)|else) \{\s*asm volatile\(\"setmaxnreg\.(?:inc|dec)\.sync\.aligned\.u32 (\d+);\"\);", src)
    assert len(found) == src.count("setmaxnreg.") == 3
    ends = [int(end) if end else threads // 32 for end, _ in found]
    assert ends == sorted(ends) and ends[-1] == threads // 32 and all(end % 4 == 0 for end in ends)
    shares = [int(n) for _, n in found]
    assert all(n % 8 == 0 and 24 <= n <= 256 for n in shares)
    launched = 65536 // threads // 8 * 8  # __launch_bounds__(kThreads, 1)
    assert sum(n * (end - begin) for n, begin, end in zip(shares, [0, *ends], ends)) <= launched * threads // 32
