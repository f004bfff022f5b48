"""What the kernels' sources must keep to and no run shows reliably."""
import glob
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_post_quantization_amd", "csrc")


def test_every_bare_barrier_stands_between_memory_clobbers():
    """The barrier builtin alone lets the compiler move reads of LDS across it
    (it counts as touching no memory); an asm statement that clobbers memory on
    either side does not."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        lines = [l.split("//")[0].strip() for l in open(path, encoding="utf-8")]
        lines = [l for l in lines if l]
        for i, l in enumerate(lines):
            if "__builtin_amdgcn_s_barrier" in l:
                seen += 1
                assert l == "__builtin_amdgcn_s_barrier();", (path, l)
                for side in (lines[i - 1], lines[i + 1]):
                    assert side.startswith("asm volatile(") and '"memory"' in side, (path, lines[i - 1:i + 2])
    assert seen
