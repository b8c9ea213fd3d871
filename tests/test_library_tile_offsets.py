"""Where the lanes of a 4-bit product's large tiles read the rows' scales: inside the operand, whatever is left of the last tile."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The tiles' rows (tokens or outputs) are sent for in two parts by eight waves, 16 bytes of a row a lane.  An operand of `rows` rows of `pitch`
# bytes: every load ends inside of it, and every row that exists is read into its own place, once.
CHECK = r"""
#include "ecf8x_offsets.h"
#include <cstdio>
#include <vector>

int main()
{
    long loads = 0;
    for (int tile : {128, 256})
        for (int parts : {1, 2, 4})
            for (uint32_t pitch : {4u, 16u, 20u, 160u, 260u, 32768u})
                for (int rows = 1; rows <= tile; ++rows) {
                    const int each = tile / (8 * parts);
                    std::vector<int> seen(tile);
                    for (int part = 0; part < parts; ++part)
                        for (int wave = 0; wave < 8; ++wave)
                            for (int lane = 0; lane < each; ++lane) {
                                const int place = ecf8x::scale_row(part, wave, lane, each);
                                const uint64_t at = ecf8x::scale_offset(part, wave, lane, each, rows, pitch);
                                const uint32_t last = pitch < 16 ? 0 : pitch - 16, bytes = pitch < 16 ? pitch : 16;   // the place inside of a row
                                if (place < 0 || place >= tile || at % pitch || at + last + bytes > (uint64_t)rows * pitch) return 1;
                                if (place < rows && at != (uint64_t)place * pitch) return 2;
                                ++seen[place];
                                ++loads;
                            }
                    for (int s : seen)
                        if (s != 1) return 3;
                }
    std::printf("%ld\n", loads);
    return 0;
}
"""


def test_every_lane_reads_inside_the_operand(tmp_path):
    src, exe = tmp_path / "offsets.cpp", tmp_path / "offsets"
    src.write_text(CHECK)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "lossless_entropy_coded_ecf8_amd", "csrc"), "-o", str(exe), str(src)],
                   check=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and int(p.stdout) > 0, p.returncode


def test_the_product_uses_these_offsets():
    """No load of scales counts on the range of its buffer, and no row is in the offset that is the same for all lanes."""
    csrc = os.path.join(ROOT, "lossless_entropy_coded_ecf8_amd", "csrc")
    text = open(os.path.join(csrc, "ecf8x_linear.hip")).read()
    assert "scale_offset(" in text and "part * 8 *" not in text
    assert "buffer_of(const void* p)" in open(os.path.join(csrc, "ecf8x_stream.h")).read()
