"""Rows of no sequence are set to zero by one CTA for each head and block of columns,
piece by piece.  Their count can pass what 32 bits hold: the walk over them, run here on
the host, reaches every piece of the rows once and nothing else."""
import subprocess

from state_space_sequence_chunk_gb300 import build as ssd_build

SOURCE = r"""
#include <stdio.h>
#include <vector>
#include "linattn_internal.cuh"
int main() {
    const int cases[][3] = {{1, 1, 128}, {1000, 4, 128}, {777, 12, 256}, {777, 3, 128}, {(1 << 25) + 5, 16, 256},
                            {(1 << 29) + 5, 4, 128}, {1 << 30, 1, 128}, {1 << 30, 16, 256}};
    for (const auto& c : cases) {
        const int rows = c[0], pieces = c[1], threads = c[2];
        long long seen = 0, bad = 0;
        std::vector<unsigned char> hit(rows < 100000 ? (size_t)rows * pieces : 0);
        const int some = rows < 100000 ? 1 : 37;   // every thread of the small cases, some of the large
        long long want = 0;
        for (int t = 0; t < threads; t += some) {
            long long last = -1, n = 0;
            ssd::la_zero_rows(rows, pieces, t, threads, [&](int row, int piece) {
                if (row < 0 || row >= rows || piece < 0 || piece >= pieces) { ++bad; return; }
                const long long at = (long long)row * pieces + piece;
                bad += at <= last;
                last = at;
                ++n;
                if (!hit.empty()) bad += hit[at]++ != 0;
            });
            seen += n;
            // thread t of the first floor(threads / pieces) * pieces has every step-th row
            const int step = threads / pieces;
            if (t < step * pieces) want += (rows - t / pieces + step - 1) / step;
        }
        if (some == 1 && want != (long long)rows * pieces) ++bad;
        printf("%d %d\n", (int)(seen == want), (int)bad);
    }
    return 0;
}
"""


def test_every_piece_once(tmp_path):
    src, exe = str(tmp_path / "rows.cu"), str(tmp_path / "rows")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([ssd_build.nvcc(), *ssd_build.ARCH, *ssd_build.NVCC_FLAGS, "-cudart", "static", "-o", exe, src],
                   check=True, capture_output=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=120).stdout
    assert out.split("\n")[:-1] == ["1 0"] * 8
