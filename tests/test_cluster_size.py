"""The size of the page bookkeeping's clusters where the device has no room for a large one (csrc/gdn_cluster_size.h; CPU only)."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_decode_gb300", "csrc")

DRIVER = r"""
#include <cstdio>
#include <initializer_list>
#include "gdn_cluster_size.h"
int main() {
    for (int want : {1, 2, 8, 16})
        for (int room : {-1, 0, 1, 9}) {
            int asked = 0;
            const int n = gdn::cluster_that_fits(want, [&](int m) { asked = m; return room; });
            std::printf("%d %d %d %d\n", want, room, n, asked);
        }
}
"""


def test_the_portable_size_where_more_do_not_fit(tmp_path):
    src, exe = tmp_path / "size.cpp", tmp_path / "size"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    rows = [tuple(map(int, r.split())) for r in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()]
    assert len(rows) == 16
    for want, room, n, asked in rows:
        assert (n, asked) == ((16 if room > 0 else 8, 16) if want == 16 else (want, 0))   # (what is portable is not asked for)


def test_the_bookkeeping_asks_before_it_launches_a_large_cluster():
    src = re.sub(r"//.*", "", open(os.path.join(CSRC, "gdn_pages.cu")).read())
    allowed = [m.end() for m in re.finditer("cudaFuncAttributeNonPortableClusterSizeAllowed", src)]
    assert len(allowed) == 1
    rest = src[allowed[0]:]
    assert 0 <= rest.find("cluster_that_fits(") < rest.find("launch_dependent_cluster(")
