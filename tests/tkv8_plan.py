"""Sizes at which attention takes a certain path, for the tests that compare that path with a reference and the one that
asks the host half's plan whether they do (tests/tkv8_plan_driver.cpp)."""
import os
import subprocess
from collections import namedtuple

Case = namedtuple("Case", "bits dim group heads n_seq group_heads new longest window sinks")
Plan = namedtuple("Plan", "row_tile row_blocks n_split chunk even window")
PAGE = 128

# Windows whose steps are dealt out evenly: tiles of 16 and of 32 rows, one and several of them.
EVEN_WINDOWS = [
    Case(8, 128, 0, 8, 64, 1, 1, 6000, 2500, 40),    # a server's decoding step
    Case(8, 128, 0, 8, 64, 4, 5, 6000, 2500, 0),     # 20 rows
    Case(8, 64, 0, 8, 40, 5, 12, 6000, 3000, 70),    # 60 rows, two tiles
    Case(8, 96, 0, 8, 64, 2, 1, 5000, 2400, 7),
    Case(8, 256, 0, 8, 24, 2, 20, 5000, 2500, 33),   # 40 rows, three tiles of 16
    Case(4, 128, 64, 8, 64, 4, 1, 6000, 2500, 40),
    Case(4, 128, 128, 8, 64, 4, 5, 6000, 2500, 0),
    Case(4, 64, 32, 8, 64, 5, 6, 6000, 3000, 70),
    Case(4, 96, 32, 8, 64, 2, 1, 5000, 2400, 7),
    Case(4, 256, 128, 8, 24, 2, 20, 5000, 2500, 33),
]

# Many rows (a workgroup has 64 or 128 of them) whose positions go in several chunks, which are joined.  930 positions and
# 40 first ones: of 128 rows' tokens more than two chunks of 512, of the last few tokens not.
MANY_ROWS = [Case(bits, dim, group, 2, 3, 2, new, 3000, window, sinks)
             for bits, dim, group, new in ((8, 64, 0, 70), (8, 96, 0, 70), (8, 128, 0, 70), (8, 256, 0, 70), (8, 128, 0, 33),
                                           (4, 64, 32, 70), (4, 96, 32, 25), (4, 128, 64, 70), (4, 128, 128, 25),
                                           (4, 256, 64, 70), (4, 256, 128, 25))
             for window, sinks in ((0, 0), (1300, 40), (930, 40))]
# ... so many that a row's partial sums are joined by a workgroup
MANY_CHUNKS = [Case(bits, dim, group, 1, 1, 1, 90, 12000, window, sinks)
               for bits, dim, group in ((8, 128, 0), (8, 256, 0), (4, 128, 32))
               for window, sinks in ((0, 0), (9500, 100))]


def width(c):
    return -(-c.longest // PAGE) + 1


def plans(cases, directory):
    """the host half's plans, on 256 compute units"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = os.path.join(str(directory), "tkv8_plan_driver")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(root, "include"),
                    os.path.join(root, "tiled_tensor_bulk_amd", "csrc", "tkv_host.cpp"),
                    os.path.join(root, "tests", "tkv8_plan_driver.cpp"), "-o", exe], check=True, capture_output=True)
    lines = "".join(f"{c.bits} {c.dim} {c.heads} {PAGE} {c.n_seq} {c.heads * c.group_heads} {c.new} {width(c)} {c.longest} "
                    f"{c.window} {c.sinks}\n" for c in cases)
    out = subprocess.run([exe], input=lines, check=True, capture_output=True, text=True).stdout
    return [Plan(*map(int, line.split())) for line in out.splitlines()]
