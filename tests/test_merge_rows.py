"""Rows that the tree pass and merge over the 8-bit cache touches, for every row
count and launch grid, compiled with g++ on the CPU
(tests/native/merge_rows_check.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_row_read_is_one_of_the_units(tmp_path):
    exe = os.path.join(tmp_path, "merge_rows_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I",
                    os.path.join(ROOT, "speculative_decoding_tree_split_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "native", "merge_rows_check.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stdout + r.stderr
