"""The cuts of the vocabulary that test_vocab_pieces_gpu.py relies on: several pieces, dx in
slices over them, a last piece of its own number of slices (host code only)."""
import os
import subprocess

import pytest

from test_sanitizers import HERE, HIP_INCLUDE, _need

# rows, width, vocab -> (with dx and dweight, with dx alone): pieces, columns, slices of dx, and of the last piece
CUTS = {
    (40000, 64, 8300): ((2, 8192, 1, 1), (2, 8192, 1, 1)),
    (13000, 264, 12100): ((2, 10240, 1, 1), (2, 10240, 2, 2)),
    (5000, 72, 26876): ((2, 18944, 4, 4), (2, 25088, 8, 7)),
    (3000, 136, 50280): ((2, 26624, 8, 8), (2, 41984, 8, 8)),
    (600, 72, 300007): ((2, 195840, 8, 8), (2, 195840, 8, 8)),
    (16, 64, 4200001): ((2, 4194304, 8, 8), (2, 4194304, 8, 8)),
}


def test_cuts(tmp_path):
    _need("g++")
    if not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("HIP headers not found")
    exe = str(tmp_path / "pieces_driver")
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", f"-I{HIP_INCLUDE}", os.path.join(HERE, "sanitize", "pieces_driver.cpp"),
                    "-o", exe], check=True)
    asked = [(*size, 1, dw) for size in CUTS for dw in (1, 0)]
    text = subprocess.run([exe, *(str(v) for a in asked for v in a)], check=True, capture_output=True, text=True).stdout
    got = [tuple(map(int, line.split())) for line in text.splitlines()]
    want = [c for both in CUTS.values() for c in both]
    for a, g, w in zip(asked, got, want, strict=True):
        assert (g[0], g[1], g[2], g[4]) == w, (a, g)
