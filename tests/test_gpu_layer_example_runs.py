"""examples/retention_layer.py runs as a program: its lines, in order, with the
norms of the heads and the clipping, and with the times of the 7B-shaped layer."""
import re

import pytest

from tests.gpu_util import torch_dev
from tests.test_gpu_layer_example import example

pytestmark = pytest.mark.gpu


def test_the_example_runs_as_a_program(capsys):
    torch_dev()
    example().main()
    lines = capsys.readouterr().out.strip().split("\n")
    assert len(lines) == 6, lines
    assert "relative difference" in lines[0] and lines[1].count("float32") >= 4
    norm, clipped = map(float, re.search(r"norm ([\d.]+), clipped to ([\d.]+)", lines[2]).groups())
    # gradients of 2 x 193 tokens of unit variance are clipped; bf16 ones among them are off by 2^-8 of themselves at most
    assert norm > 1 and abs(clipped - 1) <= 2.0 ** -8 + 5e-4
    for line, name in zip(lines[3:], ("prompt", "token", "train")):
        assert line.startswith(f"7B-shaped layer, {name}:") and "tokens/s" in line
