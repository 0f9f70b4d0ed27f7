"""GPU: examples/expert_layer.py runs as a user runs it, at small sizes."""
import importlib.util
import os

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "expert_layer.py")


@pytest.mark.parametrize("tokens", [1, 20, 150])
def test_expert_layer(tokens, capsys):
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    us = example.main(["--tokens", str(tokens), "--steps", "3", "--hidden", "512", "--inter", "256",
                       "--experts", "8", "--top-k", "3", "--out", "1040", "--adapters", "5", "--rank", "24"])
    assert us > 0
    assert "replays equal the eager step" in capsys.readouterr().out
