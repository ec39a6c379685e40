"""The example layer trains, prefills and decodes on the GPU (its own checks are in it)."""
import os
import runpy

import pytest

pytestmark = pytest.mark.gpu


def test_linear_attention_layer(capsys):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "linear_attention_layer.py")
    runpy.run_path(path)["main"]()
    assert "ok" in capsys.readouterr().out
