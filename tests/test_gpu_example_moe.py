"""The mixture-of-experts example runs, and its blocks stay near the unquantized
ones (the 4-bit formats' own error; a wiring error is off by 100%)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_mixture_of_experts_example(capsys):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixture_of_experts.py")
    spec = importlib.util.spec_from_file_location("mixture_of_experts_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errs = example.main(["--d", "512", "--hidden", "256", "--experts", "16", "--prompt", "130", "--steps", "2"])
    assert len(errs) == 3 and all(e < 0.5 for e in errs)
    assert capsys.readouterr().out.count("us,") == 3
