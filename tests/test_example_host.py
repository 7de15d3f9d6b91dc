"""The example's command line, as far as it runs without a GPU."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from adaln_video_dit_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("dit_block", os.path.join(ROOT, "examples", "dit_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("args", [["--dropout", "0.1"], ["--top-k", "3"], ["--experts", "0", "--dropout", "0.5"]])
def test_what_only_a_mixture_has_is_refused_without_one(example, capsys, monkeypatch, args):
    monkeypatch.setattr(example.torch, "manual_seed", lambda s: pytest.fail("ran"))
    with pytest.raises(SystemExit):
        example.main(args)
    assert args[-2] in capsys.readouterr().err
