"""The build and smoke entry points."""
import os
import runpy

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ENTRY = os.path.join(ROOT, "__graft_entry__.py")


@pytest.mark.parametrize("argv", [[], ["--smoke"]])
def test_run_as_a_script(argv, monkeypatch):
    # with nothing to build and no GPU to run on: build() first, then smoke() where it is asked
    # for, up to its first step on the device
    from oracle import c_oracle
    from vocabulary_cross_entropy_gb300 import build
    import workloads

    class Reached(Exception):
        pass

    def reached(*args):
        raise Reached

    built = []
    monkeypatch.setattr(build, "build", lambda *a, **k: built.append("library"))
    monkeypatch.setattr(c_oracle, "build", lambda *a, **k: built.append("oracle"))
    monkeypatch.setattr(workloads, "normal_matrix", reached)
    monkeypatch.setattr("vocabulary_cross_entropy_gb300.library", lambda: None)
    monkeypatch.setattr("sys.argv", [ENTRY, *argv])
    if argv:
        with pytest.raises(Reached):
            runpy.run_path(ENTRY, run_name="__main__")
        assert built == ["library", "oracle", "library"]
    else:
        runpy.run_path(ENTRY, run_name="__main__")
        assert built == ["library", "oracle"]


@pytest.mark.gpu
def test_smoke_covers_the_output_head(capsys, monkeypatch):
    import vocabulary_cross_entropy_gb300 as vce
    called = set()
    for name in ("linear_cross_entropy", "rms_norm_forward", "rms_norm_mx", "mx_quantize", "mx_dequantize",
                 "linear_sample"):
        def noted(*a, _fn=getattr(vce, name), _name=name, **k):
            called.add(_name)
            return _fn(*a, **k)
        monkeypatch.setattr(vce, name, noted)
    runpy.run_path(ENTRY)["smoke"]()
    assert capsys.readouterr().out.endswith("smoke ok\n")
    assert len(called) == 6, called
