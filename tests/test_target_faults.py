"""The target's side of a step without a GPU: refusals at the ends of its arguments' ranges (nothing is
launched), and the module that checks its calls in C where that cannot be built or loaded."""
import math
import os
import sysconfig

import pytest

from speculative_decoding_03_gb300 import _build, target
from test_target_abi import INVALID, OK, attend


def test_attention_of_scales_at_the_end_of_fp32():
    """Scores are formed times scale log2(e): a scale for which that is infinite makes a score of 0 NaN."""
    nothing = dict(B=0, rows=0, pages=None, lengths=None, q=None, out=None)
    most = (2.0 ** 128 - 2.0 ** 103) * math.log(2.0)            # what rounds to the largest number
    assert attend(**nothing, scale=most * (1 - 2.0 ** -20)) == OK
    for scale in (most * (1 + 2.0 ** -20), 3.0e38, (2.0 - 2.0 ** -23) * 2.0 ** 127):
        assert attend(**nothing, scale=scale) == INVALID, scale
    assert attend(**nothing, scale=2.0 ** -149) == OK


# ------------------------------------------------- the module that checks calls in C

def test_the_module_is_named_after_the_interpreter():
    """It is compiled against the interpreter's own C API, so another interpreter does not find it."""
    assert os.path.basename(_build.CALLS) == "_dspark_calls" + sysconfig.get_config_var("EXT_SUFFIX")


def test_the_library_is_built_without_the_module(monkeypatch, tmp_path):
    """Without Python's headers, or a compiler, the module is left out with a warning, an older one too."""
    _build.build()
    old = tmp_path / "calls.so"
    monkeypatch.setattr(_build, "CALLS", str(old))
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    old.write_bytes(b"")
    with pytest.warns(RuntimeWarning, match="not built"):
        assert not _build.build_calls(force=True)
    assert not old.exists()
    with pytest.warns(RuntimeWarning, match="not built"):
        assert _build.build() == _build.LIB
    monkeypatch.setattr(_build.shutil, "which", lambda name: str(tmp_path / "no compiler"))
    with pytest.warns(RuntimeWarning, match="not built"):
        assert not _build.build_calls()
    assert target._module() is None


def test_a_module_that_cannot_be_loaded_is_left_out(monkeypatch, tmp_path):
    bad = tmp_path / "calls.so"
    bad.write_bytes(b"not a module")
    monkeypatch.setattr(_build, "CALLS", str(bad))
    with pytest.warns(RuntimeWarning, match="cannot be loaded"):
        assert target._module() is None


def test_only_a_stale_module_is_built_again(monkeypatch, tmp_path):
    mine = tmp_path / "calls.so"
    monkeypatch.setattr(_build, "CALLS", str(mine))
    assert _build.build_calls() and mine.exists()
    when = os.path.getmtime(mine)
    os.utime(mine, (when + 100, when + 100))
    assert _build.build_calls() and os.path.getmtime(mine) == when + 100
    os.utime(mine, (0, 0))
    assert _build.build_calls() and os.path.getmtime(mine) > 0
