"""A compile that succeeds shows what ptxas says about spilled registers."""
import stat

from paged_kv_cache_70_gb300 import build as B


def test_spills_are_shown_and_other_output_is_not(tmp_path, monkeypatch, capsys):
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\necho "ptxas warning : Registers are spilled in x" >&2\n'
                    'echo "note: something else" >&2\n'
                    'while [ "$1" != -o ]; do shift; done\ntouch "$2"\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(B, "_nvcc", lambda: str(nvcc))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "out" / "libpagedkv.so"))
    B.build()
    err = capsys.readouterr().err
    assert err.count("Registers are spilled") == len(B.sources())
    assert "something else" not in err
