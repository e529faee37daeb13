"""When the library is built anew."""
from recsys_feature_interaction_b200 import build as wk_build


def test_other_flags_make_the_library_stale(monkeypatch):
    wk_build.build()
    assert not wk_build._stale()
    flags = wk_build.nvcc_flags()
    monkeypatch.setattr(wk_build, "nvcc_flags", lambda: flags + ["-DWK_SOMETHING=1"])
    assert wk_build._stale()
    # where the headers lie is not one of them: a copy of the tree elsewhere is as fresh as the original
    monkeypatch.setattr(wk_build, "nvcc_flags", lambda: flags + ["-I/elsewhere"])
    assert not wk_build._stale()


def test_the_command_builds_everything(monkeypatch, capsys):
    calls = []
    monkeypatch.setattr(wk_build, "build", lambda **kw: calls.append(kw) or "lib")
    wk_build.main()
    assert calls == [{"force": True}] and capsys.readouterr().out == "lib\n"
