"""The binding's compiled argument helper is optional: the library builds without a C++ compiler for it, and a helper
that was built against another PyTorch is not used."""
import pytest


@pytest.mark.parametrize("cxx", ["/bin/false", "/nonexistent/c++"])
def test_library_builds_without_the_helper(cxx, tmp_path, monkeypatch):
    from gated_delta_rule_07_amd import build as b
    stale, linked = tmp_path / "_kda_args.so", []
    stale.write_bytes(b"an earlier build")
    monkeypatch.setenv("CXX", cxx)
    monkeypatch.setattr(b, "PKG", tmp_path)
    monkeypatch.setattr(b, "ARGS_HELPER", stale, raising=False)
    monkeypatch.setattr(b, "_compile", lambda src, verbose, defines=(): tmp_path / src)
    monkeypatch.setattr(b, "_link", lambda objs, lib, verbose: linked.append(lib))
    with pytest.warns(UserWarning, match="argument helper"):
        assert b.build() == b.LIB
    assert linked == [b.LIB, b.TEST_LIB]
    assert not stale.exists(), "a helper of an earlier build is left to be loaded"


def test_a_helper_of_another_pytorch_is_not_used(monkeypatch):
    import torch

    import gated_delta_rule_07_amd as kda
    helper = pytest.importorskip("gated_delta_rule_07_amd._kda_args")
    assert helper.torch_version == torch.__version__
    assert kda._argument_forms() == (helper.need, helper.rows)
    monkeypatch.setattr(helper, "torch_version", "1.0")
    need, rows = kda._argument_forms()
    assert need is kda._need_in_words and rows(None, torch.float32, 0) is None
    monkeypatch.delattr(helper, "torch_version")  # (a build that does not say)
    assert kda._argument_forms()[0] is kda._need_in_words
