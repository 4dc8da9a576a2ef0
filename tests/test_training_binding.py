"""CPU checks of the compiled binding: a stale one is not used."""

import pytest

torch = pytest.importorskip("torch")


def test_the_loaded_binding_matches():
    from powersgd_rank_gradient_gb300 import _lib, build, training

    library, torch_version, own = training._bind.built_with()
    assert library == _lib.lib().psgd_build_id().decode() and torch_version == torch.__version__
    assert own == "psgd-bind-hash:" + build.bind_hash()


@pytest.mark.parametrize("library,version,word", [("psgd-source-hash:other", "2.11.0", "library"), ("psgd-source-hash:a", "2.9.1", "torch")])
def test_another_library_or_torch_is_an_error(library, version, word):
    from powersgd_rank_gradient_gb300 import training

    built = ("psgd-source-hash:a", "2.11.0", "psgd-bind-hash:b")
    training._check_binding(built, *built[:2])
    with pytest.raises(RuntimeError, match=f"another {word}"):
        training._check_binding(built, library, version)
