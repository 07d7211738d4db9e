"""The package's public names are those of its binding, at every lookup."""

import pytest


def test_a_replaced_function_is_seen_through_the_package(lib_path, monkeypatch):
    import fp8_block_scaled_04_amd as fb
    from fp8_block_scaled_04_amd import fp8bs
    for name in fb.__all__:
        assert getattr(fb, name) is getattr(fp8bs, name)
    for name in ("moe_experts_tile", "library"):
        monkeypatch.setattr(fp8bs, name, lambda: "another")
        assert getattr(fb, name)() == "another"
        monkeypatch.undo()
        assert getattr(fb, name) is getattr(fp8bs, name)
    with pytest.raises(AttributeError):
        fb.no_such_name
