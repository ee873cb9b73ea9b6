"""The compiled marshalling module is rebuilt for another PyTorch or Python
(no GPU needed)."""
import torch

from mxfp8_moe_quantization_gb300 import build as B


def test_binding_of_another_installation_is_stale(tmp_path, monkeypatch):
    B.build()
    assert B.up_to_date()
    own = B._made_for()
    assert torch.__version__ in own
    monkeypatch.setattr(B, "STAMP", str(tmp_path / "stamp"))
    assert not B.up_to_date()                                  # made by nobody knows what
    (tmp_path / "stamp").write_text(own)
    assert B.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.0")         # another PyTorch in the same place
    assert not B.up_to_date()
    monkeypatch.undo()
    monkeypatch.setattr(B, "STAMP", str(tmp_path / "stamp"))
    (tmp_path / "stamp").write_text(own.replace(B._torch_dir(), "/elsewhere"))
    assert not B.up_to_date()
