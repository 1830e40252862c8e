"""Which device a call's stream belongs to, without a GPU."""
import pytest


def test_one_device_is_the_current_one(monkeypatch):
    """Where a process sees one device, calls do not ask which is current; where it
    sees several, device 0 is compared like the others."""
    import block_quantized_matmul_repack_amd as tq
    from block_quantized_matmul_repack_amd import ops
    asked = []
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(ops, "_current_device", lambda: asked.append(0) or 1)
    monkeypatch.setattr(ops, "_several_devices", lambda: False)
    assert ops._stream_of(0) == 0 and not asked
    monkeypatch.setattr(ops, "_several_devices", lambda: True)
    with pytest.raises(tq.TiledqError, match="current"):
        ops._stream_of(0)
    assert ops._stream_of(1) == 0 and len(asked) == 2
