"""Workspaces' sizes are those of the device that is current at the call."""
import pytest

from quantized_matmul_speculative_gb300 import binding


class Library:
    """A C library on a machine whose current device changes."""

    sms = 0

    def size(self, *sizes):
        return self.sms * 1000 + sum(sizes)

    qmm_paged_attention_workspace = qmm_shared_prefix_attention_workspace = qmm_lora_workspace = size


@pytest.mark.parametrize("function,sizes", [(binding.paged_attention_workspace, (2, 3, 4, 2, 64)),
                                            (binding.shared_prefix_attention_workspace, (2, 3, 4, 2, 64)),
                                            (binding.lora_workspace, (5, 3, 16))])
def test_another_device(monkeypatch, function, sizes):
    library = Library()
    monkeypatch.setattr(binding, "lib", lambda: library)
    for library.sms in (100, 152, 100):
        assert function(*sizes) == library.sms * 1000 + sum(sizes)
