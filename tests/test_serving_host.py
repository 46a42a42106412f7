"""Host logic of the serving calls' binding (CPU only)."""
from speculative_decoding_tree_split_gb300 import _serving


class _Answers:
    """Stands for the device of a call whose library gives these answers."""
    dev = 0

    def __init__(self, *answers):
        self.answers, self.asked = list(answers), 0

    def call(self, name, *args):
        assert name == "tree_attn_workspace_size"
        self.asked += 1
        return self.answers.pop(0)


def test_a_workspace_size_is_kept_only_when_the_library_gave_one(monkeypatch):
    monkeypatch.setattr(_serving, "_WORKSPACE", {})
    at = _Answers(0, 4096, 8192)
    sizes = (2, 8, 2, 128, 4, 64)
    assert _serving._workspace_bytes(at, *sizes) == 0      # an error of that moment
    assert _serving._workspace_bytes(at, *sizes) == 4096   # is not remembered
    assert _serving._workspace_bytes(at, *sizes) == 4096 and at.asked == 2
    assert _serving._workspace_bytes(at, 3, *sizes[1:]) == 8192
