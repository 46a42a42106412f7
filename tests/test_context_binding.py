"""The binding keeps nothing that grows with the sizes a server has had (CPU only)."""
import speculative_decoding_tree_split_gb300 as ta
from speculative_decoding_tree_split_gb300 import _pages


class Place:
    """A device whose library wants no workspace."""

    dev, stream = 0, None
    calls = 0

    def call(self, name, *sizes):
        Place.calls += 1
        return 0


def test_sizes_of_workspaces_are_not_kept_without_end():
    assert callable(ta.kv_fork)
    at = Place()

    def held():
        kept = sum(len(x) for x in vars(_pages).values() if isinstance(x, dict))
        return kept + sum(f.cache_info().currsize for f in vars(_pages).values()
                          if hasattr(f, "cache_info"))
    before = held()
    for n in range(20000):
        assert _pages._workspace(None, at, "tree_kv_fork_workspace_size", n, n + 1, 4096) is None
    assert held() - before <= 1024
