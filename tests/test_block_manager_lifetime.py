"""A block manager's memory goes back to the library that it came from."""


def test_destroyed_by_its_library(monkeypatch):
    """Whenever it is collected: also while the module's library is another one."""
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_03_gb300 as pkv
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0
    bm = pkv.BlockManager(8)
    assert bm.allocate(0, 20)
    monkeypatch.setattr(pkv, "_L", Lib())
    del bm
    assert made == []
