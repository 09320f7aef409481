"""Workspace sizes that the attention over shared keys keeps (CPU only, against a stand-in for the library)."""

import exact_io_aware_31_gb300 as fa


class Library:
    def __init__(self, answers):
        self.answers, self.asked = list(answers), []

    def fa_fwd_paged_shared_workspace_size(self, *args):
        self.asked.append(args)
        return self.answers.pop(0)


def test_a_size_that_could_not_be_had_is_asked_for_again(monkeypatch):
    lib = Library([0, 0, 4096, 512])
    monkeypatch.setattr(fa, "load_library", lambda: lib)
    shape = (12345, 678, 9, 8, 64, 0)             # (no other test's)
    assert [fa._shared_room(*shape) for _ in range(2)] == [0, 0]
    assert [fa._shared_room(*shape) for _ in range(3)] == [4096] * 3     # kept from then on
    assert fa._shared_room(*shape[:-1], 1) == 512                        # another device's is its own
    assert lib.asked == [shape[:-1]] * 4


def test_sizes_of_changing_batches_are_few(monkeypatch):
    lib = Library(range(256, 256 + 20000))
    monkeypatch.setattr(fa, "load_library", lambda: lib)
    for T in range(20000):
        assert fa._shared_room(50000 + T, 1, 0, 8, 64, 0) == 256 + T
    assert len(fa._shared_rooms) <= 4096
