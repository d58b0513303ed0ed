"""The training operators' first call: what it sets up is there for the others only when it is whole
(CPU tensors: the calls end at the check for a GPU, or at the loading of the library)."""
import threading

import pytest
import torch

from delta_rule_linear_gdn2_amd import binding

X = torch.zeros(3, 16)


@pytest.fixture
def fresh(monkeypatch):
    """The binding as a new process has it."""
    monkeypatch.setattr(binding, "torch", None)
    monkeypatch.setattr(binding, "_LIB", None)
    monkeypatch.setattr(binding, "_CODES", {})


def test_every_call_says_that_the_library_is_missing(fresh, monkeypatch, tmp_path):
    load = binding.load
    monkeypatch.setattr(binding, "load", lambda: load(str(tmp_path / "libgdn2.so")))
    for _ in range(3):
        with pytest.raises(RuntimeError, match="is not built; build it with"):
            binding.gdn2_dropout(X, 0.1, 1)


def test_a_second_thread_waits_for_what_the_first_sets_up(fresh, monkeypatch):
    """A call that comes while the first one loads the library finds everything in place when it goes on."""
    load, entered, go = binding.load, threading.Event(), threading.Event()

    def slow():
        entered.set()
        assert go.wait(60)
        return load()

    monkeypatch.setattr(binding, "load", slow)
    errors = []

    def call():
        try:
            binding.gdn2_dropout(X, 0.1, 1)
        except Exception as e:
            errors.append((e, binding._LIB is not None and len(binding._CODES) == 2))

    first = threading.Thread(target=call)
    first.start()
    assert entered.wait(60)
    second = threading.Thread(target=call)
    second.start()
    second.join(0.5)  # it either waits with the first call or has gone on without the library
    go.set()
    first.join()
    second.join()
    assert len(errors) == 2
    for e, ready in errors:
        assert isinstance(e, ValueError) and "must be on a GPU" in str(e) and ready
