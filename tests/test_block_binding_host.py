"""Host-only checks of the block operators' binding: what it hands to the library, and what it refuses."""
import copy
import dataclasses
import pickle

import pytest
import torch

import tile_level_copy_gb300 as tlc


class Library:
    """Stands for the loaded library: `on` maps an entry point to a function, the others return MOE_OK."""

    def __init__(self, **on):
        self.on, self.calls = on, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return self.on[name](*args) if name in self.on else tlc.MOE_OK
        return call


def test_adamw_step_hands_over_its_own_step(monkeypatch):
    """Another thread steps with the same config while the call of this one is under way (the call releases
    the interpreter's lock): made here by a step from within the call."""
    cfg, seen = tlc.AdamWConfig(lr=1e-3), []
    lst = tlc.AdamWList(cfg, [], [], [], [])

    def step(ref, *_):
        if not seen:
            seen.append(None)
            tlc.adamw_step(cfg, lst, 9, stream=0)
        seen.append(ref._obj.step)
        return tlc.MOE_OK

    monkeypatch.setattr(tlc, "lib", lambda: Library(moe_adamw_step=step))
    tlc.adamw_step(cfg, lst, 5, stream=0)
    assert seen == [None, 9, 5]
    assert cfg.ref()[1].step == 1  # the config's own struct stays as it was made


@pytest.mark.parametrize("cfg", [tlc.FFNConfig(4, 128, 256), tlc.LayerNormConfig(4, 64), tlc.AdamWConfig(lr=1e-3, seed=7)],
                         ids=lambda c: type(c).__name__)
def test_a_used_config_is_copied_and_pickled(built_library, cfg):
    cfg.ref()
    for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), dataclasses.replace(cfg)):
        assert other == cfg and type(other) is type(cfg)
        assert other.ref()[1] is not cfg.ref()[1]  # a C form of its own
        assert bytes(other.ref()[1]) == bytes(cfg.ref()[1])
