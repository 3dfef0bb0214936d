"""CPU checks of how the context operators' calls reach the library: streams, devices and workspaces, with stand-ins for
what needs a GPU."""
import ctypes
import math
import os
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from schnet_cfconv_force_amd import binding


class Stand:
    """A tensor, a stream or the library that notes what is done to it, in order."""

    def __init__(self, name, log, raw=0, device="cuda:0", dtype=torch.uint8):
        self.name, self.log, self.cuda_stream = name, log, raw
        self.device, self.dtype = torch.device(device), dtype

    def record_stream(self, stream):
        self.log.append(("tied", self.name, stream.name))

    def wait_stream(self, other):
        self.log.append(("waits", self.name, other.name))

    def data_ptr(self):
        return 256

    def numel(self):
        return 1024

    def get_device(self):
        return -1 if self.device.index is None else self.device.index

    def is_contiguous(self):
        return True


@pytest.fixture
def world(monkeypatch):
    """A plan on cuda:0 whose current stream is 7, and an entry point that notes its stream and the current device."""
    log, state = [], SimpleNamespace(device=0)
    current = Stand("current", log, raw=7)

    def entry(*args):
        log.append(("call", args[-1], state.device))
        return state.status

    class Guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state.device = state.device, self.index

        def __exit__(self, *_):
            state.device = self.before

    state.status = 0
    monkeypatch.setattr(binding, "lib", lambda: SimpleNamespace(sn_status_string=lambda status: b"refused"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    plan = SimpleNamespace(device=torch.device("cuda:0"), index=0, byte=torch.uint8, current_stream=lambda index: 7,
                           current_device=lambda: state.device, pointers=(Stand("pointers", log),))

    def call(stream=None, **ws):
        tensors = (Stand("input", log), None, Stand("output", log))
        binding._launch(plan, entry, stream, Stand("ws", log, **ws), tensors)

    return SimpleNamespace(log=log, plan=plan, state=state, call=call)


def test_a_call_on_the_current_stream_only_launches(world):
    world.call()
    world.call(Stand("same", world.log, raw=7))
    assert world.log == [("call", 7, 0)] * 2


def test_a_call_on_another_stream_is_ordered_behind_the_current_one(world):
    """Outputs come from the current stream's memory, whose blocks its pending work may still use, and inputs and the
    workspace's zeroing may be on their way there: the stream waits first, and all tensors are tied to it."""
    world.call(Stand("side", world.log, raw=9))
    assert world.log[0] == ("waits", "side", "current")
    assert world.log[-1] == ("call", 9, 0)
    assert {e[1] for e in world.log if e[0] == "tied" and e[2] == "side"} == {"ws", "pointers", "input", "output"}


def test_a_refused_call_raises(world):
    world.state.status = binding.SN_ERR_INVALID
    with pytest.raises(binding.SnError):
        world.call()


def test_a_call_launches_on_the_plans_device(world):
    """The default stream's handle is the same on every device: the plan's has to be the current one."""
    world.state.device = 1
    world.call()
    world.call(Stand("side", world.log, raw=9))
    assert [e for e in world.log if e[0] == "call"] == [("call", 7, 0), ("call", 9, 0)]
    assert world.state.device == 1


def test_a_stream_of_another_device_is_refused(world):
    with pytest.raises(ValueError):
        world.call(Stand("side", world.log, raw=9, device="cuda:1"))
    assert not world.log


@pytest.mark.parametrize("ws", [{"device": "cpu"}, {"device": "cuda:1"}, {"dtype": torch.float32}], ids=str)
def test_a_workspace_that_the_plans_gpu_cannot_use_is_refused(world, ws):
    with pytest.raises(ValueError):
        world.call(**ws)
    assert not world.log


def test_a_plan_on_the_host_makes_no_call(world):
    world.plan.device, world.plan.index = torch.device("cpu"), None
    with pytest.raises(ValueError):
        world.call(device="cpu")
    assert not world.log


# ------------------------------------------------------------------ grids

def _lib():
    if not os.path.exists(binding.LIB_PATH):
        from schnet_cfconv_force_amd import build
        build.build(verbose=False)
    return binding.lib()


@pytest.mark.parametrize("segments,fits", [(1 << 10, True), (1 << 14, True), (1 << 16, False)])
def test_sizes_whose_grids_a_launch_cannot_hold_are_refused(segments, fits):
    """One long segment among many: 64 tiles of 128 rows and 8 heads, or 16 chunks of 16 slabs, for each of them; a
    launch has at most 2^32 threads, 2^24 blocks of 256 or 2^23 of 512."""
    lib = _lib()
    for side in ("q", "k"):
        n = {"q": (segments, 1), "k": (segments, 1), side: (segments + 8191, 8192)}
        d = binding.SnCrossAttention(segments, n["q"][0], n["k"][0], n["q"][1], n["k"][1], 256, 256, 8, 8, 32, binding.SN_BF16, 1.0,
                                     256, 256, 256, 256, 32, 256, 32, 256, 32)
        assert (lib.sn_cross_attention_workspace_bytes(ctypes.byref(d)) > 0) == fits, side
        if not fits:
            assert lib.sn_cross_attention_forward(ctypes.byref(d), 256, None, 256, 1 << 60, None) == binding.SN_ERR_INVALID
    d = binding.SnGroupNorm(segments, segments + 8191, 8192, 256, 512, 32, binding.SN_ACT_SSP, binding.SN_F32, 1e-5, 256, 512)
    assert (lib.sn_group_norm_workspace_bytes(ctypes.byref(d)) > 0) == fits
    if not fits:
        assert lib.sn_group_norm_forward(ctypes.byref(d), 256, None, None, 256, 1 << 60, None) == binding.SN_ERR_INVALID


# ------------------------------------------------------------------ thresholds of other conventions

@pytest.mark.parametrize("n_buckets,far", [(8, 20), (32, 128), (64, 128)])
def test_thresholds_of_tables_by_absolute_distance(n_buckets, far):
    """Logarithmic buckets by |rel| on both sides, one offset at a time: the thresholds above 1 lowered by one give the
    same classes, in order of rel."""
    _lib()
    half, near = n_buckets // 2, n_buckets // 4

    def by_distance(rel):
        d = abs(rel)
        j = d if d < near else min(half - 1, near + int(math.log(d / near) / math.log(far / near) * (half - near) + 1e-12))
        return half - 1 - j if rel <= 0 else half + j

    thr = binding.relative_thresholds(n_buckets, far)
    thr[thr > 1] -= 1
    rel = np.arange(-2 * far, 2 * far + 1)
    assert np.searchsorted(thr, rel, side="right").tolist() == [by_distance(int(r)) for r in rel]
