"""Calls from several host threads on one stream share the scratch that the package keeps for it.  Each call enqueues
several operations on that scratch, so one call must have enqueued all of its own before the next begins.  Here the
library is a stand-in that says when a call is inside it (and lets other threads run meanwhile, as the real one does)."""
from __future__ import annotations

import threading
import time

import pytest
import torch

import paged_kv_cache_457_b200 as pa
from paged_kv_cache_457_b200 import build_lib, cascade, fp8


class Library:
    """Every attribute is a call: workspace sizes are 64 bytes, the others take a while and count who is inside."""

    def __init__(self):
        self.inside, self.most, self.calls = 0, 0, []

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 64

        def call(*args):
            self.inside += 1
            self.most = max(self.most, self.inside)
            self.calls.append((name, args))
            time.sleep(0.02)
            self.inside -= 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    build_lib.build()
    plan = pa.cascade_plan(2, 4, 2, 16, 32)
    lib = Library()
    monkeypatch.setattr(pa, "load_library", lambda: lib)
    monkeypatch.setattr(pa, "_stream", lambda dev: 7)
    monkeypatch.setattr(pa, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(fp8, "stream_of", lambda dev: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(pa, "_workspaces", {})
    monkeypatch.setattr(fp8, "_workspaces", {})
    lib.plan = plan
    return lib


def calls(lib):
    q = torch.zeros((2, 4, 64), dtype=torch.float16)
    cache = torch.zeros((8, 2, 16, 64), dtype=torch.float16)
    tables, ctx = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    plan = torch.from_numpy(lib.plan.plan)
    cpu = torch.device("cpu")
    return {
        "decode": lambda: pa.decode(q, cache, cache, tables, ctx, 0.1, 32),
        "cascade": lambda: cascade.decode_cascade(q, cache, cache, tables, ctx, 0.1, lib.plan, plan),
        "fp8": lambda: fp8._run(cpu, "pa_decode_fp8", lib.pa_decode_fp8_workspace_size, (), lib.pa_decode_fp8, (), None),
    }


@pytest.mark.parametrize("kinds", [("fp8", "fp8"), ("decode", "decode"), ("cascade", "cascade"),
                                   ("fp8", "decode", "cascade", "fp8")])
def test_one_call_at_a_time_on_the_kept_workspace(lib, kinds):
    failed = []

    def work(kind):
        try:
            for _ in range(3):
                calls(lib)[kind]()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in kinds]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert len(lib.calls) == 3 * len(kinds)
    assert lib.most == 1


def test_a_workspace_of_the_callers_own_is_not_waited_for(lib):
    """Such a workspace is the caller's to keep apart; the call does not queue behind others."""
    own = torch.zeros(64, dtype=torch.uint8)
    cpu = torch.device("cpu")
    threads = [threading.Thread(target=fp8._run, args=(cpu, "pa_decode_fp8", None, (), lib.pa_decode_fp8, (), own))
               for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert lib.most == 2


def test_8_bit_calls_leave_the_16_bit_calls_workspace_alone(lib, monkeypatch):
    """A captured decode graph goes on using the workspace that was kept for its stream: an 8-bit call there that needs
    a larger one neither frees it nor works in it."""
    q = torch.zeros((2, 4, 64), dtype=torch.float16)
    cache = torch.zeros((8, 2, 16, 64), dtype=torch.float16)
    tables, ctx = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    pa.decode(q, cache, cache, tables, ctx, 0.1, 32)
    ours = pa._workspaces[(None, 7)]
    used = []

    def call(*args):
        used.append(args[-3])
        return 0 if args[-2] >= 4096 else fp8.PA_ERR_WORKSPACE
    fp8._run(torch.device("cpu"), "pa_decode_fp8", lambda: 4096, (), call, (), None)
    assert pa._workspaces[(None, 7)] is ours
    assert ours.data_ptr() not in used
    pa.decode(q, cache, cache, tables, ctx, 0.1, 32)
    assert lib.calls[-1][1][-3] == ours.data_ptr()
