"""moe_operators_status loses no error that is recorded while it runs, and names both kinds."""

import threading
import time

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


def _call(bad):
    X = torch.ones(16, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(2, 64, 64, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, 20 if bad else 8, 16], dtype=torch.int32, device="cuda")
    return lambda **kw: capi.grouped_forward(X, W, offs, **kw)


def test_both_errors_are_named():
    good, bad = _call(False), _call(True)
    good()
    assert capi.operators_status() == capi.MOE_OK
    lib = capi.load()
    capi.check(lib.moe_operators_wait_limit(0), "moe_operators_wait_limit")
    try:
        good()
        bad()
        assert capi.operators_status() == capi.MOE_ERR_DEVICE_CHECK
        assert "offsets" in lib.moe_last_error().decode() and "bound" in lib.moe_last_error().decode()
    finally:
        capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
    bad()
    assert capi.operators_status() == capi.MOE_ERR_DEVICE_CHECK
    assert "bound" not in lib.moe_last_error().decode()
    assert capi.operators_status() == capi.MOE_OK


def test_an_error_recorded_meanwhile_is_reported():
    """One thread asks without a pause.  Another makes a call whose waits run out and, at some moment
    after it has ended (the first thread is then about to read and clear what it recorded), a call with
    bad offsets on another stream, which has to be reported as well."""
    good, bad = _call(False), _call(True)
    lib, first, second = capi.load(), torch.cuda.Stream(), torch.cuda.Stream()
    out = [good(), bad()]
    torch.cuda.synchronize()
    capi.operators_status()
    reports, stop = {capi.MOE_OK: 0, capi.MOE_ERR_TIMEOUT: 0, capi.MOE_ERR_DEVICE_CHECK: 0}, threading.Event()

    def ask():
        while not stop.is_set():
            reports[capi.operators_status()] += 1

    thread = threading.Thread(target=ask)
    thread.start()
    lost, ended = 0, torch.cuda.Event()
    try:
        for i in range(400):
            before = reports[capi.MOE_ERR_DEVICE_CHECK]
            capi.check(lib.moe_operators_wait_limit(0), "moe_operators_wait_limit")
            good(out=out[0], stream=first)
            capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
            ended.record(first)
            while not ended.query():
                pass
            due = time.perf_counter() + (i % 80) * 0.5e-6
            while time.perf_counter() < due:
                pass
            bad(out=out[1], stream=second)
            limit = time.monotonic() + 0.25  # of some 30 us a call
            while reports[capi.MOE_ERR_DEVICE_CHECK] == before and time.monotonic() < limit:
                time.sleep(0)
            lost += reports[capi.MOE_ERR_DEVICE_CHECK] == before
            if lost > 3:
                break
    finally:
        capi.check(lib.moe_operators_wait_limit(-1), "moe_operators_wait_limit")
        stop.set()
        thread.join()
    assert lost == 0
    assert capi.operators_status() == capi.MOE_OK
