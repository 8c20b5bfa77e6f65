"""hsl_mx_check: it takes the report and clears it in one step, behind the work of its own stream and no other."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hsl():
    from sparse_rank_linear_03_b200 import hsl as mod
    return mod


def test_the_check_waits_for_its_own_stream_only(hsl):
    hsl.mx_check()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    before, after = torch.cuda.Event(), torch.cuda.Event()
    before.record()
    torch.cuda._sleep(2_000_000_000)                     # about a second of the default stream
    after.record()
    hsl.mx_check(stream=s)
    assert not after.query()
    torch.cuda.synchronize()
    assert before.query() and after.query()


def test_a_report_is_given_once(hsl, monkeypatch):
    """HSL_FAULT_INJECT=mxwait: the check finds what a wait that gave up leaves behind."""
    hsl.mx_check()
    monkeypatch.setenv("HSL_FAULT_INJECT", "mxwait")
    for stream in (None, torch.cuda.Stream()):
        with pytest.raises(hsl.HslError) as e:
            hsl.mx_check(stream=stream)
        assert e.value.name == "HSL_ERR_TIMEOUT"
    monkeypatch.delenv("HSL_FAULT_INJECT")
    hsl.mx_check()


def test_checks_from_many_threads(hsl):
    """Each takes and clears by itself; none finds a report where there is none."""
    found = []

    def run():
        s = torch.cuda.Stream()
        for _ in range(200):
            try:
                hsl.mx_check(stream=s)
            except Exception as e:                       # noqa: BLE001
                found.append(e)
    threads = [threading.Thread(target=run) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not found
