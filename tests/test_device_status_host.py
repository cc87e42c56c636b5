"""check_device_status() with several reports in one status word: the word is
cleared by the read, so the one exception has to name them all."""
import itertools

import pytest

import scaled_fp8_linear_gb300 as F

# by how much a report spoils: the type of the exception is the first one's
REPORTS = ((F.STATUS_TIMEOUT, F.Fp8Error, "bounded wait"), (F.STATUS_OFFSETS, ValueError, "multiples of 128"),
           (F.STATUS_NONFINITE, F.Fp8NumericsError, "non-finite"))


@pytest.mark.parametrize("reports", [c for n in (1, 2, 3) for c in itertools.combinations(REPORTS, n)])
def test_every_report_is_named(monkeypatch, reports):
    word = [sum(bit for bit, _, _ in reports)]

    def read(clear=True):
        st = word[0]
        if clear:
            word[0] = 0
        return st

    monkeypatch.setattr(F, "fp8_device_status", read)
    with pytest.raises(reports[0][1]) as e:
        F.check_device_status()
    for bit, _, words in REPORTS:
        assert (words in str(e.value)) == any(bit == b for b, _, _ in reports), str(e.value)
    assert e.value.device_status == sum(bit for bit, _, _ in reports)
    F.check_device_status()                    # read and cleared
