"""The sanitizer tests skip where their drivers' sources are missing; in the
repository they are not."""
import os

import pytest

from conftest import ROOT


@pytest.mark.parametrize("name", ["abi_driver.c", "oracle_driver.c", "block_driver.cpp"])
def test_driver_is_there(name):
    assert os.path.getsize(os.path.join(ROOT, "tests", "sanitize", name)) > 0
