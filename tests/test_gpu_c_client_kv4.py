"""The plain C client of the rotary positions, the 4-bit cache and its
attention (tests/c_client_kv4.c, built by __graft_entry__.build()) on the GPU."""
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

CLIENT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "gq_c_client_kv4")


def test_c_client_kv4():
    assert os.path.exists(CLIENT), "tests/gq_c_client_kv4 is built by __graft_entry__.build()"
    print("[c client] running tests/gq_c_client_kv4", flush=True)
    r = subprocess.run([CLIENT], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "c client ok" in r.stdout
