"""The host code of the operators around the routed experts under AddressSanitizer
(tests/asan/layer_host_checks.c, built as in test_host_asan.py)."""
from test_host_asan import _driver, asan_objects, pytestmark  # noqa: F401


def test_layer_host_checks_under_address_sanitizer(asan_objects):   # noqa: F811
    r = _driver(asan_objects, "layer_host_checks")
    assert "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "all passed" in r.stdout
