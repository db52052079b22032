"""What the microscaled entry points and their binding refuse, at sizes that wrap around and with arguments
that contradict each other (no GPU: the checks come first)."""
from test_mx_api import FAKE, F32, lib, refused, router  # noqa: F401 (lib: a fixture)


def test_token_counts_that_wrap_around(lib):  # noqa: F811
    r = (router(), FAKE, 64, F32, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, None)
    refused(lib.gq_route, r, [(10, 1 << 27), (10, 1 << 61), (10, (1 << 61) + 1), (10, (1 << 63) - 1), (10, -1)])
