import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_sessionstart(session):
    """Build what is not there: the library, or the Python entry beside it."""
    from moe_expert_ffn_route_amd import build
    if not (os.path.exists(build.LIB) and os.path.exists(build.PYCALL)):
        build.build()


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
