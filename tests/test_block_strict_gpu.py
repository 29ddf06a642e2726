"""Every test of test_block_gpu once more, with a comparison in which a NaN is off:
a value passes where its error is at most a finite tolerance, or where both sides
are the same infinity."""
import pytest

from tests import test_block_gpu as T
from tests.test_block_edges_gpu import within

pytestmark = pytest.mark.gpu

globals().update({name: f for name, f in vars(T).items() if name.startswith("test_")})


@pytest.fixture(autouse=True)
def _strict(monkeypatch):
    monkeypatch.setattr(T, "_within", within)
