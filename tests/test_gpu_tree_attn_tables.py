"""The tests of attention over the paged cache once more with page tables that could hold long
contexts: the kernel is chosen by what the table can hold, so short sequences then take the
kernels of long ones."""
import pytest

import tests.test_gpu_tree_attn as base
from tests.serve_util import Paged
from tests.test_gpu_tree_attn import *  # noqa: F401,F403
from tests.test_gpu_tree_attn import _built  # noqa: F401

pytestmark = pytest.mark.gpu


class WideTable(Paged):
    def __init__(self, *args, **kw):
        kw["extra_pages"] = 20000
        super().__init__(*args, **kw)


@pytest.fixture(autouse=True)
def _wide(monkeypatch):
    monkeypatch.setattr(base, "Paged", WideTable)
