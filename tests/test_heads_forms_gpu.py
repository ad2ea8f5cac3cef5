"""Every form of the heads' kernel against the definitions in 64 bits."""
import pytest

import layer_forms as F
import test_heads_gpu as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", F.ROPE, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("layout", ["in place", "part of a row"])
def test_rope(case, layout):
    H.test_rope(*case, layout)


@pytest.mark.parametrize("kind", F.KINDS)
@pytest.mark.parametrize("case", F.WRITE, ids=lambda c: "-".join(map(str, c)))
def test_cache_write(case, kind):
    H.test_cache_write(kind, *case)
