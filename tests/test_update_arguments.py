"""Arguments of the node-update operators, checked before any launch: these tests need no GPU."""
import ctypes

import pytest

from clebsch_gordan_tensor_receiver_gb300 import uvu

A = 4096  # a pointer that nothing may follow


def refused(f, *args):
    with pytest.raises(uvu.UVUError) as e:
        f(*args)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("missing", ["gamma", "beta"])
@pytest.mark.parametrize("rows", [0, 3])
def test_group_norm_without_parameters(missing, rows):
    """The kernel reads gamma and beta for an empty batch too."""
    gamma, beta = (None if missing == n else A for n in ("gamma", "beta"))
    status, text = refused(uvu.uvu_group_norm_fwd, uvu.UVU_F32, rows, 1, rows, 8, 2, 0, 1e-5, A, A, gamma, beta, A, A, A, None, 0, None)
    assert status == 1 and f"{missing} is NULL" in text
