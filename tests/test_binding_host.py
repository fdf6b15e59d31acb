"""How the binding takes its arguments' addresses. No GPU."""
import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk


def test_addresses_of_what_may_be_passed():
    t = torch.zeros(4)
    a = np.zeros(4)
    assert pk._ptr(None) is None and pk._ptr(5) == 5
    assert pk._ptr(t) == t.data_ptr() and pk._ptr(a) == a.ctypes.data
    for x in ("text", 1.5, object()):
        with pytest.raises(TypeError):
            pk._ptr(x)


def test_an_error_inside_data_ptr_reaches_the_caller():
    """An object that has data_ptr is asked for it once; an AttributeError from inside is
    not taken for its absence."""
    class Lazy:
        ctypes = np.zeros(1).ctypes

        def data_ptr(self):
            return self.storage.address  # never set

    with pytest.raises(AttributeError, match="storage"):
        pk._ptr(Lazy())
