"""The layer's steps on a stream of a device that is not the current one.  On the CPU: nothing is launched."""
import types

import pytest

from tests.test_kv4_binding import Elsewhere
from tests.test_layer_binding import calls_of, launched  # noqa: F401


def test_a_stream_of_a_device_that_is_not_current_is_refused(launched):  # noqa: F811
    """A launch would fail there, and leave its error to whatever asks the device next."""
    away = types.SimpleNamespace(cuda_stream=77, device_index=1)
    for call, args in calls_of():
        launched.clear()
        with pytest.raises(ValueError, match="current"):
            call(*[t.as_subclass(Elsewhere) for t in args], stream=away)
        assert launched == []
