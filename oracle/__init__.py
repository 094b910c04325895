"""CPU oracle of the SLoPe 2:4 sparse linear layer (test infrastructure only).

Only the test suite, the entry module's smoke check and the benchmark's CPU
baseline may import this package.  It shares no code with the GPU library.
"""
from .slope_ref import *  # noqa: F401,F403
from .slope_ref import __all__ as _slope_all
from .int8_ref import *  # noqa: F401,F403
from .int8_ref import __all__ as _int8_all
from .mx_ref import *  # noqa: F401,F403
from .mx_ref import __all__ as _mx_all

__all__ = [*_slope_all, *_int8_all, *_mx_all]
