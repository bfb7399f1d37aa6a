"""fp64 CPU oracle: test infrastructure, not part of the library.

Only ``tests/``, ``__graft_entry__.smoke()`` and the CPU-baseline leg of
``bench.py`` may import this package. The CUDA path never does. See
``oracle/attention.py`` (attention over a paged cache, prefill, merges) and
``oracle/flat_gemm.py`` (the decode-phase flat GEMM) for the definitions and the
passages they follow, and ``oracle/cache_ops.py`` for the operators around them (cache
write, accumulated weights, eviction, linear layer).
"""
from .attention import *  # noqa: F401,F403
from .attention import __all__ as _attention_all
from .flat_gemm import *  # noqa: F401,F403
from .flat_gemm import __all__ as _flat_gemm_all
from .cache_ops import *  # noqa: F401,F403
from .cache_ops import __all__ as _cache_ops_all

__all__ = list(_attention_all) + list(_flat_gemm_all) + list(_cache_ops_all)
