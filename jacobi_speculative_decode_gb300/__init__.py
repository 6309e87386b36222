"""GB300-native XPress Jacobi refinement pass, and the target's side of its step: attention
over a paged cache, verification of the drafts, the cache's pages.

The compute path is the CUDA library ``libxp.so`` (hand-written sm_103a
kernels behind a C ABI declared in ``include/xp.h``); ``xp`` is its thin
ctypes binding and ``inputs`` the seeded synthetic-input generator.
"""
