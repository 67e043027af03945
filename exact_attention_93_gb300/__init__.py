"""libfattn: exact tiled attention (FlashAttention forward with online
softmax, recompute backward) as hand-written sm_103a kernels behind a C ABI.

``exact_attention_93_gb300.fattn`` is the ctypes binding to ``libfattn.so``;
``attention`` has the autograd functions and attention over a paged cache,
``kvcache`` the cache and its tables, ``rotary`` rotary positions and norms;
``exact_attention_93_gb300.workloads`` draws seeded synthetic inputs.  Import
the submodule you need; importing the package itself loads neither, so that
drawing inputs needs no built library.
"""
