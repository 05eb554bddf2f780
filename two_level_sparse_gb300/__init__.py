"""GB300 (sm_103a) two-level candidate sparse-attention indexer.

``two_level_sparse_gb300.ci`` binds the C ABI of ``libci.so`` (declared in
``include/ci.h``); ``two_level_sparse_gb300.cache`` binds the paged key-value
cache beside it (``include/ci_cache.h``: attention, norm + rotation + append,
pages) and ``two_level_sparse_gb300.paged`` puts its calls together;
``two_level_sparse_gb300.synth`` draws seeded synthetic
inputs.  Importing the package itself loads nothing.
"""
