"""CSA indexer for GB300: FP8 paged compressed-K scoring and top-k selection, and the
latent cache and attention around it.

The compute lives in the C-ABI library `libcsa_index.so` (hand-written CUDA for
sm_103a, see include/csa_index.h and include/csa_latent.h). This package holds the
thin Python bindings (`native` for the indexer, `latent` for block tables, the
latent cache and latent attention), their build step (`build`) and the seeded
synthetic workloads (`synth`). Importing the package does not load the library;
the first call into a binding does, and raises if it is missing.
"""
__all__ = ["native", "latent", "synth", "build"]
