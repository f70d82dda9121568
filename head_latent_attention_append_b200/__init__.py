"""B200-native multi-head latent attention on a paged latent cache.

Submodules: ``mla`` (ctypes binding over libmla's C ABI; importing it fails if
libmla.so is not built; the ragged-step calls go through the compiled module
``_ragged``), ``synth`` (seeded synthetic inputs), ``workload``
(device-resident workload setup), ``build`` (nvcc build of libmla.so, g++ build
of ``_ragged.so``).
"""
