"""GB300 (sm_103a) speculative-decoding verify step of one Gated DeltaNet layer.

* ``gdn``      - ctypes binding of the C ABI in include/gdn.h (libgdn_sm103a.so)
* ``runtime``  - device buffers of one layer and the verify -> rollback round
* ``kv``       - ctypes binding of the paged key/value cache, of rotation and of prompts (include/gdn_kv.h)
* ``kv_runtime`` - device buffers of a paged cache and its part of the round and of prompts
* ``rope``     - frequencies of rotary positions
* ``synth``    - seeded synthetic inputs of the named workloads
* ``build``    - in-tree nvcc build of the library for sm_103a

Importing the package loads nothing; ``gdn.load_library()`` (called by every
binding function) raises if the library has not been built.
"""
