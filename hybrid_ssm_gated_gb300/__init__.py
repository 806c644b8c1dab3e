"""GB300-native GDN (Gated DeltaNet) recurrent-state decode library.

The compute path is a C-ABI shared library of hand-written CUDA kernels for
sm_103a (include/gdn.h; include/kv.h for the attention layers' cache);
`hybrid_ssm_gated_gb300.gdn` and `hybrid_ssm_gated_gb300.kv` are its thin ctypes
bindings. `hybrid_ssm_gated_gb300.workload` draws the seeded synthetic inputs.
"""
__all__ = ["gdn", "kv", "workload"]
