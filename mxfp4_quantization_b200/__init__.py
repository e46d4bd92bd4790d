"""B200 (sm_100a) fused residual-add + RMSNorm + activation quantization.

`mxfp4_quantization_b200.fusednorm` is the binding of libfusednorm.so (the
kernels and their C ABI, include/fusednorm.h), `.fusedmx` that of libfusedmx.so
(the products and operators that consume MXFP4 rows, include/fusedmx.h).  They
are not imported here, so that `mxfp4_quantization_b200.synth` and `.build`
work before the libraries are built; importing one without its library raises
ImportError.
"""
__all__ = ["fusednorm", "fusedmx", "synth", "build"]
