"""B200-native fused decode of lattice-rANS compressed weights.

The library (``libeptile.so``, C ABI in ``include/eptile.h``) holds the host compressor,
the stream parser and the sm_100a decode kernel; ``binding`` marshals torch tensors to
it.  Importing the package loads nothing; the first use of a binding name imports
``binding``, whose ``lib()`` fails loudly when the built library is missing.
"""
_BINDING_NAMES = ("BF16", "FP16", "FP32", "INT8", "FP8E4M3", "EpError", "compress", "compress_device", "prepare",
                  "decompress", "decompress_host", "stream_info", "lib", "StreamInfo")
# the 4-bit calls: small ones are bound by the host's 11 us, of which looking their name up took 0.6
_BINDING_CALLS = ("int4_quantize", "int4_dequantize", "int4_linear", "int4_linear_dx", "int4_scale_grad", "act8_pack",
                  "act8_unpack")


_COMPRESSED_NAMES = ("CompressedTensor", "LatticeRANSConfig", "TileANSConfig")
_LINEAR_NAMES = ("CompressedLinear", "CompressedFP8Linear", "CompressedINT8Linear", "GroupedINT4Linear")
_LINEAR_CALLS = ("int4_group_linear",)


def __getattr__(name):
    # names are looked up in their module on every use (one replaced there is replaced here), the 4-bit calls once
    if name in _BINDING_NAMES or name in _BINDING_CALLS:
        from . import binding as module
    elif name in _COMPRESSED_NAMES:
        from . import compressed as module
    elif name in _LINEAR_NAMES or name in _LINEAR_CALLS:
        from . import linear as module
    else:
        raise AttributeError(name)
    value = getattr(module, name)
    if name in _BINDING_CALLS or name in _LINEAR_CALLS:
        globals()[name] = value
    return value
