"""B200-native fused decode of lattice-rANS compressed weights.

The library (``libeptile.so``, C ABI in ``include/eptile.h``) holds the host compressor,
the stream parser and the sm_100a decode kernel; ``binding`` marshals torch tensors to
it.  Importing the package loads nothing; the first use of a binding name imports
``binding``, whose ``lib()`` fails loudly when the built library is missing.
"""
import importlib
import sys

_BINDING_NAMES = ("BF16", "FP16", "FP32", "INT8", "FP8E4M3", "EpError", "compress", "compress_device", "prepare",
                  "decompress", "decompress_host", "stream_info", "lib", "StreamInfo", "int4_quantize",
                  "int4_dequantize", "int4_linear", "int4_linear_dx", "int4_scale_grad", "act8_pack", "act8_unpack")


_COMPRESSED_NAMES = ("CompressedTensor", "LatticeRANSConfig", "TileANSConfig")
_LINEAR_NAMES = ("CompressedLinear", "CompressedFP8Linear", "CompressedINT8Linear", "GroupedINT4Linear",
                 "int4_group_linear")


_HOME = {name: __name__ + "." + module
         for module, names in (("binding", _BINDING_NAMES), ("compressed", _COMPRESSED_NAMES), ("linear", _LINEAR_NAMES))
         for name in names}


def __getattr__(name):
    home = _HOME.get(name)
    if home is None:
        raise AttributeError(name)
    # looked up in its module each time (0.3 us), so that a name replaced there is replaced here
    return getattr(sys.modules.get(home) or importlib.import_module(home), name)
