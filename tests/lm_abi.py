"""The C ABI of libpararnn_lm.so through ctypes, for the tests that call it directly."""
import ctypes
import struct

# pararnn_lm_scan, pararnn_lm_scan_grad and a pair of strides as the C compiler lays them out
SCAN = struct.Struct("@if3q3P6qPPPq")
SCAN_GRAD = struct.Struct("@6P8qPP")
PAIR = struct.Struct("@2q")


def load(path):
    lib = ctypes.CDLL(path)
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    for name, res, args in (
            ("abi_version", i32, []),
            ("scan_chunks", i64, [i64]),
            ("scan_workspace_bytes", sz, [i64, i64, i64]),
            ("gated_scan", i32, [vp, vp, vp, vp, vp, vp, sz, vp]),
            ("gated_scan_vjp", i32, [vp, vp, vp, sz, vp]),
            ("layer_norm", i32, [i32, i64, i64, vp, i64, vp, i64, vp, vp, f32, vp, i64, vp, i64, vp, vp]),
            ("layer_norm_vjp_workspace_bytes", sz, [i64, i64]),
            ("layer_norm_vjp", i32, [i32, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, vp, sz, vp]),
            ("token_logprobs_workspace_bytes", sz, [i64, i64, i32]),
            ("token_logprobs", i32, [i32, i64, i64, vp, i64, vp, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]),
            ("token_logprobs_vjp", i32, [i32, i64, i64, vp, i64, vp, i32, vp, vp, vp, vp, vp, i64, vp])):
        fn = getattr(lib, "pararnn_lm_" + name, None)      # the stress variant holds the recurrence only
        if fn is not None:
            fn.restype, fn.argtypes = res, args
    return lib
