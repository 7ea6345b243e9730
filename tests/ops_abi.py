"""The argument structures of include/gtr_ssm.h for calls of the C entry points by ctypes."""
import ctypes


class Conv(ctypes.Structure):
    """gtr_conv_t"""
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "Hgrid", "Wgrid", "D", "K", "direction", "dtype", "activation")]
                + [("x", ctypes.c_void_p), ("ldx", ctypes.c_longlong), ("w", ctypes.c_void_p),
                   ("bias", ctypes.c_void_p), ("init_state", ctypes.c_void_p)])


class Ssm(ctypes.Structure):
    """gtr_ssm_t"""
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "Hgrid", "Wgrid", "D", "S", "direction", "dtype", "dt_softplus")]
                + [(n, ctypes.c_void_p) for n in ("u", "dt", "Bm", "Cm", "z")]
                + [(n, ctypes.c_longlong) for n in ("ldu", "lddt", "ldb", "ldc", "ldz")]
                + [(n, ctypes.c_void_p) for n in ("A", "Dskip", "dt_bias", "init_state")])


class SsmGrads(ctypes.Structure):
    """gtr_ssm_grads_t"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("u", "dt", "Bm", "Cm", "z", "A", "Dskip", "dt_bias", "init_state")]
